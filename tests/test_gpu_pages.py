"""Upkeep of the pages on the GPU, against a plain model that works through the pairs one by one."""
import random

import pytest
import torch

from kv_indexing_b200 import lsa as L
from tests.paged_ref import ints

pytestmark = pytest.mark.gpu


class Model:
    """Table, counts and lengths as Python lists; a pool's page as the number it was filled with."""

    def __init__(self, S, max_pages, n_pages, P):
        self.S, self.M, self.N, self.P = S, max_pages, n_pages, P
        self.table = [[-1] * max_pages for _ in range(S)]
        self.ref, self.len, self.data = [0] * n_pages, [0] * S, list(range(n_pages))

    def lowest(self):
        return next((p for p in range(self.N) if self.ref[p] <= 0), None)

    def reserve(self, lens):
        ok = True
        for s, n in enumerate(lens):
            for j in range(min(self.M, (n + self.P - 1) // self.P)):
                if self.table[s][j] < 0:
                    p = self.lowest()
                    if p is None:
                        ok = False
                        continue
                    self.table[s][j], self.ref[p] = p, 1
        return ok

    def free(self, seqs):
        for s in seqs:
            for p in self.table[s]:
                if p >= 0:
                    self.ref[p] -= 1
            self.table[s], self.len[s] = [-1] * self.M, 0

    def fork(self, parent, child):
        ok, good = True, []
        for i, (p, c) in enumerate(zip(parent, child)):
            inside = 0 <= p < self.S and 0 <= c < self.S
            if not inside or c in child[:i] or p in [x for x in child if 0 <= x < self.S]:
                ok = False
            else:
                good.append((p, c))
        old = [list(r) for r in self.table]
        fresh = []
        for p, c in good:
            tail = self.len[p] % self.P > 0
            q = self.lowest() if tail else None
            if tail and q is not None:
                self.ref[q] = 1
            fresh.append((tail, q))
        for (p, c), (tail, q) in zip(good, fresh):
            full = self.len[p] // self.P
            self.table[c] = old[p][:full] + [-1] * (self.M - full)
            for e in old[p][:full]:
                self.ref[e] += 1
            self.len[c] = self.len[p]
            if tail and q is None:
                self.len[c], ok = full * self.P, False
            elif tail:
                self.table[c][full] = q
                self.data[q] = self.data[old[p][full]]
        return ok

    def compact(self):
        n = sum(r > 0 for r in self.ref)
        holes = iter([p for p in range(n) if self.ref[p] <= 0])
        to = {p: next(holes) for p in range(n, self.N) if self.ref[p] > 0}
        old = list(self.ref)
        for a, b in to.items():
            self.ref[b], self.ref[a], self.data[b] = old[a], 0, self.data[a]
        self.table = [[to.get(e, e) for e in row] for row in self.table]
        return n


class Device:
    def __init__(self, m, n_pools=2):
        self.m = m
        self.table, self.ref = torch.tensor(m.table, dtype=torch.int32, device="cuda"), ints(m.ref)
        self.len = ints(m.len)
        self.pools = []
        for i in range(n_pools):
            width = (8, 24, 576)[i % 3]
            dt = (torch.float32, torch.bfloat16, torch.uint8)[i % 3]
            store = torch.zeros(m.N, 2, m.P, width, device="cuda", dtype=dt)    # every other block of a wider pool
            pool = store[:, 0]
            pool.copy_(((torch.arange(m.N, device="cuda") + i) % 251).to(dt)[:, None, None].expand(m.N, m.P, width))
            self.pools.append(pool)

    def check(self):
        m = self.m
        assert self.table.tolist() == m.table
        assert self.ref.tolist() == m.ref
        assert self.len.tolist() == m.len
        for i, pool in enumerate(self.pools):
            want = ((torch.tensor(m.data, device="cuda") + i) % 251).to(pool.dtype)
            assert torch.equal(pool, want[:, None, None].expand_as(pool))


def script(seed, S, M, N, P, n_pools, steps=12):
    rng = random.Random(seed)
    m = Model(S, M, N, P)
    d = Device(m, n_pools)
    for _ in range(steps):
        what = rng.choice(["reserve", "reserve", "free", "fork", "fork", "compact"])
        if what == "reserve":
            lens = [min(M * P, n + rng.choice([0, 0, 1, P, rng.randint(0, 3 * P)])) for n in m.len]
            ok = m.reserve(lens)
            L.lsa_pages_reserve(d.table, d.ref, ints(lens), P)
            m.len = [min(n, P * sum(e >= 0 for e in r)) for n, r in zip(lens, m.table)]
            d.len.copy_(ints(m.len))
        elif what == "free":
            seqs = [rng.randrange(S) for _ in range(rng.randint(1, S))]         # repeats among them
            m.free(dict.fromkeys(seqs))
            ok = True
            L.lsa_pages_free(d.table, d.ref, d.len, ints(seqs))
        elif what == "fork":
            kids = rng.sample(range(S), rng.randint(1, max(1, S // 2)))
            rest = [s for s in range(S) if s not in kids] or kids
            m.free(kids)
            L.lsa_pages_free(d.table, d.ref, d.len, ints(kids))
            par = [rng.choice(rest) for _ in kids]
            ok = m.fork(par, kids)
            L.lsa_pages_fork(d.table, d.ref, d.len, P, ints(par), ints(kids), d.pools)
        else:
            ok = True
            n = m.compact()
            got = L.lsa_pages_compact(d.table, d.ref, d.pools)
            assert got[0] is d.table and got[1] is d.ref and got[2].tolist() == [n]
        if ok:
            assert L.lsa_device_status() == 0
        else:
            with pytest.raises(L.LsaError):
                L.lsa_device_status()
        d.check()


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("S,M,N,P,n_pools", [(1, 1, 1, 16, 1), (5, 9, 33, 16, 2), (7, 40, 64, 32, 3), (40, 65, 1000, 128, 1),
                                             (9, 2100, 5000, 16, 2), (3, 33, 31, 64, 0)])
def test_scripts(seed, S, M, N, P, n_pools):
    script(seed, S, M, N, P, n_pools)


def test_more_pools_than_one_launch_takes():
    script(5, 4, 6, 20, 16, 70, steps=8)


def test_many_sequences():
    """More sequences than a block has threads, and a planning table in more than 48 KB of shared memory."""
    S, P = 8192, 16
    m = Model(S, 3, 3 * S, P)
    d = Device(m, 0)
    lens = [(7 * s) % 40 for s in range(S)]
    want, at, table = [], 0, []
    for n in lens:
        k = (n + P - 1) // P
        table.append(list(range(at, at + k)) + [-1] * (3 - k))
        at += k
    L.lsa_pages_reserve(d.table, d.ref, ints(lens), P)
    assert d.table.tolist() == table and d.ref.tolist() == [1] * at + [0] * (3 * S - at)
    d.len.copy_(ints(lens))
    par, kids = list(range(0, S, 2)), list(range(1, S, 2))
    L.lsa_pages_free(d.table, d.ref, d.len, ints(kids))
    L.lsa_pages_fork(d.table, d.ref, d.len, P, ints(par), ints(kids), [])
    assert L.lsa_device_status() == 0
    t, ref = d.table.tolist(), d.ref.tolist()
    assert d.len.tolist() == [lens[s - s % 2] for s in range(S)]
    counts = [0] * (3 * S)
    for r in t:
        for e in r:
            if e >= 0:
                counts[e] += 1
    assert counts == ref
    for s in range(0, S, 2):
        full = lens[s] // P
        assert t[s][:full] == t[s + 1][:full] and (lens[s] % P == 0 or t[s][full] != t[s + 1][full])


def test_refused_pairs_and_ids():
    m = Model(6, 4, 40, 16)
    d = Device(m, 1)
    m.reserve([40, 20, 0, 0, 0, 0])
    L.lsa_pages_reserve(d.table, d.ref, ints([40, 20, 0, 0, 0, 0]), 16)
    m.len = [40, 20, 0, 0, 0, 0]
    d.len.copy_(ints(m.len))
    # out of range, the same child twice, a parent that is a child of the call, its own parent
    par, kids = [0, 6, -1, 1, 0, 2, 1, 5], [2, 3, 3, 7, 2, 4, -1, 5]
    assert not m.fork(par, kids)
    L.lsa_pages_fork(d.table, d.ref, d.len, 16, ints(par), ints(kids), d.pools)
    with pytest.raises(L.LsaError, match="refused"):
        L.lsa_device_status()
    d.check()
    L.lsa_pages_free(d.table, d.ref, d.len, ints([-1, 6, 2, 2]))
    m.free([2])
    with pytest.raises(L.LsaError):
        L.lsa_device_status()
    d.check()
    # a length past the table is clamped, and reported
    m.reserve([65, 0, 0, 0, 0, 0])
    L.lsa_pages_reserve(d.table, d.ref, ints([65, -3, 0, 0, 0, 0]), 16)
    with pytest.raises(L.LsaError):
        L.lsa_device_status()
    d.check()
    # a table entry past the pool, a page whose count is 0 already
    d.table[3, 0], d.table[4, 0] = 40, 39
    L.lsa_pages_free(d.table, d.ref, d.len, ints([3, 4]))
    with pytest.raises(L.LsaError):
        L.lsa_device_status()
    d.check()


def test_no_pages_left():
    m = Model(3, 8, 6, 16)
    d = Device(m, 1)
    m.reserve([70, 0, 0])
    L.lsa_pages_reserve(d.table, d.ref, ints([70, 0, 0]), 16)
    m.len = [70, 0, 0]
    d.len.copy_(ints(m.len))
    assert not m.fork([0, 0], [1, 2])                      # one page is left for two partly filled ones
    L.lsa_pages_fork(d.table, d.ref, d.len, 16, ints([0, 0]), ints([1, 2]), d.pools)
    with pytest.raises(L.LsaError, match="ran out"):
        L.lsa_device_status()
    d.check()
    assert not m.reserve([71, 100, 0])
    L.lsa_pages_reserve(d.table, d.ref, ints([71, 100, 0]), 16)
    with pytest.raises(L.LsaError, match="ran out"):
        L.lsa_device_status()
    d.check()


@pytest.mark.parametrize("past", [1, 15, 16, 4096])
def test_fork_of_a_length_past_the_table(past):
    """The child gets what the parent's row holds, and the length is reported, whole pages past it or not."""
    m = Model(3, 4, 12, 16)
    d = Device(m, 1)
    m.reserve([64, 0, 0])
    L.lsa_pages_reserve(d.table, d.ref, ints([64, 0, 0]), 16)
    m.len = [64, 0, 0]
    assert m.fork([0], [2])
    d.len.copy_(ints([64 + past, 0, 0]))
    L.lsa_pages_fork(d.table, d.ref, d.len, 16, ints([0]), ints([2]), d.pools)
    with pytest.raises(L.LsaError, match="out of range"):
        L.lsa_device_status()
    m.len[0] += past
    d.check()


def test_reserving_more_pages_than_32_bits_count():
    """8192 rows that want 2^18 pages each: the first row takes what there is, and the rest is reported."""
    S, M = 8192, 1 << 18
    table = torch.full((S, M), -1, dtype=torch.int32, device="cuda")
    ref = torch.zeros(64, dtype=torch.int32, device="cuda")
    ref[5] = 1
    L.lsa_pages_reserve(table, ref, torch.full((S,), 16 * M, dtype=torch.int32, device="cuda"), 16)
    with pytest.raises(L.LsaError, match="ran out"):
        L.lsa_device_status()
    assert ref.tolist() == [1] * 64
    assert table[0, :64].tolist() == list(range(5)) + list(range(6, 64)) + [-1]
    assert int((table >= 0).sum()) == 63


@pytest.mark.parametrize("n_pages,n", [(2, 1), (33, 5), (2000, 700), (2100, 1025), (1 << 19, 2000)])
def test_copy(n_pages, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    src, dst = perm[:n].clone(), perm[n_pages - n:].clone()
    src[n // 2:] = src[n // 2].item()                              # one page read by many pairs
    pools = [torch.randn(n_pages, 16, 4 if n_pages > 10000 else 200, generator=g, device="cuda"),
             torch.randint(0, 255, (n_pages, 16), generator=g, device="cuda", dtype=torch.uint8)]
    want = [p.clone() for p in pools]
    for p in want:
        p[dst.long()] = p[src.long()]
    L.lsa_pages_copy(pools, src, dst)
    assert L.lsa_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(pools, want))


@pytest.mark.parametrize("extra", [0, 1100])
def test_copy_refuses_pairs_that_depend_on_order(extra):
    """`extra` further pairs, all fine: beyond 1024 the list is checked by a kernel of its own."""
    pool = torch.arange((20 + 2 * extra) * 16, device="cuda", dtype=torch.float32).reshape(-1, 16)
    want = pool.clone()
    want[9] = want[1]
    want[20 + extra:] = want[20:20 + extra].clone()
    #        fine, out of range, the same dst twice, dst read by another, onto itself
    src, dst = [1, 20, 2, 3, 4, 5, 6, 7], [9, 3, -1, 10, 10, 6, 11, 7]
    want[11] = want[6]
    src[1] = 20 + 2 * extra
    src, dst = src + list(range(20, 20 + extra)), dst + list(range(20 + extra, 20 + 2 * extra))
    L.lsa_pages_copy([pool], ints(src), ints(dst))
    with pytest.raises(L.LsaError, match="refused"):
        L.lsa_device_status()
    # 5 -> 6 is refused (6 is read); 6 -> 11 runs
    assert torch.equal(pool, want)


@pytest.mark.parametrize("n_pages,live", [(1, 0.0), (1, 1.0), (31, 0.5), (32, 0.3), (1024, 0.0), (1024, 1.0), (70001, 0.4), (1 << 19, 0.6)])
def test_compact(n_pages, live):
    g = torch.Generator(device="cuda").manual_seed(n_pages)
    ref = (torch.rand(n_pages, generator=g, device="cuda") < live).int() * 3
    pages = torch.nonzero(ref).flatten().int()
    n = pages.numel()
    table = torch.full((2, n // 2 + 2), -1, dtype=torch.int32, device="cuda")
    pages = pages[torch.randperm(n, generator=g, device="cuda")]
    table[0, :n // 2], table[1, :n - n // 2] = pages[:n // 2], pages[n // 2:]
    pool = torch.arange(n_pages, device="cuda", dtype=torch.float32)[:, None].repeat(1, 8)
    i = torch.arange(n_pages, device="cuda")
    a, b = torch.nonzero((ref > 0) & (i >= n)).flatten(), torch.nonzero((ref == 0) & (i < n)).flatten()
    to, want_pool, want_ref = i.clone(), pool.clone(), ref.clone()
    to[a], want_pool[b], want_ref[b] = b, pool[a], ref[a]
    want_ref[a] = 0
    want_table = torch.where(table >= 0, to[table.clamp_min(0).long()].int(), table)
    t0, r0 = table.clone(), ref.clone()
    t, r, k = L.lsa_pages_compact(table, ref, [pool], table_out=torch.empty_like(table), ref_out=torch.empty_like(ref))
    assert L.lsa_device_status() == 0
    assert k.tolist() == [n] and torch.equal(t, want_table) and torch.equal(r, want_ref) and torch.equal(pool, want_pool)
    assert torch.equal(table, t0) and torch.equal(ref, r0)


def test_compact_unmaps_entries_of_free_pages():
    """Stale entries on both sides of n_live: left alone they would name pages of other sequences afterwards."""
    ref = torch.zeros(100, dtype=torch.int32, device="cuda")
    ref[[0, 2, 40, 70, 99]] = 1                             # five live pages: holes at 1, 3 and 4
    pool = torch.arange(100, device="cuda", dtype=torch.float32)[:, None].repeat(1, 8)
    table = ints([[0, 40, 99], [2, 70, -1], [1, 4, 69]])    # the last row's pages are all free
    t, r, n = L.lsa_pages_compact(table, ref, [pool])
    with pytest.raises(L.LsaError, match="out of range"):
        L.lsa_device_status()
    assert n.tolist() == [5] and t.tolist() == [[0, 1, 4], [2, 3, -1], [-1, -1, -1]]
    assert r.tolist() == [1] * 5 + [0] * 95 and pool[:5, 0].tolist() == [0, 40, 2, 70, 99]


def test_wide_pages_past_32_bits():
    """A page of several pieces, and pools whose last pages lie past 4 GB."""
    pool = torch.zeros(70, 64 << 20, dtype=torch.uint8, device="cuda")
    pool[69] = torch.arange(64 << 20, device="cuda", dtype=torch.int32).to(torch.uint8)
    L.lsa_pages_copy([pool], ints([69]), ints([67]))
    assert L.lsa_device_status() == 0
    assert torch.equal(pool[67], pool[69]) and not pool[66].any() and not pool[68].any()


def test_captured_step():
    """Free, fork and reserve in one graph, replayed on new lengths."""
    m = Model(4, 6, 24, 16)
    d = Device(m, 2)
    par, kids, lens = ints([0, 0]), ints([2, 3]), ints([50, 18, 0, 0])
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    m.reserve([50, 18, 0, 0])
    L.lsa_pages_reserve(d.table, d.ref, lens, 16)
    m.len = [50, 18, 0, 0]
    d.len.copy_(ints(m.len))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.lsa_pages_free(d.table, d.ref, d.len, kids)
        L.lsa_pages_fork(d.table, d.ref, d.len, 16, par, kids, d.pools, workspace=ws)
        L.lsa_pages_reserve(d.table, d.ref, lens, 16)
    for n in (50, 70, 33):
        grow = [n, 18, n + 20, n + 1]
        lens.copy_(ints(grow))
        m.free([2, 3])
        assert m.fork([0, 0], [2, 3])
        assert m.reserve(grow)
        g.replay()
        assert L.lsa_device_status() == 0
        d.check()
