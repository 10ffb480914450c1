"""Attention over a paged cache on the GPU, against the definition in 64 bits."""
import math

import pytest
import torch

from kv_indexing_b200 import lsa as L
from tests.paged_ref import BF16, E4M3, FP32, Cache, attend, check_attention, ints, plan_numbers, rotate, weight_floor

pytestmark = pytest.mark.gpu


def call(c, q, scale, pools, ql=None, **kw):
    B, T, Hq, d = q.shape
    dv = 512 if d == 576 else d
    out = torch.full((B, T, Hq, dv), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, T, Hq), 5.0, device="cuda")
    kv = dict(kv=pools[0], kv_scale=c.k_scale) if d == 576 else dict(k=pools[0], v=pools[1])
    got = L.lsa_paged_attn(q, c.table, c.seq_len, scale, q_len=None if ql is None else ints(ql), out=out, lse=lse, **kv, **kw)
    assert got[0] is out
    return out, lse


def run(lens, qlens, Hq, Hkv, d, P, *, T=None, kind="bf16", seed=0, wide=0, scale=None, spread=1.0):
    latent = d == 576
    shape = (576,) if latent else (Hkv, d)
    c = Cache(lens, P, shape, dtype=torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16, seed=seed, wide=wide,
              scales=kind == "e4m3")
    pools, rows = zip(*[c.pool(spread) for _ in range(1 if latent else 2)])
    T = T or max(max(qlens), 1)
    q = torch.randn(len(lens), T, Hq, d, generator=c.gen, device="cuda").to(torch.bfloat16)
    for b, n in enumerate(qlens):
        q[b, n:] = float("nan")                            # behind a chunk: never used
    scale = scale or 1 / math.sqrt(d)
    out, lse = call(c, q, scale, pools, qlens)
    assert L.lsa_device_status() == 0
    k = [r[:, None] for r in rows[0]] if latent else rows[0]
    v = [r[:, None, :512] for r in rows[0]] if latent else rows[1]
    check_attention(out, lse, attend(q, lens, qlens, scale, k, v), d, max(lens), c.floor)
    for b, n in enumerate(qlens):                          # rows behind a chunk stay as they were
        assert (out[b, n:] == 5.0).all() and (lse[b, n:] == 5.0).all()
    return c, q, pools, out, lse


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700]


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("d,Hq,Hkv,kind", [(64, 4, 2, "bf16"), (128, 5, 1, "bf16"), (576, 16, 1, "bf16"), (576, 16, 1, "e4m3")])
def test_one_token(P, d, Hq, Hkv, kind):
    run(LENS, [1] * len(LENS), Hq, Hkv, d, P, kind=kind, seed=P)


@pytest.mark.parametrize("P", [16, 128])
@pytest.mark.parametrize("d,Hq,Hkv,kind", [(64, 3, 3, "bf16"), (128, 14, 2, "bf16"), (576, 7, 1, "bf16"), (576, 7, 1, "e4m3")])
def test_ragged_chunks(P, d, Hq, Hkv, kind):
    """Chunks of 0 to 70 tokens; the third and fourth bring more new tokens than the sequence has (padding in
    front), the last is empty with tokens asked for."""
    run([70, 300, 5, 33, 129, 500, 0], [70, 0, 9, 34, 1, 65, 3], Hq, Hkv, d, P, kind=kind, seed=P + d)


@pytest.mark.parametrize("d,Hq,Hkv,kind", [(64, 1, 1, "bf16"), (64, 32, 1, "bf16"), (128, 32, 4, "bf16"), (128, 130, 1, "bf16"),
                                           (576, 1, 1, "bf16"), (576, 128, 1, "bf16"), (576, 128, 1, "e4m3"), (576, 100, 1, "bf16")])
@pytest.mark.parametrize("lens,qlens", [([400], [400]), ([1000, 600], [33, 200]), ([129], [128])])
def test_chunks_of_many_rows(d, Hq, Hkv, kind, lens, qlens):
    """Several row tiles: tiles that end inside a token's heads, prompts from position 0, diagonal blocks."""
    run(lens, qlens, Hq, Hkv, d, 32, kind=kind, seed=Hq)


@pytest.mark.parametrize("d,Hq,Hkv,kind", [(64, 2, 1, "bf16"), (128, 8, 8, "bf16"), (576, 32, 1, "bf16"), (576, 32, 1, "e4m3")])
@pytest.mark.parametrize("lens", [[30001], [9000, 20, 17000, 1]])
def test_long_sequences_are_split(d, Hq, Hkv, kind, lens):
    run(lens, [1] * len(lens), Hq, Hkv, d, 64, kind=kind, seed=4)


@pytest.mark.parametrize("d,Hq,Hkv,kind,T", [(64, 24, 24, "bf16", 1), (128, 4, 2, "bf16", 2), (128, 160, 1, "bf16", 2),
                                             (576, 5, 1, "bf16", 1), (576, 5, 1, "e4m3", 2)])
def test_many_sequences(d, Hq, Hkv, kind, T):
    """More sequences than workers: a worker goes through many tiles, empty ones among them."""
    lens = [(37 * i) % 290 for i in range(350)]
    run(lens, [min(T, n) if i % 7 else 0 for i, n in enumerate(lens)], Hq, Hkv, d, 16, T=T, kind=kind, seed=9)


@pytest.mark.parametrize("d,Hq,Hkv,kind", [(64, 4, 2, "bf16"), (128, 4, 2, "bf16"), (576, 16, 1, "bf16")])
def test_rows_of_wider_pages(d, Hq, Hkv, kind):
    run([300, 77], [2, 2], Hq, Hkv, d, 16, kind=kind, wide=1)


@pytest.mark.parametrize("d,kind", [(64, "bf16"), (128, "bf16"), (576, "bf16"), (576, "e4m3")])
@pytest.mark.parametrize("T", [1, 40])
def test_large_scores(d, kind, T):
    """Scores in the hundreds: the softmax is close to one key, the running maximum moves often."""
    run([1000, 200], [T, T], 8, 1 if d == 576 else 4, d, 32, kind=kind, scale=2.0, spread=3.0)


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("down", [1e-30, 1e-6, 1.0, 1e6, 1e30])
def test_e4m3_queries_and_scales_of_any_size(T, down):
    """Rows of q from 1e-30 to 1e30 and of zeros (fp16 holds neither end: they are scaled by row), keys whose scales
    differ by 2^40, rising and falling along the sequence, and the product of the two kept moderate."""
    lens, qlens = [900, 333], [T, T]
    c = Cache(lens, 32, (576,), dtype=torch.float8_e4m3fn, scales=True, seed=T)
    pool, _ = c.pool()
    rows, c.floor = [], []
    for b, n in enumerate(lens):
        s = torch.arange(n, device="cuda")
        page, slot = c.table[b].long()[s // 32], s % 32
        sc = torch.exp2(torch.linspace(-30, 10, n, device="cuda") * (1 if b else -1) + (0 if b else -20)) * 0.01 / down
        c.k_scale[page, slot] = sc
        codes = pool.view(torch.uint8)[page, slot].view(pool.dtype)
        rows.append(codes.double() * sc.double()[:, None])
        c.floor.append(weight_floor(codes, sc))
    q = (torch.randn(2, T, 8, 576, generator=c.gen, device="cuda") * down).to(torch.bfloat16)
    q[:, :, 1] = 0.0
    q[:, :, 2, 1:] = 0.0
    out, lse = call(c, q, 0.02, [pool], qlens)
    assert L.lsa_device_status() == 0
    want = attend(q, lens, qlens, 0.02, [r[:, None] for r in rows], [r[:, None, :512] for r in rows])
    check_attention(out, lse, want, 576, 900, c.floor)


@pytest.mark.parametrize("d,kind", [(64, "bf16"), (128, "bf16"), (576, "bf16"), (576, "e4m3")])
@pytest.mark.parametrize("T,n", [(1, 5000), (1, 300), (90, 700)])
def test_rising_scores(d, kind, T, n):
    """Every key scores higher than all before it: every block rescales what is there."""
    Hq, Hkv, P = 4, 1, 16
    c = Cache([n], P, (576,) if d == 576 else (1, d), dtype=torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16,
              scales=kind == "e4m3")
    ramp = torch.linspace(1.0, 240.0, n, device="cuda")
    s = torch.arange(n, device="cuda")
    page, slot = c.table[0].long()[s // P], s % P
    pools, rows = [], []
    for i in range(1 if d == 576 else 2):
        pool, _ = c.pool()
        x = torch.randn((n,) + c.shape, generator=c.gen, device="cuda")
        if i == 0:
            x[..., 0] = ramp.view([n] + [1] * (x.dim() - 2)) if x.dim() > 2 else ramp
        x = x.to(c.dtype)
        if kind == "e4m3":
            c.k_scale[page, slot] = 1.0
            pool.view(torch.uint8)[page, slot] = x.view(torch.uint8)
        else:
            pool[page, slot] = x
        pools.append(pool)
        rows.append([x.double()])
    q = torch.zeros(1, T, Hq, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 2.0
    q[..., 1] = torch.randn(1, T, Hq, generator=c.gen, device="cuda").to(torch.bfloat16)
    out, lse = call(c, q, 1.0, pools)
    assert L.lsa_device_status() == 0
    k = [r[:, None] for r in rows[0]] if d == 576 else rows[0]
    v = [r[:, None, :512] for r in rows[0]] if d == 576 else rows[1]
    floor = [weight_floor(x, torch.ones(n, device="cuda"))] if kind == "e4m3" else None
    check_attention(out, lse, attend(q, [n], [T], 1.0, k, v), d, n, floor)


@pytest.mark.parametrize("d,kind", [(64, "bf16"), (128, "bf16"), (576, "bf16"), (576, "e4m3")])
@pytest.mark.parametrize("T", [1, 60])
def test_unmapped_pages_are_left_out_and_reported(d, kind, T):
    lens, P = [300, 64, 40], 16
    Hq, Hkv = (3, 1) if d == 576 else (4, 2)
    c = Cache(lens, P, (576,) if d == 576 else (Hkv, d), dtype=torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16,
              scales=kind == "e4m3")
    pools, rows = zip(*[c.pool() for _ in range(1 if d == 576 else 2)])
    c.table[0, 3], c.table[0, 18] = -1, c.n_pages
    c.table[1] = -7                                        # nothing of sequence 1 is there
    dropped = [(0, s) for s in list(range(48, 64)) + list(range(288, 300))] + [(1, s) for s in range(64)]
    qlens = [T, min(T, 64), min(T, 40)]
    q = torch.randn(3, T, Hq, d, generator=c.gen, device="cuda").to(torch.bfloat16)
    out, lse = call(c, q, d ** -0.5, pools, qlens)
    with pytest.raises(L.LsaError, match="out of range"):
        L.lsa_device_status()
    k = [r[:, None] for r in rows[0]] if d == 576 else rows[0]
    v = [r[:, None, :512] for r in rows[0]] if d == 576 else rows[1]
    check_attention(out, lse, attend(q, lens, qlens, d ** -0.5, k, v, dropped), d, 300, c.floor)


@pytest.mark.parametrize("d", [64, 576])
def test_a_length_past_the_table_is_reported(d):
    c = Cache([64], 32, (576,) if d == 576 else (1, d), max_pages=2)
    pools, rows = zip(*[c.pool() for _ in range(1 if d == 576 else 2)])
    q = torch.randn(1, 1, 2, d, generator=c.gen, device="cuda").to(torch.bfloat16)
    want = call(c, q, 0.1, pools)
    assert L.lsa_device_status() == 0
    c.seq_len.fill_(65)
    got = call(c, q, 0.1, pools)
    with pytest.raises(L.LsaError, match="out of range"):
        L.lsa_device_status()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("d,kind", [(128, "bf16"), (576, "bf16"), (576, "e4m3")])
def test_pools_past_32_bit_offsets(d, kind):
    """A pool of 2^31 elements and more, the sequence in its last pages; without q_len and lse."""
    P, Hkv = 64, 1 if d == 576 else 8
    width = 576 if d == 576 else Hkv * d
    n_pages = (1 << 31) // (P * width) + 40
    dt = torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(1)
    shape = (n_pages, P, 576) if d == 576 else (n_pages, P, Hkv, d)
    scales = torch.ones(n_pages, P, device="cuda") if kind == "e4m3" else None
    n = 30 * P + 5
    table = (n_pages - 1 - torch.arange(32, device="cuda", dtype=torch.int32))[None].contiguous()
    pools, rows = [], []
    for _ in range(1 if d == 576 else 2):
        pool = torch.empty(shape, dtype=dt, device="cuda")
        x = torch.randn((31 * P,) + shape[2:], generator=g, device="cuda").to(dt)
        part = pool[n_pages - 31:]
        part.view(torch.uint8)[:] = x.view((31, P) + shape[2:]).flip(0).view(torch.uint8)
        pools.append(pool)
        rows.append([x[:n].double()])
    q = torch.randn(1, 2, 8, d, generator=g, device="cuda").to(torch.bfloat16)
    kv = dict(kv=pools[0], kv_scale=scales) if d == 576 else dict(k=pools[0], v=pools[1])
    out, lse = L.lsa_paged_attn(q, table, ints([n]), d ** -0.5, **kv)
    assert L.lsa_device_status() == 0 and lse is None
    k = [r[:, None] for r in rows[0]] if d == 576 else rows[0]
    v = [r[:, None, :512] for r in rows[0]] if d == 576 else rows[1]
    floor = [weight_floor(x[:n], torch.ones(n, device="cuda"))] if kind == "e4m3" else None
    check_attention(out, None, attend(q, [n], [2], d ** -0.5, k, v), d, n, floor)


@pytest.mark.parametrize("d,kind", [(64, "bf16"), (128, "bf16"), (576, "bf16"), (576, "e4m3")])
def test_calls_repeat_bit_for_bit(d, kind):
    """On another stream, and after other calls: nothing is kept, no order of additions changes."""
    c, q, pools, out, lse = run([5000, 130], [2, 2], 8, 1, d, 32, kind=kind)
    st = torch.cuda.Stream()
    for _ in range(3):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            o2, l2 = call(c, q, 1 / math.sqrt(d), pools, [2, 2])
        st.synchronize()
        assert torch.equal(o2, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("d,kind", [(64, "bf16"), (128, "bf16"), (576, "bf16"), (576, "e4m3")])
@pytest.mark.parametrize("T", [1, 20])
def test_captured_call_follows_new_lengths(d, kind, T):
    lens = [2000, 900]
    c, q, pools, _, _ = run(lens, [T, T], 8, 1, d, 32, kind=kind)
    kv = dict(kv=pools[0], kv_scale=c.k_scale) if d == 576 else dict(k=pools[0], v=pools[1])
    ql = ints([T, T])
    pi = L.paged_attn_in(q, c.table, c.seq_len, 0.1, q_len=ql, **kv)
    ws = torch.empty(max(256, L.workspace_size(L.LSA_OP_PAGED_ATTN, paged=pi)), dtype=torch.uint8, device="cuda")
    out = torch.zeros(2, T, 8, 512 if d == 576 else d, dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.lsa_paged_attn(q, c.table, c.seq_len, 0.1, q_len=ql, out=out, workspace=ws, **kv)
    for a, b in ((2000, 900), (T, 77), (0, 555)):
        c.seq_len.copy_(ints([a, b]))
        g.replay()
        got = out.clone()
        want, _ = L.lsa_paged_attn(q, c.table, c.seq_len, 0.1, q_len=ql, **kv)
        assert torch.equal(got, want)
    assert L.lsa_device_status() == 0


@pytest.mark.parametrize("d,Hq,Hkv,kind", [(64, 8, 2, "bf16"), (128, 6, 1, "bf16"), (576, 8, 1, "bf16"), (576, 8, 1, "e4m3")])
@pytest.mark.parametrize("T", [1, 50])
def test_queries_that_are_not_numbers(d, Hq, Hkv, kind, T):
    """A NaN or an infinity in a query row makes that row NaN, in pieces that are merged too, and no other."""
    lens, qlens = [5000, 200, 0], [T, T, T]
    c, q, pools, out, lse = run(lens, qlens, Hq, Hkv, d, 32, kind=kind, seed=T)
    bad = torch.zeros(3, T, Hq, dtype=torch.bool, device="cuda")
    for i, (b, t, h, col, v) in enumerate([(0, T - 1, 1, 0, float("nan")), (0, 0, 2, d - 1, float("nan")),
                                           (1, T // 2, 0, d // 2, float("nan")), (1, 0, 3, 5, float("inf")), (2, 0, 0, 1, float("nan"))]):
        q[b, t, h, col] = v
        bad[b, t, h] = b < 2
    q[1, 0, 4] = float("nan")
    bad[1, 0, 4] = True
    o2, l2 = call(c, q, 1 / math.sqrt(d), pools, qlens)
    assert L.lsa_device_status() == 0
    assert torch.isnan(o2[bad]).all() and torch.isnan(l2[bad]).all()
    assert torch.equal(o2[~bad], out[~bad]) and torch.equal(l2[~bad], lse[~bad])


def test_stream_argument_orders_what_the_call_allocates():
    """Outputs and workspaces of a call on `stream` belong to that stream: the current one is busy for a while, and
    allocates right after the call."""
    d, st = 128, torch.cuda.Stream()
    c = Cache([5000, 130], 32, (2, d))
    pools = [c.pool()[0] for _ in range(2)]
    q = torch.randn(2, 3, 8, d, generator=c.gen, device="cuda").to(torch.bfloat16)
    ql, plan = ints([3, 2]), L.lsa_rope_plan(64, 10000.0)
    want, _ = L.lsa_paged_attn(q, c.table, c.seq_len, 0.1, k=pools[0], v=pools[1], q_len=ql)
    turned = L.lsa_rope(q, plan, c.seq_len, q_len=ql)
    torch.cuda.synchronize()
    for handle in (st, st.cuda_stream):
        torch.cuda._sleep(50_000_000)                       # a quarter of the wait limit at most, on the current stream
        got, _ = L.lsa_paged_attn(q, c.table, c.seq_len, 0.1, k=pools[0], v=pools[1], q_len=ql, stream=handle)
        rot = L.lsa_rope(q, plan, c.seq_len, q_len=ql, stream=handle)
        st.synchronize()
        assert torch.equal(got, want) and torch.equal(rot, turned)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(rot, turned)


def test_two_calls_at_once():
    """Calls on two streams, with workspaces of their own."""
    sets = []
    for seed, d, kind in ((1, 128, "bf16"), (2, 576, "bf16"), (3, 576, "e4m3")):
        c, q, pools, out, lse = run([3000, 40], [5, 5], 8, 1, d, 32, kind=kind, seed=seed)
        sets.append((c, q, pools, out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for c, q, pools, out, st in sets:
            with torch.cuda.stream(st):
                got.append((call(c, q, 1 / math.sqrt(q.shape[-1]), pools, [5, 5])[0], out))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)
    assert L.lsa_device_status() == 0


# ------------------------------------------------------------------ together
class Server:
    """A decoder layer's paged cache as a serving loop keeps it: latent rows (576 columns, the last 64 rotated)."""

    def __init__(self, S, P, e4m3, seed):
        self.S, self.P, self.n_pages = S, P, 64
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.table = torch.full((S, 12), -1, dtype=torch.int32, device="cuda")
        self.ref = torch.zeros(self.n_pages, dtype=torch.int32, device="cuda")
        self.len = torch.zeros(S, dtype=torch.int32, device="cuda")
        dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        self.kv = torch.full((self.n_pages, P, 576), 0x7F, dtype=torch.uint8, device="cuda").view(dt) if e4m3 else \
            torch.full((self.n_pages, P, 576), float("nan"), dtype=dt, device="cuda")
        self.scales = torch.full((self.n_pages, P), float("nan"), device="cuda") if e4m3 else None
        self.pools = [self.kv, self.scales] if e4m3 else [self.kv]
        self.plan = L.lsa_rope_plan(64, 10000.0, interleaved=True)
        self.rows = [torch.zeros(0, 576, dtype=torch.float64, device="cuda") for _ in range(S)]   # unrotated, in 64 bits
        self.e4m3 = e4m3

    def step(self, new):
        """new[s] tokens for each sequence: reserve, append, rotate q, attend."""
        T = max(new)
        ql = ints(new)
        x = torch.randn(self.S, T, 576, generator=self.gen, device="cuda").to(torch.bfloat16)
        q = torch.randn(self.S, T, 16, 576, generator=self.gen, device="cuda").to(torch.bfloat16)
        self.len += ql
        L.lsa_pages_reserve(self.table, self.ref, self.len, self.P)
        L.lsa_pages_append(x, self.table, self.len, self.kv, q_len=ql, scale_pool=self.scales, plan=self.plan, offset=512)
        qr = L.lsa_rope(q, self.plan, self.len, q_len=ql, offset=512, out=q.clone())
        out, _ = L.lsa_paged_attn(qr, self.table, self.len, 576 ** -0.5, kv=self.kv, kv_scale=self.scales, q_len=ql)
        assert L.lsa_device_status() == 0
        num = plan_numbers(64, 10000.0)
        for s, n in enumerate(new):
            self.rows[s] = torch.cat([self.rows[s], x[s, :n].double()])
            if not n:
                continue
            total = self.rows[s].shape[0]
            pos = torch.arange(total, device="cuda")
            # the cached rows: each within one rounding of the rotated row it was made of
            page, slot = self.table[s].long()[pos // self.P], pos % self.P
            if self.e4m3:
                sc = self.scales[page, slot].double()[:, None]
                k = self.kv.view(torch.uint8)[page, slot].view(self.kv.dtype).double() * sc
            else:
                sc, k = 0.0, self.kv[page, slot].double()
            want, m = rotate(self.rows[s], pos, num, 512, True)
            assert ((k - want).abs() <= 1.01 * ((E4M3 if self.e4m3 else BF16) * want.abs() + 2.0 ** -10 * sc + 16 * FP32 * m)).all()
            y, m = rotate(q[s, :n], pos[total - n:, None], num, 512, True)
            o, _, mag, big = attend(y[None], [total], [n], 576 ** -0.5, [k[:, None]], [k[:, None, :512]])
            # q's rotated columns are rounded to bf16, which moves a score by half a step of its sum over them
            turned = torch.einsum("hd,nd->hn", m.flatten(0, 1)[:, 512:], k[:, 512:].abs()).max().item() * 576 ** -0.5
            delta = turned * (BF16 + 8 * FP32) + 640 * FP32 * big
            tol = 1.01 * (BF16 * (mag[0] + o[0].abs()) + (math.expm1(2 * delta) + (total + 16) * FP32) * mag[0])
            assert ((out[s, :n].double() - o[0]).abs() <= tol).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("P", [16, 64])
def test_a_serving_loop(P, e4m3):
    """Prompts in chunks, decoding, branches forked from a prompt, a sequence freed, the pool compacted, decoding on."""
    sv = Server(6, P, e4m3, 3)
    sv.step([50, 3, 0, 0, 17, 0])
    sv.step([1, 40, 0, 0, 1, 0])
    kids, par = [2, 3], [0, 0]
    # the scales' pages are P fp32: a pool of their own
    L.lsa_pages_fork(sv.table, sv.ref, sv.len, P, ints(par), ints(kids), sv.pools)
    for c, p in zip(kids, par):
        sv.rows[c] = sv.rows[p].clone()
    sv.step([1, 1, 1, 1, 1, 0])                            # the branches part
    L.lsa_pages_free(sv.table, sv.ref, sv.len, ints([0, 4]))
    sv.rows[0] = sv.rows[4] = sv.rows[5]
    sv.step([0, 1, 2, 1, 0, 9])
    _, _, n_live = L.lsa_pages_compact(sv.table, sv.ref, sv.pools)
    assert int(sv.table.max()) < int(n_live) == int((sv.ref > 0).sum())
    sv.step([5, 1, 1, 1, 0, 1])
    sv.step([1, 1, 1, 1, 1, 1])
    held = torch.zeros(sv.n_pages, dtype=torch.int32, device="cuda")
    e = sv.table[sv.table >= 0].long()
    held.index_add_(0, e, torch.ones_like(e, dtype=torch.int32))
    assert torch.equal(held, sv.ref)
