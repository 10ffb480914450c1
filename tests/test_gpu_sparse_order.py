"""Sparse latent attention with the streaming-prefix promise, right behind calls that write or read its data.

Its prefix splits need no index row and may start before the selection in front of them has ended; behind any other
call they have to wait. Every sequence of calls is compared with itself, the device waited for after each call."""
import threading

import pytest
import torch

from kv_indexing_b200 import lsa as L
from tests.paged_ref import ints

pytestmark = pytest.mark.gpu

B, T, HQ, LMAX, K, SINK, WINDOW, P = 4, 8, 128, 4096, 1024, 64, 512, 64
BUDGET = (K, SINK, WINDOW)
SCALE = 576 ** -0.5


class Step:
    """A chunk of T queries over B sequences: a dense latent cache whose rows are pages 0, 1, 2, ... of a pool too."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

        self.kv = normal(B, LMAX, 576)
        self.pool = self.kv.view(B * LMAX // P, P, 576)
        self.table = torch.arange(B * LMAX // P, device="cuda", dtype=torch.int32).view(B, LMAX // P)
        self.seq_len = ints([LMAX - 100 * b for b in range(B)])
        self.q, self.rows = normal(B, T, HQ, 576), normal(B, T, 576)
        self.iq, self.ik = normal(B, T, 64, 128), normal(B, LMAX, 128)
        self.iw = torch.randn(B, T, 64, generator=g, device="cuda")
        self.plan = L.lsa_rope_plan(64, 10000.0)
        self.idx = L.lsa_index_flat(self.iq, self.iw, self.ik, self.seq_len, BUDGET)
        torch.cuda.synchronize()

    def sparse(self, **kw):
        return L.lsa_sparse_attn(self.q, self.idx, self.seq_len, SCALE, kv=self.kv, d_v=512, stream_budget=BUDGET, **kw)[0]


def rope(s):
    L.lsa_rope(s.q, s.plan, s.seq_len, offset=512, out=s.q)


def append(s):
    L.lsa_pages_append(s.rows, s.table, s.seq_len, s.pool, plan=s.plan, offset=512)


def paged(s):
    return L.lsa_paged_attn(s.q, s.table, s.seq_len, SCALE, kv=s.pool)[0]


def copy(s):
    first = torch.arange(8, device="cuda", dtype=torch.int32)
    L.lsa_pages_copy([s.pool], first + 32, first)            # the sink's pages of sequence 0 among them


def free(s):
    L.lsa_pages_free(s.table, torch.ones(B * LMAX // P, dtype=torch.int32, device="cuda"), s.seq_len, ints([1]))


def index(s):
    s.idx = L.lsa_index_flat(s.iq, s.iw, s.ik, s.seq_len, BUDGET)
    return s.idx


def sparse(s):
    return s.sparse()


@pytest.mark.parametrize("before", [rope, append, paged, copy, free, index, sparse])
def test_behind(before):
    """Outputs and workspaces from the allocator, which hands out again what the call before has just released."""
    for seed in range(6):
        got, want = Step(seed), Step(seed)
        a = [before(got), got.sparse(), before(got), got.sparse()]
        torch.cuda.synchronize()
        b = []
        for f in (before, Step.sparse) * 2:
            b.append(f(want))
            torch.cuda.synchronize()
        for x, y in zip(a, b):
            assert x is None and y is None or torch.equal(x, y)
        assert torch.equal(got.q, want.q) and torch.equal(got.kv, want.kv)
    assert L.lsa_device_status() == 0


def test_behind_in_a_graph():
    got, want = Step(9), Step(9)
    st = torch.cuda.Stream()
    got.sparse()
    outs = torch.empty(2, B, T, HQ, 512, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        rope(got)
        got.sparse(out=outs[0])
        index(got)
        append(got)
        got.sparse(out=outs[1])
    for _ in range(4):
        g.replay()
        torch.cuda.synchronize()
        ref = []
        for f in (rope, Step.sparse, index, append, Step.sparse):
            ref.append(f(want))
            torch.cuda.synchronize()
        assert torch.equal(outs[0], ref[1]) and torch.equal(outs[1], ref[4])
    assert L.lsa_device_status() == 0


def test_two_threads_on_one_stream():
    """One thread selects, the other rotates q and attends to it: neither knows what the other launches in between."""
    got, want, other = Step(1), Step(1), Step(2)
    rows = []
    for _ in range(40):
        rope(want)
        rows.append(want.sparse())
        torch.cuda.synchronize()
    st, outs = torch.cuda.Stream(), []

    def select():
        with torch.cuda.stream(st):
            for _ in range(120):
                index(other)

    def attend():
        with torch.cuda.stream(st):
            for _ in range(40):
                rope(got)
                outs.append(got.sparse())

    threads = [threading.Thread(target=f) for f in (select, attend)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(outs) == 40 and all(torch.equal(a, b) for a, b in zip(outs, rows))
    assert L.lsa_device_status() == 0


def test_behind_a_fork_that_writes_the_lengths():
    """4000 branches of one parent; the last four are the sequences of the attention, and only the fork gives them the
    length that their index rows belong to."""
    S, n = 4100, 4000
    for seed in range(4):
        s = Step(seed)
        s.seq_len.fill_(LMAX)
        s.idx = L.lsa_index_flat(s.iq, s.iw, s.ik, s.seq_len, BUDGET)
        want = s.sparse()
        table = torch.full((S, LMAX // P), -1, dtype=torch.int32, device="cuda")
        table[0] = s.table[0]
        ref = torch.zeros(B * LMAX // P, dtype=torch.int32, device="cuda")
        ref[:LMAX // P] = 1
        lens = torch.zeros(S, dtype=torch.int32, device="cuda")
        lens[0] = LMAX
        lens[-B:] = 1000
        parent, child = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(S - n, S, device="cuda", dtype=torch.int32)
        s.seq_len = lens[-B:]
        torch.cuda.synchronize()
        L.lsa_pages_fork(table, ref, lens, P, parent, child, [s.pool])
        got = s.sparse()
        assert torch.equal(got, want) and (lens[-n:] == LMAX).all()
    assert L.lsa_device_status() == 0
