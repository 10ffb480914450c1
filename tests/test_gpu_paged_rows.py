"""Rotary positions and appending rows to pages on the GPU, against 64-bit forms."""
import itertools

import pytest
import torch

from kv_indexing_b200 import lsa as L
from tests.paged_ref import BF16, E4M3, FP32, Cache, ints, plan_numbers, rotate

pytestmark = pytest.mark.gpu

# fp32 steps of a rotated column: sine, cosine (2 each with the amplitude), two products, one sum,
# against m (|x0| + |x1|)
TURN = 8 * FP32


def positions(seq_len, q_len, T):
    n = seq_len if q_len is None else q_len
    return [[s - (T if q_len is None else m) + t if t < (T if q_len is None else m) else -1 for t in range(T)]
            for s, m in zip(seq_len, n)]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot,offset", [(64, 64, 0), (128, 32, 96), (576, 64, 512), (33, 10, 3), (100, 100, 0), (8, 2, 1)])
def test_rope(inter, dtype, d, rot, offset):
    g = torch.Generator(device="cuda").manual_seed(d + rot)
    B, T, H = 3, 5, 7
    x = torch.randn(B, T, H, d, generator=g, device="cuda").to(dtype)
    sl, ql = [5, 131072, 2], [5, 3, 5]                     # the last sequence has padding in front
    plan = L.lsa_rope_plan(rot, 10000.0, interleaved=inter)
    pos = torch.tensor(positions(sl, ql, T), device="cuda")
    want, mag = rotate(x, pos[..., None].clamp_min(0), plan_numbers(rot, 10000.0), offset, inter)
    out = torch.full_like(x, 7.0)
    L.lsa_rope(x, plan, ints(sl), q_len=ints(ql), offset=offset, out=out)
    live = pos >= 0
    half = BF16 if dtype == torch.bfloat16 else FP32
    tol = 1.01 * (half * want.abs() + TURN * mag) + 1e-38
    assert ((out.double() - want).abs() <= tol)[live].all()
    assert (out[~live] == 7.0).all()
    keep = torch.ones(d, dtype=torch.bool)
    keep[offset:offset + rot] = False
    assert torch.equal(out[live][..., keep], x[live][..., keep])     # columns outside are copied bit by bit
    mine = x.clone()
    got = L.lsa_rope(mine, plan, ints(sl), q_len=ints(ql), offset=offset, out=mine)
    assert got is mine and torch.equal(mine[live], out[live]) and torch.equal(mine[~live], x[~live])


@pytest.mark.parametrize("scaling,factor,orig,amp", [("none", 1.0, 0, 0.0), ("linear", 8.0, 0, 0.0), ("yarn", 32.0, 4096, 0.0),
                                                     ("yarn", 0.5, 2048, 0.0), ("yarn", 4.0, 8192, 1.0)])
def test_rope_scaling_at_far_positions(scaling, factor, orig, amp):
    plan = L.lsa_rope_plan(64, 10000.0, interleaved=True, scaling=scaling, factor=factor, orig_len=orig, amplitude=amp)
    f, m = plan_numbers(64, 10000.0, scaling, factor, orig, amplitude=amp)
    assert max(abs(plan.freq[i] / f[i] - 1) for i in range(32)) < 1e-14 and abs(plan.amplitude - m) < 1e-15
    x = torch.randn(4, 1, 2, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    sl = [1, 4097, 1 << 20, (1 << 30) - 1]
    want, mag = rotate(x, ints(sl)[:, None, None] - 1, (f, m), 0, True)
    out = L.lsa_rope(x, plan, ints(sl))
    assert ((out.double() - want).abs() <= FP32 * want.abs() + TURN * mag).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,H", [(1, 1, 1), (1, 1, 128), (8, 1, 128), (1, 2047, 3), (5, 33, 16), (2, 3, 5000)])
def test_rope_shapes_and_strides(dtype, B, T, H):
    d, rot = 64, 32
    g = torch.Generator(device="cuda").manual_seed(B * T + H)
    wide = torch.randn(T, B, H + 1, 3 * d, generator=g, device="cuda").to(dtype)
    x = wide.permute(1, 0, 2, 3)[:, :, 1:, d:2 * d]        # transposed, cut out of wider rows
    store = torch.zeros(B, T, H, 2 * d, device="cuda", dtype=dtype)
    plan = L.lsa_rope_plan(rot, 500000.0)
    sl = [T + 1000 * b for b in range(B)]
    want, mag = rotate(x, torch.tensor(positions(sl, None, T), device="cuda")[..., None], plan_numbers(rot, 500000.0), 16,
                       False)
    out = L.lsa_rope(x, plan, ints(sl), offset=16, out=store[..., d:])
    half = BF16 if dtype == torch.bfloat16 else FP32
    assert ((out.double() - want).abs() <= 1.01 * (half * want.abs() + TURN * mag)).all()
    assert (store[..., :d] == 0).all()


def test_rope_shared_head_is_broadcast():
    """One rotary head read by every query head: a stride of 0 on the input side."""
    x = torch.randn(2, 3, 1, 64, device="cuda").to(torch.bfloat16)
    plan = L.lsa_rope_plan(64, 10000.0)
    one = L.lsa_rope(x, plan, ints([9, 70]))
    assert torch.equal(L.lsa_rope(x.expand(2, 3, 6, 64), plan, ints([9, 70])), one.expand(2, 3, 6, 64))
    with pytest.raises(L.LsaError):
        L.lsa_rope(x.expand(2, 3, 6, 64), plan, ints([9, 70]), out=torch.empty_like(x).expand(2, 3, 6, 64))


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient(inter):
    """The inverse call is the transposed map: against the formula's gradient and against differences."""
    B, T, H, d, rot = 2, 3, 4, 48, 32
    plan = L.lsa_rope_plan(rot, 100.0, interleaved=inter, scaling="yarn", factor=4.0, orig_len=64)
    num = plan_numbers(rot, 100.0, "yarn", 4.0, 64)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, gy = (torch.randn(B, T, H, d, generator=g, device="cuda") for _ in range(2))
    sl = ints([3, 500])
    pos = torch.tensor(positions([3, 500], None, T), device="cuda")[..., None]
    gx = L.lsa_rope(gy, plan, sl, offset=8, inverse=True)
    leaf = x.double().requires_grad_()
    f, m = num
    cols = [(8 + 2 * i, 8 + 2 * i + 1) if inter else (8 + i, 8 + i + rot // 2) for i in range(rot // 2)]
    loss = (leaf * gy.double())[..., [c for c in range(d) if c not in sum(cols, ())]].sum()
    for (a, b), w in zip(cols, f):
        c, s = m * torch.cos(pos.double() * w), m * torch.sin(pos.double() * w)
        loss = loss + ((leaf[..., a] * c - leaf[..., b] * s) * gy[..., a].double() +
                       (leaf[..., b] * c + leaf[..., a] * s) * gy[..., b].double()).sum()
    loss.backward()
    mag = rotate(gy, pos, num, 8, inter, -1.0)[1]
    assert ((gx.double() - leaf.grad).abs() <= FP32 * leaf.grad.abs() + TURN * mag).all()
    # the map is linear: a step along v changes the output by the map of v, and <R v, gy> = <v, R^T gy>
    v = torch.randn(B, T, H, d, generator=g, device="cuda")
    step = (L.lsa_rope(x + v, plan, sl, offset=8).double() - L.lsa_rope(x - v, plan, sl, offset=8).double()) / 2
    a, b = (step * gy.double()).sum(), (v.double() * gx.double()).sum()
    terms = (step.abs() * gy.double().abs()).sum() + (x.double().abs() * gy.double().abs()).sum() * 2 * m
    assert abs(a - b) <= 2 * (TURN + 2 * FP32) * m * terms


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("H,d,rot,offset,inter,wide", [(1, 576, 64, 512, True, 0), (8, 128, 128, 0, False, 0), (2, 64, 0, 0, False, 1),
                                                       (3, 72, 16, 8, True, 1), (1, 8, 0, 0, False, 0)])
def test_append(P, H, d, rot, offset, inter, wide):
    sl, ql = [2 * P + 1, 40, P, 3, 0], [P + 3, 1, 0, 5, 2]        # the 4th has padding in front, the 5th nothing at all
    T = max(ql)
    c = Cache(sl, P, (H, d), wide=wide, seed=P)
    pool = c.pool()[0]
    before = pool.clone()
    x = torch.randn(len(sl), T, H, d, generator=c.gen, device="cuda").to(torch.bfloat16)
    plan = L.lsa_rope_plan(rot, 10000.0, interleaved=inter) if rot else None
    L.lsa_pages_append(x, c.table, c.seq_len, pool, q_len=ints(ql), plan=plan, offset=offset)
    assert L.lsa_device_status() == 0
    want, tol, new = before.double(), torch.zeros_like(before.double()), torch.zeros(pool.shape[:2], dtype=torch.bool, device="cuda")
    for b, t in itertools.product(range(len(sl)), range(T)):
        pos = sl[b] - ql[b] + t
        if t >= ql[b] or pos < 0:
            continue
        at = (int(c.table[b, pos // P]), pos % P)
        y, mag = rotate(x[b, t], torch.tensor(float(pos), device="cuda"), plan_numbers(rot, 10000.0) if rot else ([], 1.0),
                        offset, inter)
        want[at], tol[at], new[at] = y, 1.01 * (BF16 * y.abs() + TURN * mag) if rot else 0.0, True
    assert torch.equal(pool[~new].view(torch.int16), before[~new].view(torch.int16))    # nothing else is touched
    assert ((pool.double() - want).abs() <= tol)[new].all()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("H,d,rot,offset", [(1, 576, 64, 512), (1, 576, 0, 0), (4, 256, 32, 224), (2, 8, 0, 0), (1, 1024, 128, 0)])
def test_append_e4m3(inter, H, d, rot, offset):
    P, sl, ql = 32, [70, 33, 5], [40, 2, 5]
    T = max(ql)
    c = Cache(sl, P, (H, d), dtype=torch.bfloat16, scales=True)
    pool = torch.full((c.n_pages, P, H, d), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    x = torch.randn(3, T, H, d, generator=c.gen, device="cuda") * torch.logspace(-3, 3, T, device="cuda")[:, None, None]
    x = x.to(torch.bfloat16)
    x[1, 0] = 0.0                                           # a row of zeros: scale 1
    plan = L.lsa_rope_plan(rot, 10000.0, interleaved=inter) if rot else None
    L.lsa_pages_append(x, c.table, c.seq_len, pool, q_len=ints(ql), scale_pool=c.k_scale, plan=plan, offset=offset)
    assert L.lsa_device_status() == 0
    touched = 0
    for b in range(3):
        for t in range(ql[b]):
            pos = sl[b] - ql[b] + t
            page, slot = int(c.table[b, pos // P]), pos % P
            y, mag = rotate(x[b, t], torch.tensor(float(pos), device="cuda"), plan_numbers(rot, 10000.0) if rot else ([], 1.0),
                            offset, inter)
            s, off = float(c.k_scale[page, slot]), (TURN * mag if rot else torch.zeros_like(y))
            amax = float(y.abs().max())
            assert abs(s - (amax / 448 if amax else 1.0)) <= 2 * FP32 * s + float(off.max()) / 448
            got = pool[page, slot].double() * s
            # half a step of the code (or of the subnormals' 2^-9), on a quotient that carries the rotation's error
            tol = 1.01 * (E4M3 * y.abs() + 2.0 ** -10 * s + 2 * off + 4 * FP32 * y.abs())
            assert ((got - y).abs() <= tol).all()
            touched += 1
    assert int(torch.isfinite(c.k_scale).sum()) == touched
    live = torch.isfinite(c.k_scale)
    assert (pool.view(torch.uint8)[~live] == 0x7F).all()


def test_append_reports_unmapped_pages():
    c = Cache([40, 20], 16, (64,))
    pool = c.pool()[0]
    before = pool.clone()
    x = torch.ones(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    c.table[0, 2] = -1
    c.table[1, 1] = c.n_pages                               # past the pool
    L.lsa_pages_append(x, c.table, c.seq_len, pool)
    with pytest.raises(L.LsaError, match="out of range"):
        L.lsa_device_status()
    assert torch.equal(pool.view(torch.int16), before.view(torch.int16))
    assert L.lsa_device_status() == 0


def test_append_past_32_bit_offsets():
    """A pool of 2^31 elements and more: the slots of its last pages."""
    P, n_pages = 64, 58400
    pool = torch.zeros(n_pages, P, 576, dtype=torch.bfloat16, device="cuda")
    assert pool.numel() > 1 << 31
    table = ints([[n_pages - 1, 3], [n_pages - 2, n_pages - 3]])
    x = torch.randn(2, 2, 576, device="cuda").to(torch.bfloat16)
    L.lsa_pages_append(x, table, ints([2, 66]), pool)
    assert torch.equal(pool[n_pages - 1, :2], x[0]) and torch.equal(pool[n_pages - 3, :2], x[1])
    assert int((pool[:n_pages - 3] != 0).sum()) == 0


def test_rope_and_append_on_another_stream_and_captured():
    st = torch.cuda.Stream()
    plan = L.lsa_rope_plan(64, 10000.0, interleaved=True)
    x = torch.randn(2, 1, 4, 64, device="cuda").to(torch.bfloat16)
    want = L.lsa_rope(x, plan, ints([100, 7]))
    sl = ints([100, 7])
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = L.lsa_rope(x, plan, sl)
    st.synchronize()
    assert torch.equal(got, want)
    got.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.lsa_rope(x, plan, sl, out=got)
    for n in (3, 4000):
        sl.fill_(n)
        g.replay()
        assert torch.equal(got, L.lsa_rope(x, plan, ints([n, n])))
