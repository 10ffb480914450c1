"""Attention over an e4m3 latent cache whose token scales lie far apart, on the GPU.

The bound is check_attention's without a floor: weights and output each rounded to bf16 (half a step), whatever the
scales of other tokens are. It holds for weights down to 2^-126, which none of these reach."""
import pytest
import torch

from kv_indexing_b200 import lsa as L
from tests.paged_ref import Cache, attend, check_attention, ints

pytestmark = pytest.mark.gpu


def cached(c, pool):
    """The cached rows of every sequence as 64-bit values [n, 1, 576]."""
    rows = []
    for b, n in enumerate(c.lens):
        s = torch.arange(n, device="cuda")
        page, slot = c.table[b].long()[s // c.P], s % c.P
        codes = pool.view(torch.uint8)[page, slot].view(pool.dtype).double()
        rows.append((codes * c.k_scale[page, slot].double()[:, None])[:, None])
    return rows


def check(c, pool, q, qlens, scale):
    out = torch.full(q.shape[:3] + (512,), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:3], 5.0, device="cuda")
    L.lsa_paged_attn(q, c.table, c.seq_len, scale, kv=pool, kv_scale=c.k_scale, q_len=ints(qlens), out=out, lse=lse)
    assert L.lsa_device_status() == 0
    k = cached(c, pool)
    assert all(torch.isfinite(r).all() for r in k)
    check_attention(out, lse, attend(q, c.lens, qlens, scale, k, [r[..., :512] for r in k]), 576, max(c.lens))


def draw(c, n):
    return (torch.randn(n, 576, generator=c.gen, device="cuda") * 100).clamp(-448, 448)


def put(c, pool, b, codes, scales):
    s = torch.arange(c.lens[b], device="cuda")
    page, slot = c.table[b].long()[s // c.P], s % c.P
    pool.view(torch.uint8)[page, slot] = codes.to(pool.dtype).view(torch.uint8)
    c.k_scale[page, slot] = scales


@pytest.mark.parametrize("T", [1, 70])
@pytest.mark.parametrize("amp", [1.0, 0.005, 1e-5, 1e-6, 1e-7, 1e-20])
def test_a_row_of_zeros_among_small_rows(T, amp):
    """Appending writes scale 1 for the row of zeros, 2^-9 to 2^-78 for the others."""
    lens, P = [1000, 131], 32
    c = Cache(lens, P, (576,), dtype=torch.float8_e4m3fn, scales=True, seed=T)
    pool, _ = c.pool()
    x = (torch.randn(2, 1000, 576, generator=c.gen, device="cuda") * amp).to(torch.bfloat16)
    x[0, 77] = x[1, 130] = 0.0
    L.lsa_pages_append(x, c.table, c.seq_len, pool, q_len=ints(lens), scale_pool=c.k_scale)
    assert int((c.k_scale == 1.0).sum()) == 2
    q = torch.randn(2, T, 16, 576, generator=c.gen, device="cuda").to(torch.bfloat16)
    check(c, pool, q, [T, T], 576 ** -0.5)


@pytest.mark.parametrize("octaves", [20, 60])
def test_scales_that_rise_along_a_prompt(octaves):
    """A prompt from position 0: no query may depend on the scales of the tokens behind it."""
    n = 300
    c = Cache([n], 16, (576,), dtype=torch.float8_e4m3fn, scales=True)
    pool, _ = c.pool()
    codes = draw(c, n)
    codes[:, 512:] = 0.0
    put(c, pool, 0, codes, torch.exp2(torch.linspace(-octaves, 0, n, device="cuda")))
    q = torch.zeros(1, n, 4, 576, dtype=torch.bfloat16, device="cuda")
    q[..., 512:] = 1.0                                      # columns that are 0 in every key: equal weights
    check(c, pool, q, [n], 1.0)


@pytest.mark.parametrize("octaves", [20, 30, 60])
@pytest.mark.parametrize("at", [0, 700, 1499])
def test_a_large_scale_without_weight(octaves, at):
    """One key of a scale 2^20 to 2^60 above the others', its score 24 below theirs and its first 512 columns zero."""
    n = 1500
    c = Cache([n], 64, (576,), dtype=torch.float8_e4m3fn, scales=True)
    pool, _ = c.pool()
    codes = draw(c, n)
    scales = torch.rand(n, generator=c.gen, device="cuda") * 0.005 + 0.005
    codes[:, 512:] = 0.0
    codes[at] = 0.0
    codes[at, 575] = -1.0
    scales[at] = 2.0 ** (octaves - 7)
    put(c, pool, 0, codes, scales)
    q = torch.zeros(1, 2, 16, 576, dtype=torch.bfloat16, device="cuda")
    q[..., 575] = 24.0 * 2.0 ** (7 - octaves)
    check(c, pool, q, [2], 1.0)


@pytest.mark.parametrize("first,last", [(-60, 60), (60, -60), (-100, 20), (20, -100)])
def test_scales_2_to_the_120_apart(first, last):
    """Rising and falling within a sequence, equal weights: the keys of the largest scales make the output."""
    n = 700
    c = Cache([n, n], 32, (576,), dtype=torch.float8_e4m3fn, scales=True)
    pool, _ = c.pool()
    for b in range(2):
        codes = draw(c, n)
        codes[:, 512:] = 0.0
        put(c, pool, b, codes, torch.exp2(torch.linspace(first, last, n, device="cuda")))
    q = torch.randn(2, 3, 8, 576, generator=c.gen, device="cuda").to(torch.bfloat16)
    q[..., :512] = 0.0
    check(c, pool, q, [3, 3], 1.0)


@pytest.mark.parametrize("scale", [1e-14, 1e-20, 1e-37])
def test_rows_of_zeros_under_a_small_scale(scale):
    """Equal weights: the scale times the power of two of a row of zeros (or of columns below 2^-86) stays above 0, which
    a masked key's score of -inf is multiplied by."""
    lens, qlens = [300, 40], [60, 40]
    c = Cache(lens, 32, (576,), dtype=torch.float8_e4m3fn, scales=True)
    pool, _ = c.pool()
    q = torch.zeros(2, 60, 4, 576, dtype=torch.bfloat16, device="cuda")
    q[:, :, 1] = 2.0 ** -90
    q[:, :, 2] = 1.0
    check(c, pool, q, qlens, scale)
