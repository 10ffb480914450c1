"""The paged-cache calls without a GPU: plans, workspace sizes, refusals on the host."""
import ctypes
import math

import pytest
import torch

from kv_indexing_b200 import lsa as L
from tests.test_boundary_cpu import _DeviceTensor

MB = 1 << 20
INVALID, UNSUPPORTED, WORKSPACE = L.LSA_ERR_INVALID_ARG, L.LSA_ERR_UNSUPPORTED, L.LSA_ERR_WORKSPACE


@pytest.mark.parametrize("rot,theta", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (256, 1.5)])
def test_plan_frequencies(rot, theta):
    p = L.lsa_rope_plan(rot, theta, interleaved=True)
    assert (p.rot_dim, p.interleaved, p.amplitude) == (rot, 1, 1.0)
    for i in range(128):
        want = theta ** (-2.0 * i / rot) if i < rot // 2 else 0.0
        assert abs(p.freq[i] - want) <= 1e-15 * want
    lin = L.lsa_rope_plan(rot, theta, scaling="linear", factor=4.0)
    assert all(lin.freq[i] == p.freq[i] / 4.0 for i in range(rot // 2)) and lin.interleaved == 0


def test_plan_yarn_ramp():
    """Pairs that turn often keep their frequency, slow ones are interpolated, between lies a line."""
    rot, theta, orig, factor = 64, 10000.0, 4096, 16.0
    p = L.lsa_rope_plan(rot, theta, scaling="yarn", factor=factor, orig_len=orig)
    base = L.lsa_rope_plan(rot, theta)
    low = math.floor(rot * math.log(orig / (32 * 2 * math.pi)) / (2 * math.log(theta)))
    high = math.ceil(rot * math.log(orig / (2 * math.pi)) / (2 * math.log(theta)))
    for i in range(rot // 2):
        r = min(max((i - low) / (high - low), 0.0), 1.0)
        want = base.freq[i] * (1 - r + r / factor)
        assert abs(p.freq[i] - want) <= 1e-14 * want
    assert 0 < low < high < 32 and p.freq[low] == base.freq[low] and abs(p.freq[high] * factor / base.freq[high] - 1) < 1e-14
    assert p.amplitude == 0.1 * math.log(factor) + 1.0
    assert L.lsa_rope_plan(rot, theta, scaling="yarn", factor=factor, orig_len=orig, amplitude=0.75).amplitude == 0.75


@pytest.mark.parametrize("kw,code", [
    (dict(rot_dim=0), INVALID), (dict(rot_dim=63), INVALID), (dict(rot_dim=258), UNSUPPORTED), (dict(theta=1.0), INVALID),
    (dict(theta=math.nan), INVALID), (dict(theta=math.inf), INVALID), (dict(scaling="linear", factor=0.0), INVALID),
    (dict(scaling="yarn", factor=2.0), INVALID), (dict(scaling="yarn", factor=2.0, orig_len=64, beta_fast=1.0), INVALID),
    (dict(amplitude=-1.0), INVALID), (dict(amplitude=math.nan), INVALID)])
def test_plan_refusals(kw, code):
    a = dict(rot_dim=64, theta=10000.0)
    a.update(kw)
    with pytest.raises(L.LsaError) as e:
        L.lsa_rope_plan(a.pop("rot_dim"), a.pop("theta"), **a)
    assert e.value.status == code
    with pytest.raises(ValueError, match="scaling"):
        L.lsa_rope_plan(64, 10000.0, scaling="ntk")


def _fill(cls, base, kw):
    assert set(kw) <= set(base)
    base.update(kw)
    return cls(*[base[f] for f, _ in cls._fields_])


def _rope(**kw):
    return _fill(L.RopeIn, dict(B=2, T=3, H=4, d=64, dtype=L.LSA_BF16, offset=0, inverse=0, seq_len=MB, q_len=None, x=2 * MB,
                                x_stride_b=768, x_stride_t=256, x_stride_h=64, out_stride_b=768, out_stride_t=256,
                                out_stride_h=64), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(H=-1), INVALID), (dict(d=0), INVALID), (dict(dtype=L.LSA_E4M3), INVALID),
    (dict(offset=-1), INVALID), (dict(offset=33), INVALID), (dict(d=16), INVALID), (dict(x=None), INVALID),
    (dict(seq_len=None), INVALID), (dict(x=2 * MB + 1), INVALID), (dict(d=70000), UNSUPPORTED),
    (dict(B=1 << 20, T=1 << 20), UNSUPPORTED), (dict(H=(1 << 20) + 1), UNSUPPORTED), (dict(out_stride_h=0), INVALID),
    (dict(out_stride_b=0), INVALID), (dict(out_stride_t=0), INVALID)])
def test_rope_refusals(kw, code):
    lib, plan = L.load(), L.lsa_rope_plan(32, 10000.0)
    assert lib.lsa_rope(ctypes.byref(_rope(**kw)), ctypes.byref(plan), 3 * MB, None) == code, lib.lsa_last_error()


def test_rope_refusals_of_plan_and_out():
    lib, plan = L.load(), L.lsa_rope_plan(32, 10000.0)
    assert lib.lsa_rope(ctypes.byref(_rope()), None, 3 * MB, None) == INVALID
    assert lib.lsa_rope(None, ctypes.byref(plan), 3 * MB, None) == INVALID
    assert lib.lsa_rope(ctypes.byref(_rope()), ctypes.byref(plan), None, None) == INVALID
    assert lib.lsa_rope(ctypes.byref(_rope()), ctypes.byref(L.RopePlan()), 3 * MB, None) == INVALID       # never filled
    assert lib.lsa_rope(ctypes.byref(_rope(out_stride_h=128)), ctypes.byref(plan), 2 * MB, None) == INVALID   # in place


def _append(**kw):
    return _fill(L.AppendIn, dict(B=2, T=1, H=1, d=576, n_pages=40, page_size=64, max_pages=8, dtype=L.LSA_BF16, offset=512,
                                  seq_len=MB, q_len=None, table=2 * MB, x=3 * MB, pool=4 * MB, page_stride=64 * 576,
                                  row_stride=576, scales=None), kw)


E4 = dict(dtype=L.LSA_E4M3, scales=5 * MB)


@pytest.mark.parametrize("kw,code", [
    (dict(page_size=48), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED), (dict(n_pages=0), INVALID),
    (dict(n_pages=(1 << 19) + 1), UNSUPPORTED), (dict(max_pages=0), INVALID), (dict(max_pages=1 << 24), UNSUPPORTED),
    (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(table=None), INVALID), (dict(pool=None), INVALID), (dict(x=None), INVALID),
    (dict(x=3 * MB + 8), INVALID), (dict(pool=4 * MB + 2), INVALID), (dict(d=580), UNSUPPORTED), (dict(row_stride=568), INVALID),
    (dict(row_stride=580), INVALID), (dict(page_stride=0), INVALID), (dict(page_stride=64 * 576 + 4), INVALID),
    (dict(scales=5 * MB), INVALID), (dict(dtype=L.LSA_E4M3), INVALID), (dict(dtype=L.LSA_FP32), INVALID),
    (dict(offset=520), INVALID), (dict(offset=508), UNSUPPORTED), (dict(E4, d=1032, row_stride=1040), UNSUPPORTED),
    (dict(E4, d=568), UNSUPPORTED), (dict(E4, row_stride=584), INVALID), (dict(E4, scales=5 * MB + 2), INVALID)])
def test_append_refusals(kw, code):
    lib, plan = L.load(), L.lsa_rope_plan(64, 10000.0)
    assert lib.lsa_pages_append(ctypes.byref(_append(**kw)), ctypes.byref(plan), None) == code, lib.lsa_last_error()
    assert lib.lsa_pages_append(None, ctypes.byref(plan), None) == INVALID
    odd = L.lsa_rope_plan(24, 10000.0)
    assert lib.lsa_pages_append(ctypes.byref(_append()), ctypes.byref(odd), None) == UNSUPPORTED


def _paged(**kw):
    d = kw.get("d_qk", 576)
    kw = dict(kw)
    row = d * kw.get("Hkv", 1)
    return _fill(L.PagedAttnIn, dict(B=2, T=1, Hq=16, Hkv=1, d_qk=576, d_v=512 if d == 576 else d, n_pages=40, page_size=64,
                                     max_pages=8, scale=0.1, kv_dtype=L.LSA_BF16, seq_len=MB, q_len=None, table=2 * MB, q=3 * MB,
                                     k=4 * MB, v=4 * MB if d == 576 else 6 * MB, k_page_stride=64 * row, k_row_stride=row,
                                     v_page_stride=64 * row, v_row_stride=row, k_scale=None), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(B=70000), UNSUPPORTED), (dict(Hq=0), INVALID), (dict(Hq=129), UNSUPPORTED),
    (dict(Hkv=2), UNSUPPORTED), (dict(d_qk=64, d_v=64, Hkv=3), INVALID), (dict(d_qk=96, d_v=96), UNSUPPORTED),
    (dict(d_qk=128, d_v=64), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(table=None), INVALID), (dict(seq_len=None), INVALID),
    (dict(q=3 * MB + 2), INVALID), (dict(v=6 * MB), UNSUPPORTED), (dict(v_row_stride=584), UNSUPPORTED),
    (dict(k_row_stride=580, v_row_stride=580), INVALID), (dict(k_row_stride=568, v_row_stride=568), INVALID),
    (dict(k_page_stride=0, v_page_stride=0), INVALID), (dict(scale=0.0), INVALID), (dict(scale=math.inf), INVALID),
    (dict(scale=math.nan), INVALID), (dict(kv_dtype=2), INVALID), (dict(kv_dtype=L.LSA_E4M3), INVALID),
    (dict(k_scale=5 * MB), INVALID), (dict(kv_dtype=L.LSA_E4M3, k_scale=5 * MB + 1), INVALID),
    (dict(kv_dtype=L.LSA_E4M3, k_scale=5 * MB, k_row_stride=584, v_row_stride=584), INVALID),
    (dict(d_qk=64, d_v=64, kv_dtype=L.LSA_E4M3, k_scale=5 * MB), UNSUPPORTED), (dict(T=1 << 28), UNSUPPORTED)])
def test_paged_attention_refusals(kw, code):
    lib = L.load()
    pi = _paged(**kw)
    assert lib.lsa_paged_attn(ctypes.byref(pi), 7 * MB, None, None, 0, None) == code, lib.lsa_last_error()
    with pytest.raises(L.LsaError) as e:
        L.workspace_size(L.LSA_OP_PAGED_ATTN, paged=pi)
    assert e.value.status == code


def test_paged_attention_refusals_of_out_and_workspace():
    lib = L.load()
    pi = _paged()
    n = L.workspace_size(L.LSA_OP_PAGED_ATTN, paged=pi)
    assert n > 0 and n % 256 == 0
    ok = (ctypes.byref(pi), 7 * MB, None)
    assert lib.lsa_paged_attn(ctypes.byref(pi), None, None, 256, n, None) == INVALID
    assert lib.lsa_paged_attn(ctypes.byref(pi), 7 * MB + 2, None, 256, n, None) == INVALID
    assert lib.lsa_paged_attn(ctypes.byref(pi), 7 * MB, 8 * MB + 2, 256, n, None) == INVALID
    assert lib.lsa_paged_attn(*ok, 256, n - 1, None) == WORKSPACE
    assert lib.lsa_paged_attn(*ok, None, n, None) == INVALID
    assert lib.lsa_paged_attn(*ok, 128, n, None) == INVALID
    assert lib.lsa_paged_attn(None, 7 * MB, None, None, 0, None) == INVALID
    # pieces of cut tiles: two per worker (a pair of SMs), whatever the number of rows, and a span for every tile
    big = L.workspace_size(L.LSA_OP_PAGED_ATTN, paged=_paged(B=8, T=4000, Hq=128, max_pages=4000))
    small = L.workspace_size(L.LSA_OP_PAGED_ATTN, paged=_paged(B=8, T=1, Hq=128, max_pages=4000))
    assert big - small == 8 * 4000 * 16 - 256


def test_upkeep_refusals():
    lib = L.load()
    t, r, s, x = MB, 2 * MB, 3 * MB, 4 * MB
    pools = (L.Pool * 1)(L.Pool(16 * MB, 4096, 4096))
    assert lib.lsa_pages_reserve(None, r, x, 4, 8, 40, 16, None) == INVALID
    assert lib.lsa_pages_reserve(t, r + 4, x, 4, 8, 40, 16, None) == INVALID
    assert lib.lsa_pages_reserve(t, r, None, 4, 8, 40, 16, None) == INVALID
    assert lib.lsa_pages_reserve(t, r, x, 0, 8, 40, 16, None) == INVALID
    assert lib.lsa_pages_reserve(t, r, x, 8193, 8, 40, 16, None) == UNSUPPORTED
    assert lib.lsa_pages_reserve(t, r, x, 4, 8, 40, 24, None) == UNSUPPORTED
    assert lib.lsa_pages_reserve(t, r, x, 4, 8, (1 << 19) + 1, 16, None) == UNSUPPORTED
    assert lib.lsa_pages_free(t, r, None, 4, 8, 40, x, 1, None) == INVALID
    assert lib.lsa_pages_free(t, r, s, 4, 8, 40, None, 1, None) == INVALID
    assert lib.lsa_pages_free(t, r, s, 4, 8, 40, x, -1, None) == INVALID
    assert lib.lsa_pages_free(t, r, s, 4, 8, 40, None, 0, None) == 0
    fork = lambda n, ws, nb, p=pools, np=1: lib.lsa_pages_fork(t, r, s, 4, 8, 40, 16, x, x, n, p, np, ws, nb, None)  # noqa: E731
    assert fork(2, None, 0) == WORKSPACE and fork(2, 128, 4096) == INVALID and fork(-1, 256, 4096) == INVALID
    assert fork(0, None, 0) == 0
    for bad, code in (((8, 4096, 4096), INVALID), ((16 * MB, 8, 4096), INVALID), ((16 * MB, 24, 4096), INVALID),
                      ((16 * MB, 4096, 4080), INVALID), ((None, 4096, 4096), INVALID), ((16 * MB, 65 * MB, 65 * MB), UNSUPPORTED)):
        assert fork(2, 256, 4096, (L.Pool * 1)(L.Pool(*bad))) == code, bad
    assert fork(2, 256, 4096, None) == INVALID
    assert lib.lsa_pages_copy(pools, 1, 40, x, None, 3, 256, 4096, None) == INVALID
    assert lib.lsa_pages_copy(pools, 1, 40, x, x, 1025, 256, 0, None) == WORKSPACE
    assert lib.lsa_pages_copy(pools, 1, 0, x, x, 3, 256, 4096, None) == INVALID
    n = L.workspace_size(L.LSA_OP_PAGES_COMPACT, n_pages=40)
    comp = lambda tout, rout, nb: lib.lsa_pages_compact(t, r, 4, 8, 40, pools, 1, tout, rout, None, 256, nb, None)  # noqa: E731
    assert comp(None, r, n) == INVALID and comp(t, None, n) == INVALID and comp(t, r, n - 1) == WORKSPACE
    assert comp(t, r + 8, n) == INVALID


class _Strided(_DeviceTensor):
    def __init__(self, shape, dtype, strides=None, **kw):
        super().__init__(shape, dtype, **kw)
        s, n = [], 1
        for m in reversed(shape):
            s.insert(0, n)
            n *= m
        self._strides = strides or tuple(s)
        self._contiguous = self._strides == tuple(s)

    def stride(self, i=None):
        return self._strides if i is None else self._strides[i]

    def data_ptr(self):
        return 16 * MB


def test_binding_refusals(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    bf, f32, i32, f8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn
    S = _Strided
    q, table, sl = S((2, 1, 16, 64), bf), S((2, 8), i32), S((2,), i32)
    k = S((40, 16, 4, 64), bf)
    L.paged_attn_in(q, table, sl, 0.1, k=k, v=k)           # what the cases below depart from
    for args, kw, msg in [
            ((q, S((3, 8), i32), sl, 0.1), dict(k=k, v=k), "table has shape"),
            ((q, table, S((3,), i32), 0.1), dict(k=k, v=k), "seq_len has shape"),
            ((q, table, sl, 0.1), dict(k=k, v=k, q_len=S((3,), i32)), "q_len has shape"),
            ((q, table, sl, 0.1), dict(k=k, v=S((41, 16, 4, 64), bf)), "v has shape"),
            ((q, table, sl, 0.1), dict(k=k), "v is required"),
            ((q, table, sl, 0.1), dict(), "k is required"),
            ((q, table, sl, 0.1), dict(kv=k, k=k), "not both"),
            ((q, table, sl, 0.1), dict(k=k, v=k, kv_scale=S((40, 16), f32)), "e4m3"),
            ((q, table, sl, 0.1), dict(k=S((40, 16, 4, 64), bf, strides=(8192, 512, 128, 1)), v=k), "heads of a row"),
            ((q, table, sl, 0.1), dict(k=S((40, 16, 4, 64), bf, strides=(8192, 512, 64, 2)), v=k), "dense last"),
            ((q, table, sl, 0.1), dict(k=S((40, 16, 4, 64), bf, device=1), v=k), "current device"),
            ((S((2, 1, 16, 576), bf), table, sl, 0.1), dict(kv=S((40, 16, 576), f8)), "kv_scale is required"),
            ((S((2, 1, 16, 576), bf), table, sl, 0.1), dict(kv=S((40, 16, 576), f8), kv_scale=S((40, 8), f32)), "kv_scale has shape")]:
        with pytest.raises(ValueError, match=msg):
            L.paged_attn_in(*args, **kw)
    x = S((2, 1, 1, 576), bf)
    pool = S((40, 16, 1, 576), bf)
    for args, kw, msg in [((x, table, sl, S((40, 16, 1, 64), bf)), {}, "pool has shape"),
                          ((x, table, sl, S((40, 16, 1, 576), f32)), {}, "dtype"),
                          ((x, table, sl, S((40, 16, 1, 576), f8)), {}, "scale_pool is required"),
                          ((x, table, sl, pool), dict(scale_pool=S((40, 16), f32)), "e4m3")]:
        with pytest.raises(ValueError, match=msg):
            L.lsa_pages_append(*args, **kw)
    plan = L.lsa_rope_plan(64, 10000.0)
    for args, kw, msg in [((S((2, 1, 16), bf), plan, sl), {}, "4 dims"), ((S((2, 1, 16, 64), f8), plan, sl), {}, "dtype"),
                          ((q, plan, S((3,), i32)), {}, "seq_len has shape"), ((q, plan, sl), dict(out=S((2, 1, 8, 64), bf)), "out has shape"),
                          ((S((2, 1, 16, 64), bf, strides=(2048, 2048, 128, 2)), plan, sl), dict(out=q), "dense last")]:
        with pytest.raises(ValueError, match=msg):
            L.lsa_rope(*args, **kw)
    ref, ids = S((40,), i32), S((2,), i32)
    with pytest.raises(ValueError, match="seq_len has shape"):
        L.lsa_pages_free(table, ref, S((3,), i32), ids)
    with pytest.raises(ValueError, match="lens has shape"):
        L.lsa_pages_reserve(table, ref, S((3,), i32), 16)
    with pytest.raises(ValueError, match="child has shape"):
        L.lsa_pages_fork(table, ref, sl, 16, ids, S((3,), i32), [])
    with pytest.raises(ValueError, match="at least one pool"):
        L.lsa_pages_copy([], ids, ids)
    with pytest.raises(ValueError, match="table_out has shape"):
        L.lsa_pages_compact(table, ref, [], table_out=S((2, 9), i32))
    with pytest.raises(ValueError, match="expected \\(40"):
        L.lsa_pages_fork(table, ref, sl, 16, ids, ids, [S((39, 16, 64), bf)])
