"""Plain 64-bit forms of the paged-cache operators, and the caches the tests run them on."""
import math

import torch

BF16 = torch.finfo(torch.bfloat16).eps / 2      # half a step, relative
FP32 = torch.finfo(torch.float32).eps / 2
E4M3 = torch.finfo(torch.float8_e4m3fn).eps / 2


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def plan_numbers(rot, theta, scaling="none", factor=1.0, orig=0, fast=32.0, slow=1.0, amplitude=0.0):
    """(frequencies, amplitude) of a plan, pair by pair."""
    f = []
    for i in range(rot // 2):
        w = theta ** (-2.0 * i / rot)
        if scaling == "linear":
            w /= factor
        if scaling == "yarn":
            lo, hi = (rot * math.log(orig / (t * 2 * math.pi)) / (2 * math.log(theta)) for t in (fast, slow))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
            r = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            w = w * (1 - r) + w / factor * r
        f.append(w)
    m = amplitude or (0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1 else 1.0)
    return f, m


def rotate(x, pos, numbers, offset, inter, sign=1.0):
    """x [..., d] rotated by pos [...] (without the last dimension); also sum |x0| + |x1| of each pair, times m."""
    f, m = numbers
    rot = 2 * len(f)
    y, mag = x.double().clone(), x.double().abs()
    for i, w in enumerate(f):
        a, b = (offset + 2 * i, offset + 2 * i + 1) if inter else (offset + i, offset + i + rot // 2)
        c, s = m * torch.cos(pos.double() * w), m * sign * torch.sin(pos.double() * w)
        x0, x1 = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = x0 * c - x1 * s, x1 * c + x0 * s
        mag[..., a] = mag[..., b] = m * (x0.abs() + x1.abs())
    return y, mag


class Cache:
    """Sequences of the given lengths in shuffled pages; every slot of no token holds NaN."""

    def __init__(self, lens, P, shape, *, dtype=torch.bfloat16, seed=0, spare=3, wide=0, max_pages=None, scales=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.P = lens, P
        need = [(n + P - 1) // P for n in lens]
        self.n_pages = max(1, sum(need) + spare)
        width = max(1, max(need)) + 1 if max_pages is None else max_pages
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
        perm = torch.randperm(self.n_pages, generator=g, device="cuda").to(torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.seq_len = ints(lens)
        self.gen = g
        self.shape, self.dtype, self.wide = shape, dtype, wide
        self.k_scale = None
        self.floor = None                                   # e4m3: see weight_floor
        if scales:
            self.floor = []
            self.k_scale = torch.full((self.n_pages, P), float("nan"), device="cuda")

    def pool(self, spread=1.0):
        """A pool [n_pages, P, *shape] (a part of wider rows where `wide`), its rows 64-bit values by sequence."""
        shape = (self.n_pages, self.P) + self.shape
        full = torch.full((self.n_pages, self.P + (2 if self.wide else 0)) + self.shape[:-1] +
                          (self.shape[-1] * (2 if self.wide and len(self.shape) == 1 else 1),), float("nan"), device="cuda")
        store = full.to(self.dtype)
        view = store[:, :self.P, ..., :self.shape[-1]]
        assert view.shape == shape
        rows = []
        for b, n in enumerate(self.lens):
            x = torch.randn((n,) + self.shape, generator=self.gen, device="cuda") * spread
            s = torch.arange(n, device="cuda")
            page, slot = self.table[b].long()[s // self.P], s % self.P
            if self.dtype == torch.float8_e4m3fn:
                sc = torch.rand(n, generator=self.gen, device="cuda") * 0.02 + 0.001
                codes = (x / sc[:, None]).clamp(-448, 448).to(self.dtype)
                view.view(torch.uint8)[page, slot] = codes.view(torch.uint8)
                self.k_scale[page, slot] = sc
                rows.append(codes.double() * sc.double()[:, None])
                self.floor.append(weight_floor(codes, sc))
            else:
                view[page, slot] = x.to(self.dtype)
                rows.append(x.to(self.dtype).double())
        return view, rows


def weight_floor(codes, scale):
    """How far the smallest weights of an e4m3 cache move an output, by column: codes [n, d], scales [n].
    A weight w = p s of a key with scale s (p <= 2^8, and p >= 1 for the largest, so the sum l is at least 1) is held
    in fp16 as w 2^(6 - E), with 2^E <= max s: its values below 2^-14 are multiples of 2^-24, so it is off by at most
    2^-25, that is w by 2^-25 2^(E - 6) <= 2^-31 max s. Each of the n keys adds that times its code, over l >= 1."""
    if codes.shape[0] == 0:
        return torch.zeros(codes.shape[1], dtype=torch.float64, device="cuda")
    return 2.0 ** -31 * scale.double().max() * codes.double().abs().sum(0)


def attend(q, lens, qlens, scale, k_rows, v_rows, dropped=()):
    """o, lse, sum p|v| / l and the largest sum |q k| scale, from rows of K [n, Hkv, d] and V [n, Hkv, dv]
    in 64 bits; `dropped`: (sequence, token) that no query sees. Rows past a chunk are NaN."""
    B, T, Hq, _ = q.shape
    dv = v_rows[0].shape[-1]
    o = torch.full((B, T, Hq, dv), float("nan"), dtype=torch.float64, device="cuda")
    lse, mag = torch.full((B, T, Hq), float("nan"), dtype=torch.float64, device="cuda"), torch.zeros_like(o)
    big = 0.0
    for b in range(B):
        n, nq = lens[b], qlens[b]
        k, v = k_rows[b], v_rows[b]
        G = Hq // k.shape[1]
        k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
        for t in range(nq):
            pos = n - nq + t
            keep = torch.arange(n, device="cuda") <= pos
            for bb, s in dropped:
                if bb == b and s < n:
                    keep[s] = False
            sel = torch.nonzero(keep).flatten()
            if not sel.numel():
                o[b, t], lse[b, t] = 0.0, -math.inf
                continue
            x = q[b, t].double()
            sc = torch.einsum("hd,nhd->hn", x, k[sel]) * scale
            big = max(big, float(torch.einsum("hd,nhd->hn", x.abs(), k[sel].abs()).max()) * scale)
            lse[b, t] = torch.logsumexp(sc, -1)
            p = torch.softmax(sc, -1)
            o[b, t] = torch.einsum("hn,nhd->hd", p, v[sel])
            mag[b, t] = torch.einsum("hn,nhd->hd", p, v[sel].abs())
    return o, lse, mag, big


def check_attention(out, lse, want, d, n, floor=None):
    """The bound: P and the output are rounded to bf16 (half a step each; P of an e4m3 cache to fp16, a finer one, with
    an absolute error by column and sequence: floor); a score carries d fp32 roundings of its sum |q k|, which moves
    numerator and denominator; sums over n keys are fp32."""
    o, l, mag, big = want
    delta = d * FP32 * big + 64 * FP32
    tol = BF16 * mag + BF16 * o.abs() + (2 * delta + (n + 16) * FP32) * mag
    if floor:
        tol = tol + torch.stack([f[:o.shape[-1]] for f in floor])[:, None, None]
    seen = ~torch.isnan(o)
    err = (out.double() - o).abs()
    worst = ((err - 1.01 * tol)[seen]).max().item() if seen.any() else 0.0
    assert worst <= 1e-30, f"output off by {err[seen].max().item():.3g}, {worst:.3g} more than its bound"
    if lse is not None:
        fin = torch.isfinite(l)
        assert torch.equal(torch.isneginf(l), torch.isneginf(lse.double()) & ~torch.isnan(l))
        if fin.any():
            off = ((lse.double() - l).abs() - delta - (n + 16) * FP32 - 4 * FP32 * l.abs())[fin].max().item()
            assert off <= 0, f"lse off by {off:.3g} more than its bound"
