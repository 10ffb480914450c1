"""Cases of the paged-cache operators: rotary positions, writing tokens into pages, attention of new
tokens over the pages, and the upkeep of the pages.

Sizes come from this repository's workloads (8 x 131072 decode over 576/512 latent rows with 128 heads,
4 x 262144, 64-wide MQA heads, pages of 16 to 128 tokens) or are generic.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the rotary part of one decode step's queries, written beside their latent part; long context, YaRN
        dict(name="rope_decode", op="rope", B=8, T=1, H=128, d=64, rot=64, offset=0, into=576, L=131072, inter=True,
             scaling="yarn", factor=32.0, orig=4096, theta=10000.0, dtype="bf16", grad=False),
        # a training step's heads, forward and gradient, 32 bits, odd length
        dict(name="rope_train", op="rope", B=2, T=2047, H=64, d=128, rot=128, offset=0, into=0, L=2047, inter=False,
             scaling="none", factor=1.0, orig=0, theta=500000.0, dtype="fp32", grad=True),
        # one new latent row for each sequence of a decode batch
        dict(name="append_decode", op="append", B=8, T=1, H=1, d=576, rot=64, offset=512, P=64, L=4096, ragged=True,
             e4m3=False, inter=True),
        # a prefill chunk quantised into an e4m3 latent cache, sequences of unequal chunks
        dict(name="append_chunk_e4m3", op="append", B=4, T=4097, H=1, d=576, rot=64, offset=512, P=64, L=8200,
             ragged=True, e4m3=True, inter=True),
        # the smallest serving call: one token, one short sequence, small pages
        dict(name="attn_one_token", op="attn", B=1, T=1, Hq=16, Hkv=2, d=64, P=16, L=1000, ragged=False, kind="bf16"),
        # grouped heads decoding a batch of ragged lengths (odd group of 5)
        dict(name="attn_decode_gqa", op="attn", B=16, T=1, Hq=40, Hkv=8, d=128, P=32, L=30011, ragged=True, kind="bf16"),
        # the headline decode shape over a paged latent cache
        dict(name="attn_decode_mla", op="attn", B=8, T=1, Hq=128, Hkv=1, d=576, P=64, L=131072, ragged=False, kind="bf16"),
        # an e4m3 latent cache, long ragged sequences
        dict(name="attn_decode_mla_e4m3", op="attn", B=4, T=2, Hq=64, Hkv=1, d=576, P=64, L=262144, ragged=True, kind="e4m3"),
        # a chunk of a long prompt in the latent form (largest work)
        dict(name="attn_chunk_mla", op="attn", B=1, T=500, Hq=128, Hkv=1, d=576, P=64, L=32768, ragged=False, kind="bf16"),
        # chunked prefill of grouped heads
        dict(name="attn_chunk_gqa", op="attn", B=2, T=2000, Hq=32, Hkv=4, d=128, P=64, L=16384, ragged=True, kind="bf16"),
        # one step of a parallel-sampling server: last step's branches freed, new ones forked, room reserved
        dict(name="pages_branch", op="branch", S=16, parents=4, P=16, L=1000, width=128, pools=4, room=17, spare=64),
        # a fragmented latent pool packed into its first pages
        dict(name="pages_compact", op="compact", S=64, pages=8192, P=64, width=576, pools=1, live=0.6),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["rope", "append", "attn", "attn", "attn", "branch", "compact", "copy"])
    if op == "rope":
        d = rng.choice([64, 96, 128, 192, 576])
        rot = rng.choice([r for r in (16, 32, 64, 128) if r <= d])
        T = log(1, 2000)
        return dict(op=op, B=rng.randint(1, 4), T=T, H=log(1, 64), d=d, rot=rot, offset=rng.choice([0, d - rot]), into=0,
                    L=T + log(1, 200000), inter=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "yarn"]),
                    factor=rng.choice([2.0, 4.0, 8.0]), orig=8192, theta=rng.choice([10000.0, 500000.0]),
                    dtype=rng.choice(["bf16", "fp32"]), grad=rng.random() < 0.5) if d * T < 400000 else \
            dict(op=op, B=1, T=T, H=8, d=d, rot=rot, offset=0, into=0, L=T, inter=True, scaling="none", factor=1.0,
                 orig=0, theta=10000.0, dtype="bf16", grad=False)
    if op == "append":
        e4m3 = rng.random() < 0.5
        mla = e4m3 or rng.random() < 0.5
        T = log(1, 4000)
        return dict(op=op, B=rng.randint(1, 8), T=T, H=1 if mla else rng.choice([1, 2, 8]), d=576 if mla else rng.choice([64, 128]),
                    rot=rng.choice([0, 64]), offset=512 if mla else 0, P=rng.choice([16, 32, 64, 128]), L=T + log(1, 6000),
                    ragged=rng.random() < 0.7, e4m3=e4m3, inter=rng.random() < 0.5)
    if op == "attn":
        P = rng.choice([16, 32, 64, 128])
        if rng.random() < 0.5:   # latent rows
            Hq = rng.choice([1, 7, 16, 32, 64, 128])
            L = log(1, 100000)
            T = min(L, log(1, max(2, min(700, 3000000000 // (L * Hq * 100)))))
            return dict(op=op, B=rng.randint(1, 4), T=T, Hq=Hq, Hkv=1, d=576, P=P, L=L, ragged=rng.random() < 0.5,
                        kind=rng.choice(["bf16", "bf16", "e4m3"]))
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 8])
        L = log(1, 60000)
        T = min(L, log(1, max(2, min(2500, 1500000000 // (L * Hkv * G * 20)))))
        return dict(op=op, B=rng.randint(1, 4), T=T, Hq=Hkv * G, Hkv=Hkv, d=rng.choice([64, 128]), P=P, L=L,
                    ragged=rng.random() < 0.5, kind="bf16")
    if op == "branch":
        S = rng.choice([4, 17, 64, 200])
        return dict(op=op, S=S, parents=rng.randint(1, max(1, S // 4)), P=rng.choice([16, 32, 64, 128]), L=log(1, 6000),
                    width=rng.choice([64, 576]), pools=rng.randint(1, 4), room=log(1, 300), spare=rng.randint(0, 200))
    if op == "compact":
        return dict(op=op, S=rng.randint(1, 40), pages=log(40, 5000), P=rng.choice([16, 64]), width=rng.choice([128, 576]),
                    pools=rng.randint(1, 3), live=rng.uniform(0.05, 0.95))
    return dict(op=op, n=log(1, 800), pages=2000, P=rng.choice([16, 64]), width=rng.choice([64, 128, 576]),
                pools=rng.randint(1, 3))


# ------------------------------------------------- lengths that a case stands for
def _lens(c):
    """Cached tokens of each sequence, the new ones included."""
    L, B = c["L"], c["B"]
    return [max(1, L - (b * L) // (2 * B)) if c.get("ragged") else L for b in range(B)]


def _qlens(c):
    """New tokens of each sequence (a shorter sequence of a ragged batch brings a shorter chunk)."""
    T, B = c["T"], c["B"]
    n = [max(1, T - (b * T) // (2 * B)) if c.get("ragged") else T for b in range(B)]
    return [min(x, y) for x, y in zip(n, _lens(c))]


def _pages(n, P):
    return (n + P - 1) // P


def _fork_pages(c):
    """(pages of one parent, full ones) for the branch case's parents, lengths falling from L."""
    lens = [max(1, c["L"] - 3 * i) for i in range(c["parents"])]
    return lens


def work(c):
    op = c["op"]
    if op == "rope":
        es = 2 if c["dtype"] == "bf16" else 4
        n = c["B"] * c["T"] * c["H"] * c["d"] * (2 if c["grad"] else 1)
        return {"bytes": 2 * n * es, "flops": 3 * n * c["rot"] // c["d"]}
    if op == "append":
        rows = sum(_qlens(c))
        n = rows * c["H"] * c["d"]
        return {"bytes": n * (3 if c["e4m3"] else 4) + (4 * rows if c["e4m3"] else 0), "flops": 3 * rows * c["H"] * c["rot"]}
    if op == "attn":
        dv = 512 if c["d"] == 576 else c["d"]
        lens, ql = _lens(c), _qlens(c)
        row = c["d"] + 4 if c["kind"] == "e4m3" else 1152 if c["d"] == 576 else 4 * c["Hkv"] * c["d"]
        cache = sum(lens) * row
        nq = sum(ql) * c["Hq"]
        pairs = sum(q * (n - q) + q * (q + 1) // 2 for n, q in zip(lens, ql)) * c["Hq"]
        return {"bytes": cache + nq * (2 * c["d"] + 2 * dv + 4), "flops": 2 * pairs * (c["d"] + dv)}
    if op == "branch":
        lens = _fork_pages(c)
        kids = c["S"] - c["parents"]
        tails = sum(1 for i in range(kids) if lens[i % c["parents"]] % c["P"])
        mapped = sum(_pages(lens[i % c["parents"]] + c["room"], c["P"]) for i in range(kids))
        return {"bytes": 2 * tails * c["pools"] * c["P"] * c["width"] * 2 + 12 * mapped, "flops": 0}
    if op == "compact":
        n = int(c["pages"] * c["live"])
        moved = n * (c["pages"] - n) // c["pages"]          # what a random half-full pool has to move
        return {"bytes": 2 * moved * c["pools"] * c["P"] * c["width"] * 2 + 8 * n + 8 * c["pages"], "flops": 0}
    return {"bytes": 2 * c["n"] * c["pools"] * c["P"] * c["width"] * 2, "flops": 0}


# ------------------------------------------------------------------ the inputs
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _plan(rot, theta, inter, scaling="none", factor=1.0, orig=0):
    """What a program keeps for its rotary positions: the numbers, and the framework's plan."""
    p = dict(rot=rot, theta=theta, inter=inter, scaling=scaling, factor=factor, orig=orig)
    if own:
        from kv_indexing_b200 import lsa as L
        p["plan"] = L.lsa_rope_plan(rot, theta, interleaved=inter, scaling=scaling, factor=factor, orig_len=orig)
    return p


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    op = c["op"]
    if op == "rope":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        shape = (c["B"], c["T"], c["H"], c["d"])
        s = dict(c=c, x=normal(*shape, dtype=dt), seq_len=_ints([c["L"] - 5 * b if c["L"] > c["T"] + 40 else c["L"] for b in range(c["B"])]),
                 plan=_plan(c["rot"], c["theta"], c["inter"], c["scaling"], c["factor"], c["orig"]))
        wide = torch.zeros(c["B"], c["T"], c["H"], c["into"] or c["d"], device="cuda", dtype=dt)
        s["out"] = wide[..., wide.shape[-1] - c["d"]:]       # the rotary columns of the full query rows
        if c["grad"]:
            s["gy"], s["gx"] = normal(*shape, dtype=dt), torch.zeros(shape, device="cuda", dtype=dt)
        return s
    if op in ("append", "attn"):
        lens, P = _lens(c), c["P"]
        need = [_pages(n, P) for n in lens]
        n_pages = sum(need) + 3
        perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((c["B"], max(need) + 1), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        s = dict(c=c, table=table, seq_len=_ints(lens), q_len=_ints(_qlens(c)))
        if op == "append":
            s["x"] = normal(c["B"], c["T"], c["H"], c["d"])
            s["plan"] = _plan(c["rot"], 10000.0, c["inter"]) if c["rot"] else None
            shape = (n_pages, P, c["H"], c["d"])
            if c["e4m3"]:
                s["pool"] = torch.zeros(shape, device="cuda").to(torch.float8_e4m3fn)
                s["scales"] = torch.ones(n_pages, P, device="cuda")
            else:
                s["pool"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
            return s
        s["q"] = normal(c["B"], c["T"], c["Hq"], c["d"])
        dv = 512 if c["d"] == 576 else c["d"]
        s["scale"] = 1.0 / math.sqrt(c["d"])
        s["out"] = torch.zeros(c["B"], c["T"], c["Hq"], dv, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(c["B"], c["T"], c["Hq"], device="cuda")
        if c["kind"] == "e4m3":
            s["kv"] = torch.empty(n_pages, P, 576, dtype=torch.float8_e4m3fn, device="cuda")
            s["kv_scale"] = torch.empty(n_pages, P, device="cuda")
            for at in range(0, n_pages, 2048):                # in pieces: the rows in 32 bits are four times the cache
                x = normal(min(2048, n_pages - at), P, 576, dtype=torch.float32)
                sc = x.abs().amax(-1) / 448.0
                s["kv"][at:at + 2048] = (x / sc[..., None]).to(torch.float8_e4m3fn)
                s["kv_scale"][at:at + 2048] = sc
        elif c["d"] == 576:
            s["kv"] = torch.empty(n_pages, P, 576, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        else:
            s["k"] = torch.empty(n_pages, P, c["Hkv"], c["d"], dtype=torch.bfloat16, device="cuda").normal_(generator=g)
            s["v"] = torch.empty(n_pages, P, c["Hkv"], c["d"], dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        return s
    if op == "branch":
        lens, P, S, n_par = _fork_pages(c), c["P"], c["S"], c["parents"]
        need = [_pages(n, P) for n in lens]
        kids = S - n_par
        n_pages = sum(need) + kids * (_pages(c["room"], P) + 2) + c["spare"]
        perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((S, _pages(c["L"] + c["room"], P) + 1), -1, dtype=torch.int32, device="cuda")
        ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = perm[at:at + n]
            ref[perm[at:at + n].long()] = 1
            at += n
        order = torch.randperm(kids, generator=g, device="cuda").to(torch.int32)
        parent = (torch.arange(kids, device="cuda", dtype=torch.int32) % n_par).contiguous()
        child = (order + n_par).contiguous()
        new_len = torch.zeros(S, dtype=torch.int32, device="cuda")
        all_lens = _ints(lens)
        new_len[child.long()] = all_lens[parent.long()] + c["room"]
        seq_len = torch.zeros(S, dtype=torch.int32, device="cuda")
        seq_len[:n_par] = all_lens
        return dict(c=c, table=table, ref=ref, seq_len=seq_len, new_len=new_len, parent=parent, child=child,
                    pools=[normal(n_pages, P, c["width"]) for _ in range(c["pools"])])
    if op == "compact":
        n_pages, S = c["pages"], c["S"]
        n = int(n_pages * c["live"])
        perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)[:n]
        per = _pages(max(n, 1), S)
        table = torch.full((S, per + 2), -1, dtype=torch.int32, device="cuda")
        for i in range(S):
            part = perm[i * per:(i + 1) * per]
            table[i, :part.numel()] = part
        ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        ref[perm.long()] = 1
        if S > 1 and n:                                       # a shared first page
            first = table[0, 0].clone()
            table[S - 1, per] = first
            ref[first.long()] += 1
        return dict(c=c, table=table, ref=ref, table_out=torch.empty_like(table), ref_out=torch.empty_like(ref),
                    n_live=torch.zeros(1, dtype=torch.int32, device="cuda"),
                    pools=[normal(n_pages, c["P"], c["width"]) for _ in range(c["pools"])])
    perm = torch.randperm(c["pages"], generator=g, device="cuda").to(torch.int32)
    return dict(c=c, src=perm[:c["n"]].contiguous(), dst=perm[c["n"]:2 * c["n"]].contiguous(),
                pools=[normal(c["pages"], c["P"], c["width"]) for _ in range(c["pools"])])


# ---------------------------------------------------------------- plain forms
def _freqs(p, device):
    """(rotation frequencies in 64 bits, amplitude)."""
    rot, theta = p["rot"], p["theta"]
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    f = theta ** (-2.0 * i / rot)
    if p["scaling"] == "linear":
        return f / p["factor"], 1.0
    if p["scaling"] == "yarn":
        def dim(turns):
            return rot * math.log(p["orig"] / (turns * 2.0 * math.pi)) / (2.0 * math.log(theta))
        low, high = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
        return f * (1.0 - ramp) + f / p["factor"] * ramp, 0.1 * math.log(p["factor"]) + 1.0
    return f, 1.0


def _turn(x, pos, p, offset, inverse=False):
    """x [B,T,H,d] in 32 bits with the columns [offset, offset + rot) turned by the positions [B,T]."""
    f, m = _freqs(p, x.device)
    a = pos.double()[..., None] * f
    cos, sin = (m * torch.cos(a)).float()[:, :, None], (m * torch.sin(a)).float()[:, :, None]
    if inverse:
        sin = -sin
    rot = p["rot"]
    r = x[..., offset:offset + rot]
    x0, x1 = (r[..., 0::2], r[..., 1::2]) if p["inter"] else (r[..., :rot // 2], r[..., rot // 2:])
    y0, y1 = x0 * cos - x1 * sin, x1 * cos + x0 * sin
    y = torch.stack((y0, y1), -1).flatten(-2) if p["inter"] else torch.cat((y0, y1), -1)
    return torch.cat((x[..., :offset], y, x[..., offset + rot:]), -1)


def _plain_rope(s):
    c = s["c"]
    pos = s["seq_len"][:, None] - c["T"] + torch.arange(c["T"], device="cuda")
    s["out"].copy_(_turn(s["x"].float(), pos, s["plan"], c["offset"]))
    if not c["grad"]:
        return s["out"]
    s["gx"].copy_(_turn(s["gy"].float(), pos, s["plan"], c["offset"], True))
    return s["out"], s["gx"]


def _plain_append(s):
    c, P = s["c"], s["c"]["P"]
    t = torch.arange(c["T"], device="cuda")
    pos = s["seq_len"][:, None] - s["q_len"][:, None] + t
    live = (t < s["q_len"][:, None]) & (pos >= 0)
    x = s["x"].float()
    if s["plan"] is not None:
        x = _turn(x, pos, s["plan"], c["offset"])
    at = torch.where(live, pos, 0)
    page = s["table"].gather(1, (at // P)).long()
    slot = (page * P + at % P)[live]
    rows = x[live].reshape(-1, c["H"] * c["d"])
    if c["e4m3"]:
        amax = rows.abs().amax(-1)
        scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        codes = (rows / scale[:, None]).to(torch.float8_e4m3fn)
        s["pool"].view(torch.uint8).view(-1, c["d"])[slot] = codes.view(torch.uint8)
        s["scales"].view(-1)[slot] = scale
        return s["pool"], s["scales"]
    s["pool"].view(-1, c["H"] * c["d"])[slot] = rows.to(torch.bfloat16)
    return s["pool"]


def _plain_attn(s):
    c = s["c"]
    B, T, Hq, Hkv, d = c["B"], c["T"], c["Hq"], c["Hkv"], c["d"]
    page = s["table"].clamp_min(0).long()
    if d == 576:
        kv = s["kv"][page].float()                                       # [B, pages, P, 576]
        if c["kind"] == "e4m3":
            kv = kv * s["kv_scale"][page][..., None]
        k = kv.reshape(B, 1, -1, 576)
        v = k[..., :512]
    else:
        k = s["k"][page].float().reshape(B, -1, Hkv, d).transpose(1, 2)  # [B, Hkv, tokens, d]
        v = s["v"][page].float().reshape(B, -1, Hkv, d).transpose(1, 2)
    G = Hq // Hkv
    q = s["q"].float().reshape(B, T, Hkv, G, d).transpose(1, 2).reshape(B, Hkv, T * G, d)
    sc = torch.matmul(q, k.transpose(-1, -2))
    sc *= s["scale"]
    t = torch.arange(T, device="cuda")
    pos = s["seq_len"][:, None] - s["q_len"][:, None] + t                # [B, T]
    seen = torch.arange(k.shape[2], device="cuda") <= pos[..., None]     # [B, T, tokens]
    sc.view(B, Hkv, T, G, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    sc -= m
    sc.exp_()
    l = sc.sum(-1, keepdim=True)
    o = torch.matmul(sc, v) / l
    o = o.reshape(B, Hkv, T, G, -1).transpose(1, 2).reshape(B, T, Hq, -1)
    lse = (m + l.log()).reshape(B, Hkv, T, G).transpose(1, 2).reshape(B, T, Hq)
    new = t < s["q_len"][:, None]                                        # rows past a sequence's chunk stay as they were
    s["out"].copy_(torch.where(new[..., None, None], o.to(torch.bfloat16), s["out"]))
    s["lse"].copy_(torch.where(new[..., None], lse, s["lse"]))
    return s["out"], s["lse"]


def _plain_branch(s):
    table, ref, seq_len, P = s["table"], s["ref"], s["seq_len"], s["c"]["P"]
    parent, child = s["parent"].long(), s["child"].long()
    # the last step's branches are freed
    old = table[child]
    ref.index_add_(0, old.clamp_min(0).flatten().long(), -(old >= 0).flatten().int())
    table[child] = -1
    seq_len[child] = 0
    # fork: full pages shared, a partly filled one copied into the lowest free pages
    n = seq_len[parent]
    full, rest = n // P, n % P
    j = torch.arange(table.shape[1], device="cuda")
    rows = torch.where(j < full[:, None], table[parent], -1)
    ref.index_add_(0, rows.clamp_min(0).flatten().long(), (rows >= 0).flatten().int())
    free = torch.nonzero(ref == 0).flatten()
    k = torch.cumsum((rest > 0).int(), 0) - 1
    fresh = free[k.clamp_min(0)].int()
    rows = torch.where((j == full[:, None]) & (rest[:, None] > 0), fresh[:, None], rows)
    has = torch.nonzero(rest > 0).flatten()
    src, dst = table[parent[has], full[has].long()].long(), fresh[has].long()
    for pool in s["pools"]:
        pool[dst] = pool[src]
    ref[dst] = 1
    table[child] = rows
    seq_len[child] = n
    # room for the tokens to come, sequence by sequence
    want = (s["new_len"] + P - 1) // P
    miss = (j < want[:, None]) & (table < 0)
    free = torch.nonzero(ref == 0).flatten()
    where = torch.nonzero(miss)
    got = free[:where.shape[0]].int()
    table[where[:, 0], where[:, 1]] = got
    ref[got.long()] = 1
    return table, ref, seq_len, s["pools"]


def _plain_compact(s):
    live = s["ref"] > 0
    n = live.sum()
    i = torch.arange(live.numel(), device="cuda")
    src, dst = torch.nonzero(live & (i >= n)).flatten(), torch.nonzero(~live & (i < n)).flatten()
    for pool in s["pools"]:
        pool[dst] = pool[src]
    to = i.clone()
    to[src] = dst
    s["table_out"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp_min(0).long()].int(), s["table"]))
    s["ref_out"].copy_(s["ref"])
    s["ref_out"][dst] = s["ref"][src]
    s["ref_out"][src] = 0
    s["n_live"].copy_(n)
    return s["table_out"], s["ref_out"], s["n_live"], s["pools"]


def _plain_copy(s):
    for pool in s["pools"]:
        pool[s["dst"].long()] = pool[s["src"].long()]
    return s["pools"]


# --------------------------------------------------- the framework's operators
def _own(s):
    from kv_indexing_b200 import lsa as L
    c = s["c"]
    op = c["op"]
    if op == "rope":
        y = L.lsa_rope(s["x"], s["plan"]["plan"], s["seq_len"], offset=c["offset"], out=s["out"])
        if not c["grad"]:
            return y
        return y, L.lsa_rope(s["gy"], s["plan"]["plan"], s["seq_len"], offset=c["offset"], inverse=True, out=s["gx"])
    if op == "append":
        plan = s["plan"]["plan"] if s["plan"] is not None else None
        L.lsa_pages_append(s["x"], s["table"], s["seq_len"], s["pool"], q_len=s["q_len"], scale_pool=s.get("scales"),
                           plan=plan, offset=c["offset"])
        return (s["pool"], s["scales"]) if c["e4m3"] else s["pool"]
    if op == "attn":
        kv = dict(kv=s["kv"], kv_scale=s.get("kv_scale"), d_v=512) if c["d"] == 576 else dict(k=s["k"], v=s["v"])
        return L.lsa_paged_attn(s["q"], s["table"], s["seq_len"], s["scale"], q_len=s["q_len"], out=s["out"],
                                lse=s["lse"], **kv)
    if op == "branch":
        P = c["P"]
        L.lsa_pages_free(s["table"], s["ref"], s["seq_len"], s["child"])
        L.lsa_pages_fork(s["table"], s["ref"], s["seq_len"], P, s["parent"], s["child"], s["pools"])
        L.lsa_pages_reserve(s["table"], s["ref"], s["new_len"], P)
        return s["table"], s["ref"], s["seq_len"], s["pools"]
    if op == "compact":
        L.lsa_pages_compact(s["table"], s["ref"], s["pools"], table_out=s["table_out"], ref_out=s["ref_out"],
                            n_live=s["n_live"])
        return s["table_out"], s["ref_out"], s["n_live"], s["pools"]
    L.lsa_pages_copy(s["pools"], s["src"], s["dst"])
    return s["pools"]


def run(s):
    if own:
        return _own(s)
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn, "branch": _plain_branch,
            "compact": _plain_compact, "copy": _plain_copy}[s["c"]["op"]](s)


# ------------------------------------------------ the definitions, in 64 bits
def _exact_turn(x, pos, p, offset, sign):
    """The complex form: (x0 + i x1) times m e^(i sign pos f), pair by pair."""
    rot, y = p["rot"], x.double().clone()
    for i in range(rot // 2):
        f, m = p["theta"] ** (-2.0 * i / rot), 1.0
        if p["scaling"] == "linear":
            f /= p["factor"]
        if p["scaling"] == "yarn":
            c = [rot * math.log(p["orig"] / (b * 2 * math.pi)) / (2 * math.log(p["theta"])) for b in (32.0, 1.0)]
            lo, hi = max(math.floor(c[0]), 0), min(math.ceil(c[1]), rot - 1)
            r = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f, m = f / p["factor"] * r + f * (1 - r), 1.0 + 0.1 * math.log(p["factor"])
        a, b = (offset + 2 * i, offset + 2 * i + 1) if p["inter"] else (offset + i, offset + i + rot // 2)
        z = torch.complex(x[..., a].double(), x[..., b].double())
        z = z * torch.polar(torch.full_like(pos, m), sign * pos * f)[:, :, None]
        y[..., a], y[..., b] = z.real, z.imag
    return y


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "rope":
        pos = torch.stack([torch.arange(int(n) - c["T"], int(n), device="cuda") for n in s["seq_len"]]).double()
        y = _exact_turn(s["x"], pos, s["plan"], c["offset"], 1.0)
        return (y, _exact_turn(s["gy"], pos, s["plan"], c["offset"], -1.0)) if c["grad"] else y
    if op == "append":
        lens, ql, P = _lens(c), _qlens(c), c["P"]
        out, scales = s["pool"].double(), torch.ones(s["pool"].shape[:2], dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            pos = torch.arange(lens[b] - ql[b], lens[b], device="cuda")
            x = s["x"][b:b + 1, :ql[b]].double()
            if s["plan"] is not None:
                x = _exact_turn(x, pos.double()[None], s["plan"], c["offset"], 1.0)
            page = s["table"][b].long()[pos // P]
            if c["e4m3"]:
                a = x[0].abs().amax((-1, -2))
                sc = torch.where(a > 0, a / 448.0, 1.0)
                scales[page, pos % P] = sc
                x = x / sc[None, :, None, None]
            out[page, pos % P] = x[0]
        return (out, scales) if c["e4m3"] else out
    if op == "attn":
        dv = 512 if c["d"] == 576 else c["d"]
        out, lse = s["out"].double(), s["lse"].double()
        G = c["Hq"] // c["Hkv"]
        for b, (n, nq) in enumerate(zip(_lens(c), _qlens(c))):
            tok = torch.arange(n, device="cuda")
            page, slot = s["table"][b].long()[tok // c["P"]], tok % c["P"]
            for h in range(c["Hkv"]):
                if c["d"] == 576:
                    k = s["kv"].view(torch.uint8)[page, slot].view(s["kv"].dtype).double() if c["kind"] == "e4m3" else s["kv"][page, slot].double()
                    k = k * s["kv_scale"][page, slot].double()[:, None] if c["kind"] == "e4m3" else k
                    v = k[:, :dv]
                else:
                    k, v = s["k"][page, slot, h].double(), s["v"][page, slot, h].double()
                step = max(1, 400_000_000 // (n * G))          # queries at a time
                for t in range(0, nq, step):
                    q = s["q"][b, t:min(nq, t + step), h * G:(h + 1) * G].double()
                    sc = torch.einsum("tgd,nd->tgn", q, k) * s["scale"]
                    last = n - nq + t + torch.arange(q.shape[0], device="cuda")
                    sc = sc.masked_fill((tok > last[:, None])[:, None], -math.inf)
                    lse[b, t:t + q.shape[0], h * G:(h + 1) * G] = torch.logsumexp(sc, -1)
                    out[b, t:t + q.shape[0], h * G:(h + 1) * G] = torch.einsum("tgn,nd->tgd", torch.softmax(sc, -1), v)
        return out, lse
    if op == "copy":
        src, dst = s["src"].tolist(), s["dst"].tolist()
        for pool in s["pools"]:
            old = pool.clone()
            pool[dst] = old[src]
        return [p.double() for p in s["pools"]]
    table, ref, moves = s["table"].tolist(), s["ref"].tolist(), []
    if op == "compact":
        n = sum(r > 0 for r in ref)
        holes = iter([p for p in range(n) if ref[p] == 0])
        to = {p: next(holes) for p in range(n, len(ref)) if ref[p] > 0}
        table = [[to.get(p, p) for p in row] for row in table]
        new = list(ref)
        for a, b in to.items():
            new[b], new[a] = ref[a], 0
        ref, moves, tail = new, list(to.items()), [_ints([n])]
    else:
        P, seq = c["P"], s["seq_len"].tolist()
        for p, ch in zip(s["parent"].tolist(), s["child"].tolist()):
            for j in range(seq[p] // P):
                table[ch][j] = table[p][j]
                ref[table[p][j]] += 1
            seq[ch] = seq[p]
        for p, ch in zip(s["parent"].tolist(), s["child"].tolist()):
            if seq[p] % P:
                new = ref.index(0)
                ref[new] = 1
                moves.append((table[p][seq[p] // P], new))
                table[ch][seq[p] // P] = new
        for b, n in enumerate(s["new_len"].tolist()):
            for j in range(_pages(n, P)):
                if table[b][j] < 0:
                    table[b][j] = ref.index(0)
                    ref[table[b][j]] = 1
        tail = [_ints(seq)]
    if moves:
        a, b = zip(*moves)
        for pool in s["pools"]:
            pool[list(b)] = pool[list(a)].clone()
    return (_ints(table), _ints(ref), *tail, [p.double() for p in s["pools"]])
