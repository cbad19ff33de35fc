"""Operator timing cases: attention over packed documents with capped or distance-biased scores, and a paged
key/value cache in 16 or 4 bits with its append and its attention.

    listed() / draw(rng)   cases (plain dicts)
    prepare(case, seed)    inputs on the GPU
    run(state)             one pass: the framework's kernels where `own` is set, elementary torch otherwise
    work(case)             bytes and operations that one pass cannot do without
    exact(case, seed)      the same outputs in 64 bits, straight from the definition

Case kinds:
  docs        packed documents, forward                                        -> O, lse
  docs_train  forward and backward                                             -> O, lse, dQ, dK, dV
  append      norm, rotation, and keys and values into their pages             -> Qr, pages (and scales)
  paged       the last nq tokens of every sequence against its pages           -> o, lse

A 4-bit page holds e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives) two a byte, the even channel low, and
an e4m3 scale for each 16 channels: value = code x scale x the KV head's factor.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------------------- cases
def _docs(kind, name, docs, shortest, longest, Hq, Hkv, d, cap=0.0, slopes=False, prefix=False, pad=0, empty=False,
          fused=False, mix=1):
    return {"name": name, "kind": kind, "docs": docs, "shortest": shortest, "longest": longest, "Hq": Hq, "Hkv": Hkv,
            "d": d, "cap": cap, "slopes": slopes, "prefix": prefix, "pad": pad, "empty": empty, "fused": fused, "mix": mix}


def _append(name, B, shortest, longest, Hq, Hkv, d, bits, page, rot, norm, interleaved=False, far=False, fused=False,
            pad=0, mix=1):
    return {"name": name, "kind": "append", "B": B, "shortest": shortest, "longest": longest, "Hq": Hq, "Hkv": Hkv, "d": d,
            "bits": bits, "page": page, "rot": rot, "norm": norm, "interleaved": interleaved, "far": far, "fused": fused,
            "pad": pad, "mix": mix}


def _paged(name, B, nq, shortest, longest, Hq, Hkv, d, bits, page, cap=0.0, slopes=False, mix=1):
    return {"name": name, "kind": "paged", "B": B, "nq": nq, "shortest": shortest, "longest": longest, "Hq": Hq, "Hkv": Hkv,
            "d": d, "bits": bits, "page": page, "cap": cap, "slopes": slopes, "mix": mix}


def listed():
    return [
        # prompts of a serving batch, packed, through a layer with capped scores
        _docs("docs", "docs prefill 6 prompts capped", 6, 1500, 8192, 16, 2, 128, cap=20.0),
        # one short prompt through a small layer: launch and ramp dominate
        _docs("docs", "docs prefill 300 d64", 1, 300, 300, 4, 1, 64),
        # the training workload's heads over a packed batch of documents of all lengths
        _docs("docs_train", "docs train packed", 60, 64, 2048, 16, 4, 128, pad=40),
        # one long document with capped scores
        _docs("docs_train", "docs train 8k capped", 1, 8192, 8192, 16, 2, 128, cap=20.0),
        # short documents, distance-biased scores, question prefixes that see themselves, operands from one projection
        _docs("docs_train", "docs train short biased d64", 25, 1, 400, 8, 2, 64, slopes=True, prefix=True, pad=13, empty=True,
              fused=True),
        # packed prompts of a serving batch into 16-bit pages
        _append("append 16 bit prompts", 8, 4000, 8192, 16, 2, 128, 16, 64, 128, True),
        # the same into 4-bit pages, operands from one projection, rows behind the last prompt
        _append("append 4 bit prompts", 6, 100, 2048, 32, 8, 128, 4, 64, 128, True, fused=True, pad=21),
        # serving: one token of each of 32 sequences, far positions
        _append("append 16 bit decode b32", 32, 1, 1, 32, 8, 128, 16, 16, 128, True, far=True),
        # serving: 32 sequences of up to 16K tokens
        _paged("paged 16 bit b32 16k", 32, 1, 4096, 16384, 32, 8, 128, 16, 64),
        # the same in 4 bits
        _paged("paged 4 bit b32 16k", 32, 1, 4096, 16384, 32, 8, 128, 4, 64),
        # serving: one long context, capped scores, latency
        _paged("paged 4 bit b1 128k capped", 1, 1, 131072, 131072, 16, 2, 128, 4, 64, cap=20.0),
        # four drafted tokens a sequence, three heads a group, lengths down to none, distance-biased scores
        _paged("paged 16 bit drafts d64", 6, 4, 0, 3000, 12, 4, 64, 16, 16, slopes=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["docs", "docs_train", "docs_train", "append", "append", "paged", "paged"])
    d = rng.choice([64, 128, 128])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    Hkv = rng.choice([1, 2, 4])
    mix = rng.randrange(1 << 30)
    score = rng.choice(["plain", "cap", "slopes", "both"])
    cap = rng.choice([10.0, 20.0, 50.0]) if score in ("cap", "both") else 0.0
    slopes = score in ("slopes", "both")
    if kind in ("docs", "docs_train"):
        longest = _spread(rng, 48, 4000)
        # (a softmax over one key has no gradient to compare: the longest document always has more)
        c = _docs(kind, "", _spread(rng, 1, 40), rng.choice([1, min(longest, 33), longest]), longest, Hkv * G, Hkv, d, cap, slopes,
                  rng.random() < 0.4, rng.choice([0, 0, 1, 77]), rng.random() < 0.3, rng.random() < 0.4, mix)
        while c["docs"] * c["longest"] ** 2 * c["Hq"] > 1.0e9:
            c["longest"] = max(48, c["longest"] // 2)
            c["shortest"] = min(c["shortest"], c["longest"])
            c["docs"] = max(1, c["docs"] * 2 // 3)
        return c
    bits, page = rng.choice([16, 4]), rng.choice([16, 32, 64, 128])
    if kind == "append":
        longest = rng.choice([1, _spread(rng, 1, 4000)])
        return _append("", rng.choice([1, 2, 5, 16, 31]), rng.choice([1, longest]), longest, Hkv * G, Hkv, d, bits, page,
                       rng.choice([0, 32, d // 2, d, d]), rng.random() < 0.7, rng.random() < 0.5, rng.random() < 0.5,
                       rng.random() < 0.5, rng.choice([0, 0, 1, 9]), mix)
    nq, longest = rng.choice([1, 1, 1, 2, 3, 5]), _spread(rng, 1, 30000)
    return _paged("", rng.choice([1, 2, 5, 16, 31]), nq, rng.choice([0, 1, longest // 2, longest]), longest, Hkv * G, Hkv, d, bits,
                  page, cap, slopes, mix)


def _lengths(case, n):
    """n lengths from the case's shortest to its longest: the first the longest, the last the shortest, their logarithms spread."""
    lo, hi, r = case["shortest"], case["longest"], random.Random(case["mix"])
    out = [min(hi, max(lo, _spread(r, max(1, lo), hi))) for _ in range(n)]
    out[-1] = lo
    out[0] = hi
    return out


def _doc_lengths(case):
    out = _lengths(case, case["docs"])
    return out[:1] + [0] + out[1:] if case["empty"] else out


def _prefixes(case):
    r = random.Random(case["mix"] + 1)
    return [r.randint(0, n) for n in _doc_lengths(case)] if case["prefix"] else None


# -------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(torch.bfloat16)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _slopes(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device=DEV)


def _qkv(gen, T, Hq, Hkv, d, fused, scale):
    """Q [T,Hq,d], K, V [T,Hkv,d] bf16; fused: slices of one projection's output."""
    q = _randn(gen, T, Hq, d, scale=scale)
    if not fused:
        return q, _randn(gen, T, Hkv, d), _randn(gen, T, Hkv, d)
    x = torch.cat([q, _randn(gen, T, 2 * Hkv, d)], 1)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _page_table(gen, lens, page, first=None):
    """Pages of sequences of these lengths in no order, -1 behind each sequence's own (and before the page of its
    token `first`, where earlier ones have been given back), and the pool's size."""
    need = [-(-n // page) for n in lens]
    skip = [n // page for n in first] if first else [0] * len(lens)
    width = max(1, *need)
    pool = sum(need) - sum(skip) + 3
    ids = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
    i = torch.arange(width, device=DEV)
    have = (i < torch.tensor(need, device=DEV)[:, None]) & (i >= torch.tensor(skip, device=DEV)[:, None])
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    table[have] = ids[:pool - 3]
    return table, pool


def _fill(gen, case, pool, st):
    """Pages as earlier steps left them."""
    Hkv, page, d = case["Hkv"], case["page"], case["d"]
    st["k_amp"] = st["v_amp"] = st["ks"] = st["vs"] = None
    if case["bits"] == 16:
        st["k"], st["v"] = _randn(gen, pool, Hkv, page, d), _randn(gen, pool, Hkv, page, d)
        return
    st["k_amp"], st["v_amp"] = (0.25 + torch.rand(Hkv, generator=gen, device=DEV) for _ in range(2))
    for n in ("k", "v"):
        codes, scales = _quantise(_randn(gen, pool, Hkv, page, d).float())
        st[n], st[n + "s"] = codes, scales


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["kind"] in ("docs", "docs_train"):
        lens = _doc_lengths(case)
        T = sum(lens) + case["pad"]
        st["Q"], st["K"], st["V"] = _qkv(g, T, Hq, Hkv, d, case["fused"], 3.0 if case["cap"] else 1.0)
        starts = [0]
        for n in lens:
            starts.append(starts[-1] + n)
        st["starts"] = _ints(starts)
        st["prefix"] = _ints(_prefixes(case)) if case["prefix"] else None
        st["slopes"] = _slopes(Hq) if case["slopes"] else None
        if case["kind"] == "docs_train":
            st["dO"] = _randn(g, T, Hq, d)
        return st
    lens = _lengths(case, case["B"])
    if case["kind"] == "append":
        first = [120000 + 7919 * b if case["far"] else 0 for b in range(case["B"])]
        st["table"], pool = _page_table(g, [f + n for f, n in zip(first, lens)], case["page"], first)
        T = sum(lens) + case["pad"]
        _fill(g, case, pool, st)
        st["Q"], st["K"], st["V"] = _qkv(g, T, Hq, Hkv, d, case["fused"], 1.0)
        st["seq"] = _ints([b for b, n in enumerate(lens) for _ in range(n)] + [-1] * case["pad"])
        st["pos"] = _ints([f + i for f, n in zip(first, lens) for i in range(n)] + [0] * case["pad"])
        e = torch.arange(0, case["rot"], 2, dtype=torch.float64, device=DEV) / max(1, case["rot"])
        st["inv_freq"] = (10000.0 ** -e).to(torch.float32) if case["rot"] else None
        st["wq"], st["wk"] = ((1 + 0.2 * torch.randn(d, generator=g, device=DEV)) if case["norm"] else None for _ in range(2))
        st["Qr"] = torch.zeros(T, Hq, d, dtype=torch.bfloat16, device=DEV)
        st["status"] = torch.zeros(4, dtype=torch.int32, device=DEV)
        st["valid"] = torch.arange(sum(lens), device=DEV)
        st["pairs"] = torch.tensor([[s * c for s in (1, -1) for c in CODES]], device=DEV).expand(2, 16)
        st["pairs"] = torch.stack([st["pairs"][0].repeat(16), st["pairs"][1].repeat_interleave(16)], -1).to(torch.float8_e4m3fn)
        st["pairs"] = st["pairs"].contiguous().view(torch.int16)[:, 0].contiguous()
        return st
    st["lens"] = _ints(lens)
    st["table"], pool = _page_table(g, lens, case["page"])
    _fill(g, case, pool, st)
    st["q"] = _randn(g, case["B"], case["nq"], Hq, d, scale=3.0 if case["cap"] else 1.0)
    st["slopes"] = _slopes(Hq) if case["slopes"] else None
    return st


# -------------------------------------------------------------------------------- plain forms
def _quantise(x):
    """fp32 [.., d] (already over the head's factor) -> e2m1 codes two a byte [.., d/2], e4m3 scales [.., d/16]."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    s = (g.abs().amax(-1) / 6).clamp_max(448.0).to(torch.float8_e4m3fn)
    f = s.float()[..., None]
    a = (g / torch.where(f > 0, f, torch.ones_like(f))).abs()
    c = (a > 0.25).to(torch.uint8)
    for_even = (a >= 0.75, a > 1.25, a >= 1.75, a > 2.5, a >= 3.5, a > 5.0)
    c = c + sum(for_even).to(torch.uint8)
    c = torch.where(f > 0, c, torch.zeros_like(c)) | (torch.signbit(g).to(torch.uint8) << 3)
    c = c.reshape(*x.shape[:-1], -1, 2)
    return c[..., 0] | (c[..., 1] << 4), s


def _dequantise(codes, scales, amp):
    """fp32 values of pages [.., Hkv, page, d/2] and [.., Hkv, page, d/16]."""
    lut = torch.tensor([s * c for s in (1, -1) for c in CODES], device=codes.device)
    x = lut[torch.stack([codes & 15, codes >> 4], -1).int()].flatten(-2)
    x = x.reshape(*x.shape[:-1], -1, 16) * scales.float()[..., None]
    return x.flatten(-2) * amp[:, None, None]


def _scores(x, c, dist, slopes):
    """Scores from the scaled products, and what a gradient is multiplied by on its way back through them."""
    slope = None
    if c["cap"]:
        t = torch.tanh(x.div_(c["cap"]))
        slope = 1 - t * t
        x = t.mul_(c["cap"])
    if slopes is not None:
        x = x - slopes * dist
    return x, slope


def _plain_docs(st):
    """Every document as a row of a padded batch."""
    c, Q = st["case"], st["Q"]
    T, Hq, d = Q.shape
    Hkv, M, dev = c["Hkv"], c["longest"], Q.device
    G, scale = Hq // Hkv, 1 / math.sqrt(d)
    start, end = st["starts"][:-1].long(), st["starts"][1:].long()
    n, i = len(start), torch.arange(M, device=dev)
    here = i < (end - start)[:, None]
    at = torch.where(here, start[:, None] + i, T)                       # [n, M]; T: a row of zeros behind the tokens

    def rows(x, g):                                                     # [T,H,d] -> [n,Hkv,g,M,d]
        x = torch.cat([x.float(), x.new_zeros(1, *x.shape[1:]).float()])[at]
        return x.reshape(n, M, Hkv, g, d).permute(0, 2, 3, 1, 4)

    def back(x, H, dtype):                                              # [n,Hkv,g,M,e] -> [T,H,e]
        x = x.permute(0, 3, 1, 2, 4).reshape(n, M, H, -1)
        return x.new_zeros(T + 1, H, x.shape[-1]).index_put_((at,), x)[:T].to(dtype)

    q, k, v = rows(Q, G), rows(st["K"], 1), rows(st["V"], 1)
    see = i[None] <= i[:, None]
    see = see.expand(n, M, M) if st["prefix"] is None else see | (i < st["prefix"].long()[:, None, None])
    see = (see & here[:, None] & here[:, :, None])[:, None, None]
    slopes = None if st["slopes"] is None else st["slopes"].reshape(Hkv, G, 1, 1)
    x, slope = _scores((q @ k.transpose(-1, -2)).mul_(scale), c, (i[:, None] - i).abs(), slopes)
    x = x.masked_fill_(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0.0)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    lse = m + total.log()
    p = p.div_(total.clamp_min(1e-30))
    o = p @ v
    all_lse = torch.full((T + 1, Hq), -math.inf, device=dev)
    all_lse[at] = lse[..., 0].permute(0, 3, 1, 2).reshape(n, M, Hq)
    out = {"O": back(o, Hq, torch.bfloat16), "lse": all_lse[:T].T.contiguous()}
    if c["kind"] == "docs_train":
        do = rows(st["dO"], G)
        delta = (do * o).sum(-1, keepdim=True)
        out["dV"] = back((p.transpose(-1, -2) @ do).sum(2, keepdim=True), Hkv, torch.bfloat16)
        ds = (do @ v.transpose(-1, -2)).sub_(delta).mul_(p).mul_(scale)
        if slope is not None:
            ds = ds.mul_(slope)
        out["dQ"] = back(ds @ k, Hq, torch.bfloat16)
        out["dK"] = back((ds.transpose(-1, -2) @ q).sum(2, keepdim=True), Hkv, torch.bfloat16)
    return out


def _plain_rope(x, w, cos, sin, c):
    """Norm of every head and rotation of its first `rot` elements, rounded to bf16."""
    x = x.float()
    if c["norm"]:
        x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w
    r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    half = c["rot"] // 2
    a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :half], r[..., half:])
    a, b = a * cos - b * sin, a * sin + b * cos
    r = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1).to(torch.bfloat16)


def _shown(st, pages):
    """The values that 4-bit codes stand for."""
    x = st["pairs"][pages.int()]
    return x.view(torch.float8_e4m3fn).reshape(*pages.shape[:-1], -1)


def _pages_out(st):
    out = {"Qr": st["Qr"]}
    if st["case"]["bits"] == 16:
        return out | {"k": st["k"], "v": st["v"]}
    return out | {"k": _shown(st, st["k"]), "v": _shown(st, st["v"]), "ks": st["ks"], "vs": st["vs"]}


def _plain_append(st):
    c, t = st["case"], st["valid"]
    seq, pos = st["seq"][t].long(), st["pos"][t].long()
    cos = sin = torch.zeros((), device=DEV)
    if c["rot"]:
        a = pos.double()[:, None, None] * st["inv_freq"].double()
        cos, sin = a.cos().float(), a.sin().float()
    st["Qr"][t] = _plain_rope(st["Q"][t], st["wq"], cos, sin, c)
    page, slot = st["table"][seq, pos // c["page"]].long(), pos % c["page"]
    new = {"k": _plain_rope(st["K"][t], st["wk"], cos, sin, c), "v": st["V"][t]}
    if c["bits"] == 16:
        st["k"][page, :, slot], st["v"][page, :, slot] = new["k"], new["v"]
    else:
        for_k = _quantise(new["k"].float() / st["k_amp"][:, None])
        for_v = _quantise(new["v"].float() / st["v_amp"][:, None])
        st["k"][page, :, slot], st["v"][page, :, slot] = for_k[0], for_v[0]
        st["ks"].view(torch.uint8)[page, :, slot], st["vs"].view(torch.uint8)[page, :, slot] = (x[1].view(torch.uint8)
                                                                                              for x in (for_k, for_v))
    return _pages_out(st)


def _plain_paged(st):
    c = st["case"]
    B, nq, Hq, Hkv, d = c["B"], c["nq"], c["Hq"], c["Hkv"], c["d"]
    at = st["table"].long().clamp_min(0)

    def keys(n):                                                        # [B,Hkv,1,tokens,d]
        x = st[n][at]
        x = x.float() if c["bits"] == 16 else _dequantise(x, st[n + "s"].view(torch.uint8)[at].view(torch.float8_e4m3fn), st[n + "_amp"])
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, 1, -1, d)

    k = keys("k")
    q = st["q"].float().reshape(B, nq, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4)
    j = torch.arange(k.shape[3], device=k.device)
    p = st["lens"].long()[:, None] - nq + torch.arange(nq, device=k.device)
    see = (j <= p[..., None])[:, None, None]                            # [B,1,1,nq,tokens]
    slopes = None if st["slopes"] is None else st["slopes"].reshape(Hkv, Hq // Hkv, 1, 1)
    dist = (p[..., None] - j).abs()[:, None, None]
    x, _ = _scores((q @ k.transpose(-1, -2)).div_(math.sqrt(d)), c, dist, slopes)
    x = x.masked_fill_(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0.0)
    e = x.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    o = e.div_(total.clamp_min(1e-30)) @ keys("v")

    def rows(x):                                                        # [B,Hkv,G,nq,e] -> [B,nq,Hq,e]
        return x.permute(0, 3, 1, 2, 4).reshape(B, nq, Hq, -1)

    return {"o": rows(o).to(torch.bfloat16), "lse": rows(m + total.log())[..., 0].contiguous()}


# ------------------------------------------------------------------------------------------ run
def run(st):
    if own:
        return _run_own(st, st["case"])
    if st["case"]["kind"] == "append":
        return _plain_append(st)
    return _plain_paged(st) if st["case"]["kind"] == "paged" else _plain_docs(st)


def _run_own(st, c):
    import pyramid_top_selection_gb300 as pisa
    if c["kind"] in ("docs", "docs_train"):
        shape = pisa.doc_shape_of(st["Q"], st["K"], st["V"], st["starts"], max_len=c["longest"], cap=c["cap"])
        O, lse = pisa.doc_attn_fwd(st["Q"], st["K"], st["V"], st["starts"], shape, prefix=st["prefix"], slopes=st["slopes"])
        out = {"O": O, "lse": lse}
        if c["kind"] == "docs_train":
            out["dQ"], out["dK"], out["dV"] = pisa.doc_attn_bwd(st["Q"], st["K"], st["V"], O, lse, st["dO"], st["starts"],
                                                                shape, prefix=st["prefix"], slopes=st["slopes"])
        return out
    cache = pisa.PagedCache(st["k"], st["v"], st["ks"], st["vs"], st["k_amp"], st["v_amp"])
    shape = pisa.paged_shape_of(cache, st["table"], c["Hq"], nq=c.get("nq", 1), cap=c.get("cap", 0.0))
    if c["kind"] == "append":
        rope = pisa.Rope(st["inv_freq"], c["rot"], c["interleaved"], c["norm"], EPS, 1.0, st["wq"], st["wk"])
        pisa.paged_append(shape, cache, st["table"], st["pos"], st["K"], st["V"], Q=st["Q"], seq=st["seq"], rope=rope,
                          q_out=st["Qr"], status=st["status"])
        return _pages_out(st)
    o, lse = pisa.paged_attn(shape, cache, st["table"], st["lens"], st["q"], slopes=st["slopes"])
    return {"o": o, "lse": lse}


# ----------------------------------------------------------------------------------------- work
def work(case):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["kind"] in ("docs", "docs_train"):
        lens = _doc_lengths(case)
        pre = _prefixes(case) or [0] * len(lens)
        # i <= j below the prefix: all pairs of it, not half of them
        pairs = sum(n * (n + 1) // 2 + p * (p - 1) // 2 for n, p in zip(lens, pre)) * Hq
        n, T = sum(lens), sum(lens) + case["pad"]
        size = 2 * n * (Hq + 2 * Hkv) * d + 2 * T * Hq * d + 4 * T * Hq
        if case["kind"] == "docs":
            return {"bytes": size, "flops": 4 * d * pairs}
        # dO in, dQ, dK, dV out: O, lse, Q, K, V read by the backward pass are the forward's
        return {"bytes": size + 2 * n * Hq * d + 2 * T * (Hq + 2 * Hkv) * d, "flops": 14 * d * pairs}
    held = {16: 2 * d, 4: d // 2 + d // 16}[case["bits"]]                # bytes of a page's row
    lens = _lengths(case, case["B"])
    if case["kind"] == "append":
        n = sum(lens)
        return {"bytes": n * (4 * Hq * d + 4 * Hkv * d + 2 * Hkv * held), "flops": 8 * n * (Hq + 2 * Hkv) * d}
    nq = case["nq"]
    pairs = sum(max(0, n - nq + 1 + i) for n in lens for i in range(nq)) * Hq
    return {"bytes": 2 * sum(lens) * Hkv * held + case["B"] * nq * Hq * (4 * d + 4), "flops": 4 * d * pairs}


# ---------------------------------------------------------------------------------------- exact
def _exact_docs(st, c):
    """Document by document and head by head, masks written from the rule itself."""
    Q, K, V = st["Q"].double(), st["K"].double(), st["V"].double()
    T, Hq, d = Q.shape
    G = Hq // c["Hkv"]
    O, lse = torch.zeros_like(Q), torch.full((Hq, T), -math.inf, dtype=torch.float64, device=Q.device)
    train = c["kind"] == "docs_train"
    if train:
        dO = st["dO"].double()
        dQ, dK, dV = torch.zeros_like(Q), torch.zeros_like(K), torch.zeros_like(V)
    pre = _prefixes(c)
    at = 0
    for x, n in enumerate(_doc_lengths(c)):
        a, b = at, at + n
        at = b
        if n == 0:
            continue
        i = torch.arange(n, device=Q.device)
        hide = i[None] > i[:, None]
        if pre is not None:
            hide = hide & (i[None] >= pre[x])
        for h in range(Hq):
            q, k, v = Q[a:b, h], K[a:b, h // G], V[a:b, h // G]
            s = q @ k.T / math.sqrt(d)
            if c["cap"]:
                th = torch.tanh(s / c["cap"])
                s = c["cap"] * th
            if c["slopes"]:
                s = s - st["slopes"][h].double() * (i[:, None] - i[None]).abs()
            s = s.masked_fill(hide, -math.inf)
            z = torch.logsumexp(s, 1)
            P = (s - z[:, None]).exp()
            O[a:b, h], lse[h, a:b] = P @ v, z
            if train:
                g = dO[a:b, h]
                dP = g @ v.T
                dS = P * (dP - (P * dP).sum(1, keepdim=True))
                if c["cap"]:
                    dS = dS * (1 - th * th)
                dS = dS / math.sqrt(d)
                dQ[a:b, h] = dS @ k
                dK[a:b, h // G] += dS.T @ q
                dV[a:b, h // G] += P.T @ g
    out = {"O": O, "lse": lse}
    return out | {"dQ": dQ, "dK": dK, "dV": dV} if train else out


def _exact_turned(x, w, st, c):
    """The rotation as multiplication by unit complex numbers."""
    x, t, rot = x[st["valid"]].double(), st["valid"], c["rot"]
    if c["norm"]:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["d"] + EPS) * w.double()
    if rot:
        by = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), st["pos"][t].double()[:, None, None] * st["inv_freq"].double())
        even = torch.arange(0, rot, 2, device=x.device) if c["interleaved"] else torch.arange(rot // 2, device=x.device)
        odd = even + 1 if c["interleaved"] else even + rot // 2
        z = torch.complex(x[..., even], x[..., odd]) * by
        x = x.clone()
        x[..., even], x[..., odd] = z.real, z.imag
    return x


def _exact_append(st, c):
    Qr = st["Qr"].double()
    Qr[st["valid"]] = _exact_turned(st["Q"], st["wq"], st, c)
    k, v = _exact_turned(st["K"], st["wk"], st, c), st["V"][st["valid"]].double()
    seq, pos = st["seq"][st["valid"]].long(), st["pos"][st["valid"]].long()
    page, slot = st["table"][seq, pos // c["page"]].long(), pos % c["page"]
    if c["bits"] == 16:
        out = {"Qr": Qr, "k": st["k"].double(), "v": st["v"].double()}
        out["k"][page, :, slot], out["v"][page, :, slot] = k, v
        return out
    # The nearest code of each value, ties to the even one. (Keys are rounded to bf16 before, by definition: where that
    # and the scale's rounding fall is decided in too few digits for a value in 64 bits; they have none here.)
    grid = torch.tensor(CODES, dtype=torch.float64, device=v.device)
    x = (v / st["v_amp"].double()[:, None]).reshape(*v.shape[:-1], -1, 16)
    s = ((v.float() / st["v_amp"][:, None]).reshape(x.shape).abs().amax(-1) / 6).to(torch.float8_e4m3fn)
    a = x.abs() / s.double()[..., None].clamp_min(2.0 ** -9)
    off = (a[..., None] - grid).abs()
    code = off.argmin(-1)
    up = (code + 1).clamp_max(7)
    tie = torch.gather(off, -1, up[..., None])[..., 0] == off.amin(-1)
    code = torch.where(tie & (code % 2 == 1), up, code)
    vals = (grid[code] * torch.sign(x) * (s.double()[..., None] > 0)).flatten(-2)
    held = _shown(st, st["v"]).double()
    held[page, :, slot] = vals
    scales = st["vs"].double()
    scales[page, :, slot] = s.double()
    return {"Qr": Qr, "k": None, "v": held, "ks": None, "vs": scales}


def _exact_paged(st, c):
    B, nq, Hq, Hkv, d, page = (c[k] for k in ("B", "nq", "Hq", "Hkv", "d", "page"))
    lut = torch.tensor([s * v for s in (1, -1) for v in CODES], dtype=torch.float64, device=DEV)
    o = torch.zeros(B, nq, Hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((B, nq, Hq), -math.inf, dtype=torch.float64, device=DEV)

    def row(n, b, length, h):
        ids = st["table"][b, :-(-length // page)].long()
        x = st[n][ids, h].reshape(-1, st[n].shape[-1])[:length]
        if c["bits"] == 16:
            return x.double()
        s = st[n + "s"].view(torch.uint8)[ids, h].reshape(-1, d // 16)[:length].view(torch.float8_e4m3fn).double()
        y = torch.empty(length, d, dtype=torch.float64, device=DEV)
        y[:, 0::2], y[:, 1::2] = lut[(x % 16).long()], lut[(x // 16).long()]
        return y * s.repeat_interleave(16, 1) * st[n + "_amp"][h].double()

    for b, length in enumerate(_lengths(c, B)):
        for kv in range(Hkv):
            if length == 0:
                continue
            k, v = row("k", b, length, kv), row("v", b, length, kv)
            for h in range(kv * Hq // Hkv, (kv + 1) * Hq // Hkv):
                for i in range(max(0, nq - length), nq):
                    p = length - nq + i
                    s = k[:p + 1] @ st["q"][b, i, h].double() / math.sqrt(d)
                    if c["cap"]:
                        s = c["cap"] * torch.tanh(s / c["cap"])
                    if c["slopes"]:
                        s = s - st["slopes"][h].double() * (p - torch.arange(p + 1, device=DEV))
                    lse[b, i, h] = torch.logsumexp(s, 0)
                    o[b, i, h] = (s - lse[b, i, h]).exp() @ v[:p + 1]
    return {"o": o, "lse": lse}


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "append":
        return _exact_append(st, case)
    if case["kind"] == "paged":
        return _exact_paged(st, case)
    return _exact_docs(st, case) if sum(n * n for n in _doc_lengths(case)) * case["Hq"] < 3e9 else None
