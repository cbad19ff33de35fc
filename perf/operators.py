"""Operator timing cases: sliding-window attention with sinks, and the per-head norm of queries and
keys with their position rotation.

    listed() / draw(rng)   cases (plain dicts)
    prepare(case, seed)    inputs on the GPU
    run(state)             one pass: the framework's kernels where `own` is set, elementary torch otherwise
    work(case)             bytes and operations that one pass cannot do without
    exact(case, seed)      the same outputs in 64 bits, straight from the definition

Case kinds:
  prefill   window attention forward of the last Nq of N tokens        -> O, lse
  train     forward and backward                                       -> O, lse, dQ, dK, dV
  decode    one token per sequence against a (rolling) key/value cache -> o, lse, both caches
  rope      norm + rotation of Q and K                                 -> Q', K'
  rope_train  the same and its backward                                -> Q', K', dQ, dK, dwq, dwk
"""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------------------- cases
def _attn(kind, name, B, Nq, N, Hq, Hkv, d, window, sinks, ragged=False, fused=False):
    return {"name": name, "kind": kind, "B": B, "Nq": Nq, "N": N, "Hq": Hq, "Hkv": Hkv, "d": d,
            "window": window, "sinks": sinks, "ragged": ragged, "fused": fused}


def _decode(name, B, Ncap, Hq, Hkv, d, window, sinks, far):
    return {"name": name, "kind": "decode", "B": B, "Ncap": Ncap, "Hq": Hq, "Hkv": Hkv, "d": d,
            "window": window, "sinks": sinks, "far": far}


def _rope(kind, name, B, N, Hq, Hkv, d, rot, interleaved, norm, factor, far, fused=False):
    return {"name": name, "kind": kind, "B": B, "N": N, "Hq": Hq, "Hkv": Hkv, "d": d, "rot": rot,
            "interleaved": interleaved, "norm": norm, "factor": factor, "far": far, "fused": fused}


def listed():
    return [
        # a windowed layer of the 64K prefill workload
        _attn("prefill", "window prefill 64k", 1, 65536, 65536, 16, 2, 128, 4096, 4),
        # a short prompt through a small layer: launch and ramp dominate
        _attn("prefill", "window prefill 4k d64", 1, 4096, 4096, 4, 1, 64, 512, 0),
        # a chunk of a long prompt against the keys so far, right-padded batch, three heads a group
        _attn("prefill", "window chunk ragged", 3, 777, 5003, 12, 4, 128, 1500, 5, True, False),
        # the training workload's shape with a short window
        _attn("train", "window train 16k", 4, 16384, 16384, 16, 4, 128, 1024, 4),
        # full causal attention as the widest window
        _attn("train", "window train 8k full", 1, 8192, 8192, 16, 2, 128, 8192, 0),
        # padded training batch of odd length at the smaller head size, operands from one projection
        _attn("train", "window train ragged d64", 2, 1999, 1999, 8, 2, 64, 300, 1, True, True),
        # serving: 32 sequences on rolling caches, positions far past the capacity
        _decode("window decode b32", 32, 4100, 32, 8, 128, 4096, 4, True),
        # serving: a single sequence, latency
        _decode("window decode b1", 1, 8192, 16, 2, 128, 1024, 4, False),
        # queries and keys of the 64K prefill workload
        _rope("rope", "norm rope 64k", 1, 65536, 16, 2, 128, 128, False, True, 1.0, False),
        # the training workload's queries and keys, with gradients
        _rope("rope_train", "norm rope train 16k", 4, 16384, 16, 4, 128, 128, False, True, 1.0, False),
        # part of the head rotated, interleaved pairs, stretched positions, no norm, projection slices
        _rope("rope_train", "rope partial d64", 2, 2500, 8, 2, 64, 32, True, False, 4.0, True, True),
        # serving: one token of each of 32 sequences
        _rope("rope", "norm rope decode b32", 32, 1, 32, 8, 128, 128, False, True, 1.0, True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prefill", "prefill", "train", "train", "decode", "decode", "rope", "rope_train"])
    d = rng.choice([64, 128, 128])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    Hkv = rng.choice([1, 2, 4])
    sinks = rng.choice([0, 1, 4, 7, 33])
    B = rng.choice([1, 1, 2, 3])
    if kind in ("prefill", "train"):
        # (a softmax over one key has no gradient to compare: training cases see more)
        few = 48 if kind == "train" else 1
        N = _spread(rng, few, 12000)
        Nq = N if kind == "train" or rng.random() < 0.5 else rng.randint(1, N)
        window = _spread(rng, 2 if kind == "train" else 1, max(2, min(4096, 2 * N)))
        c = _attn(kind, "", B, Nq, N, Hkv * G, Hkv, d, window, sinks, rng.random() < 0.4, rng.random() < 0.4)
        while work(c)["flops"] > 1.5e12:
            c["N"] //= 2
            c["Nq"] = min(c["Nq"], c["N"])
        return c
    if kind == "decode":
        window = _spread(rng, 1, 4096)
        return _decode("", rng.choice([1, 2, 5, 16, 31]), sinks + window + rng.choice([0, 0, 1, 100]), Hkv * G, Hkv,
                       d, window, sinks, rng.random() < 0.6)
    rot = rng.choice([16, 32, d // 2, d, d])
    return _rope(kind, "", B, _spread(rng, 1, 9000), Hkv * G, Hkv, d, rot, rng.random() < 0.5, rng.random() < 0.7,
                 rng.choice([1.0, 1.0, 8.0]), rng.random() < 0.5, rng.random() < 0.5)


def _lens(case):
    """Valid tokens of each sequence: the first is full, the others shorter, the last of three or more empty."""
    B, N = case["B"], case["N"]
    if not case["ragged"]:
        return None
    return [0 if B >= 3 and b == B - 1 else max(1, N - b * (N // 4) - b) for b in range(B)]


def _positions(case):
    """The position of each sequence's new token in a decode step."""
    cap, far = case["Ncap"], case["far"]
    return [cap + 9973 * (b + 1) + b if far else max(0, cap - 1 - (b * cap) // (case["B"] + 1) - cap // 3)
            for b in range(case["B"])]


# -------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV).to(torch.bfloat16)


def _qkv(gen, B, Nq, N, Hq, Hkv, d, fused):
    """Q [B,Nq,Hq,d], K, V [B,N,Hkv,d] bf16; fused: slices of one projection output where the lengths agree."""
    if fused and Nq == N:
        x = _randn(gen, B, N, Hq + 2 * Hkv, d)
        return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    return _randn(gen, B, Nq, Hq, d), _randn(gen, B, N, Hkv, d), _randn(gen, B, N, Hkv, d)


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    if case["kind"] in ("prefill", "train"):
        Nq, N = case["Nq"], case["N"]
        st["Q"], st["K"], st["V"] = _qkv(g, B, Nq, N, Hq, Hkv, d, case["fused"])
        lens = _lens(case)
        st["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
        if case["kind"] == "train":
            st["dO"] = _randn(g, B, Nq, Hq, d)
    elif case["kind"] == "decode":
        st["Kc"], st["Vc"] = _randn(g, B, case["Ncap"], Hkv, d), _randn(g, B, case["Ncap"], Hkv, d)
        st["q"], st["k"], st["v"] = _randn(g, B, Hq, d), _randn(g, B, Hkv, d), _randn(g, B, Hkv, d)
        st["pos"] = torch.tensor(_positions(case), dtype=torch.int32, device=DEV)
        st["status"] = torch.zeros(4, dtype=torch.int32, device=DEV)
    else:
        N, rot = case["N"], case["rot"]
        st["Q"], st["K"], _ = _qkv(g, B, N, N, Hq, Hkv, d, case["fused"])
        e = torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot
        st["inv_freq"] = (10000.0 ** -e / case["factor"]).to(torch.float32)
        st["pos"] = None
        if case["far"]:
            first = torch.arange(B, device=DEV, dtype=torch.int32)[:, None] * 7919 + 120000
            st["pos"] = (first + torch.arange(N, device=DEV, dtype=torch.int32)).contiguous()
        st["wq"] = st["wk"] = None
        if case["norm"]:
            st["wq"] = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
            st["wk"] = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
        if case["kind"] == "rope_train":
            st["dQr"], st["dKr"] = _randn(g, B, N, Hq, d), _randn(g, B, N, Hkv, d)
    return st


# -------------------------------------------------------------------------------- plain forms
def _blocks(x, start, nb, bq):
    """[B,N,H,d] -> fp32 [B,H,nb,bq,d]: tokens start .. start + nb bq, zeros outside the tensor."""
    N = x.shape[1]
    lo, hi = max(start, 0), min(start + nb * bq, N)
    x = x[:, lo:hi].float()
    x = torch.nn.functional.pad(x, (0, 0, 0, 0, lo - start, start + nb * bq - hi))
    return x.reshape(x.shape[0], nb, bq, x.shape[2], x.shape[3]).permute(0, 3, 1, 2, 4)


def _pairs(x, start, nb, bq):
    """Keys of query block i: key blocks i and i + 1, as [B,H,1,nb,2 bq,d]."""
    x = _blocks(x, start, nb + 1, bq)
    return torch.cat([x[:, :, :-1], x[:, :, 1:]], dim=3)[:, :, None]


def _plain_attn(Q, K, V, window, sinks, lens, dO=None):
    """Banded attention: a query block of bq >= window tokens sees its own and the previous key block, and
    the first `sinks` keys on their own."""
    B, Nq, Hq, d = Q.shape
    N, Hkv = K.shape[1], K.shape[2]
    G, off, scale = Hq // Hkv, N - Nq, 1 / math.sqrt(d)
    S = min(sinks, N)
    bq = min(max(window, 64), max(Nq, window if window < N else N))
    nb = -(-Nq // bq)
    q = _blocks(Q, 0, nb, bq).reshape(B, Hkv, G, nb, bq, d)
    k, v = _pairs(K, off - bq, nb, bq), _pairs(V, off - bq, nb, bq)
    ks, vs = (x[:, :S].float().permute(0, 2, 1, 3)[:, :, None, None] for x in (K, V))   # [B,Hkv,1,1,S,d]
    L = torch.full((B,), N, device=Q.device) if lens is None else lens.long()
    L = L.reshape(B, 1, 1, 1, 1, 1)
    i = torch.arange(nb, device=Q.device).reshape(nb, 1, 1)
    p = off + i * bq + torch.arange(bq, device=Q.device)[:, None]
    j = off + (i - 1) * bq + torch.arange(2 * bq, device=Q.device)
    js = torch.arange(S, device=Q.device)
    row = (p < L) & (p < N)
    hide = ~((j >= S) & (j <= p) & (p - j < window) & row)
    hide_s = ~((js <= p) & row)
    s = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(hide, -math.inf)
    z = (q @ ks.transpose(-1, -2)).mul_(scale).masked_fill_(hide_s, -math.inf)
    m = s.amax(-1, keepdim=True)
    if S:
        m = torch.maximum(m, z.amax(-1, keepdim=True))
    m = m.masked_fill(m == -math.inf, 0.0)
    s, z = s.sub_(m).exp_(), z.sub_(m).exp_()
    total = s.sum(-1, keepdim=True) + z.sum(-1, keepdim=True)
    lse = m + total.log()
    some = total.clamp_min(1e-30)
    s, z = s.div_(some), z.div_(some)
    o = s @ v + z @ vs

    def rows(x):       # [B,Hkv,G,nb,bq,c] -> [B,Nq,Hq,c]
        x = x.reshape(B, Hq, nb * bq, x.shape[-1])[:, :, :Nq]
        return x.transpose(1, 2)

    O = rows(o).to(torch.bfloat16)
    out = {"O": O.contiguous(), "lse": rows(lse)[..., 0].transpose(1, 2).contiguous()}
    if dO is None:
        return out
    do = _blocks(dO, 0, nb, bq).reshape(B, Hkv, G, nb, bq, d).masked_fill(~row, 0.0)
    delta = (do * o).sum(-1, keepdim=True)
    dv, dvs = (s.transpose(-1, -2) @ do).sum(2), (z.transpose(-1, -2) @ do).sum((2, 3))
    ds = (do @ v.transpose(-1, -2)).sub_(delta).mul_(s).mul_(scale)
    dz = (do @ vs.transpose(-1, -2)).sub_(delta).mul_(z).mul_(scale)
    dq = ds @ k + dz @ ks
    dk, dks = (ds.transpose(-1, -2) @ q).sum(2), (dz.transpose(-1, -2) @ q).sum((2, 3))

    def keys(x, xs):   # [B,Hkv,nb,2 bq,d] block pairs and [B,Hkv,S,d] -> [B,N,Hkv,d]
        t = x.new_zeros(B, Hkv, nb + 1, bq, d)
        t[:, :, :-1] += x[..., :bq, :]
        t[:, :, 1:] += x[..., bq:, :]
        t = t.reshape(B, Hkv, (nb + 1) * bq, d)
        start = off - bq
        lo, hi = max(start, 0), min(start + (nb + 1) * bq, N)
        full = x.new_zeros(B, Hkv, N, d)
        full[:, :, lo:hi] = t[:, :, lo - start:hi - start]
        full[:, :, :S] += xs
        return full.transpose(1, 2).to(torch.bfloat16).contiguous()

    out["dQ"] = rows(dq).to(torch.bfloat16).contiguous()
    out["dK"], out["dV"] = keys(dk, dks), keys(dv, dvs)
    return out


def _slots(p, sinks, cap):
    return torch.where(p < sinks, p, sinks + (p - sinks) % (cap - sinks))


def _plain_decode(st):
    c = st["case"]
    B, Hq, Hkv, d, W, S, cap = (c[k] for k in ("B", "Hq", "Hkv", "d", "window", "sinks", "Ncap"))
    p = st["pos"].long()[:, None]
    b = torch.arange(B, device=p.device)[:, None]
    own_slot = _slots(p, S, cap)
    st["Kc"][b, own_slot], st["Vc"][b, own_slot] = st["k"][:, None], st["v"][:, None]
    band = p - W + 1 + torch.arange(W, device=p.device)
    first = torch.arange(S, device=p.device).expand(B, S)
    j = torch.cat([first, band], 1)
    see = torch.cat([first <= p, band >= S], 1)
    at = _slots(j.clamp_min(0), S, cap)
    k, v = st["Kc"][b, at].float(), st["Vc"][b, at].float()
    q = st["q"].float().reshape(B, Hkv, Hq // Hkv, d)
    s = torch.einsum("bhgd,bjhd->bhgj", q, k) / math.sqrt(d)
    s = s.masked_fill(~see[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    e = (s - m).exp()
    t = e.sum(-1, keepdim=True)
    o = torch.einsum("bhgj,bjhd->bhgd", e / t, v)
    return {"o": o.reshape(B, Hq, d).to(torch.bfloat16), "lse": (m + t.log()).reshape(B, Hq), "Kc": st["Kc"], "Vc": st["Vc"]}


def _angles(st):
    c = st["case"]
    pos = st["pos"]
    if pos is None:
        pos = torch.arange(c["N"], device=DEV).expand(c["B"], c["N"])
    a = pos.double()[..., None] * st["inv_freq"].double()
    return a.cos().float()[:, :, None], a.sin().float()[:, :, None]


def _rotate(x, cos, sin, rot, interleaved):
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


EPS = 1e-6


def _plain_rope(st):
    c = st["case"]
    cos, sin = _angles(st)
    out = {}
    for n in ("Q", "K"):
        w, x = st["w" + n.lower()], st[n].float()
        r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt() if c["norm"] else torch.ones_like(x[..., :1])
        h = x * r
        y = h * w if c["norm"] else h
        out[n + "r"] = _rotate(y, cos, sin, c["rot"], c["interleaved"]).to(torch.bfloat16)
        if c["kind"] == "rope_train":
            g = _rotate(st["d" + n + "r"].float(), cos, -sin, c["rot"], c["interleaved"])
            if c["norm"]:
                out["dw" + n.lower()] = (g * h).sum((0, 1, 2))
                g = g * w
                g = r * (g - h * (g * h).mean(-1, keepdim=True))
            out["d" + n] = g.to(torch.bfloat16)
    return out


# ------------------------------------------------------------------------------------------ run
def run(st):
    c = st["case"]
    if own:
        return _run_own(st, c)
    if c["kind"] == "decode":
        return _plain_decode(st)
    if c["kind"] in ("rope", "rope_train"):
        return _plain_rope(st)
    return _plain_attn(st["Q"], st["K"], st["V"], c["window"], c["sinks"], st["lens"], st.get("dO"))


def _run_own(st, c):
    import pyramid_top_selection_gb300 as pisa
    if c["kind"] == "decode":
        shape = pisa.make_window_decode_shape(c["B"], c["Ncap"], c["Hq"], c["Hkv"], c["d"], c["window"], c["sinks"])
        o, lse, _ = pisa.window_decode_step(shape, st["pos"], st["Kc"], st["Vc"], st["q"], st["k"], st["v"],
                                            status=st["status"])
        return {"o": o, "lse": lse, "Kc": st["Kc"], "Vc": st["Vc"]}
    if c["kind"] in ("rope", "rope_train"):
        shape = pisa.rope_shape_of(st["Q"], st["K"], c["rot"], c["interleaved"], norm=c["norm"], eps=EPS)
        Qr, Kr = pisa.qk_norm_rope(st["Q"], st["K"], st["inv_freq"], shape, st["wq"], st["wk"], st["pos"])
        out = {"Qr": Qr, "Kr": Kr}
        if c["kind"] == "rope_train":
            dQ, dK, dwq, dwk = pisa.qk_norm_rope_bwd(st["Q"], st["K"], st["dQr"], st["dKr"], st["inv_freq"], shape,
                                                     st["wq"], st["wk"], st["pos"])
            out |= {"dQ": dQ, "dK": dK}
            if c["norm"]:
                out |= {"dwq": dwq, "dwk": dwk}
        return out
    shape = pisa.window_shape_of(st["Q"], st["K"], st["V"], c["window"], c["sinks"])
    O, lse = pisa.window_attn_fwd(st["Q"], st["K"], st["V"], shape, lens=st["lens"])
    out = {"O": O, "lse": lse}
    if c["kind"] == "train":
        out["dQ"], out["dK"], out["dV"] = pisa.window_attn_bwd(st["Q"], st["K"], st["V"], O, lse, st["dO"], shape,
                                                               lens=st["lens"])
    return out


# ----------------------------------------------------------------------------------------- work
def _visible(p0, p1, W, S):
    """Sum over positions p0 <= p < p1 of the keys that p sees: min(p + 1, W) + clip(p + 1 - W, 0, S)."""
    def upto(n):       # positions 0 .. n - 1
        a = min(n, W)
        t = a * (a + 1) // 2 + (n - a) * W
        m = max(0, min(n - W, S))
        return t + m * (m + 1) // 2 + max(0, n - W - S) * S
    return upto(max(p1, p0)) - upto(p0)


def work(case):
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    if case["kind"] in ("prefill", "train"):
        Nq, N, W, S = case["Nq"], case["N"], case["window"], case["sinks"]
        lens = _lens(case) or [N] * B
        pairs = keys = rows = 0
        for n in lens:
            lo = N - Nq
            pairs += _visible(min(lo, n), n, W, S) * Hq
            if n > lo:
                keys += min(n, n - lo + W - 1 + S)
                rows += n - lo
        size = 2 * rows * Hq * d + 2 * 2 * keys * Hkv * d + 2 * B * Nq * Hq * d + 4 * B * Hq * Nq
        if case["kind"] == "prefill":
            return {"bytes": size, "flops": 4 * d * pairs}
        # dO in, dQ, dK, dV out: O, lse, Q, K, V read by the backward pass are the forward's
        size += 2 * rows * Hq * d + 2 * B * Nq * Hq * d + 2 * 2 * B * N * Hkv * d
        return {"bytes": size, "flops": 14 * d * pairs}
    if case["kind"] == "decode":
        keys = sum(min(p + 1, case["window"]) + max(0, min(p + 1 - case["window"], case["sinks"])) for p in _positions(case))
        return {"bytes": 2 * 2 * (keys + B) * Hkv * d + 4 * B * Hq * d, "flops": 4 * d * keys * Hq}
    x = B * case["N"] * (Hq + Hkv) * d
    if case["kind"] == "rope":
        return {"bytes": 4 * x, "flops": 8 * x}
    return {"bytes": 8 * x, "flops": 24 * x}


# ---------------------------------------------------------------------------------------- exact
def _exact_attn(st, c):
    """Query chunks against every key they could see, masks written from the rule itself."""
    Q, K, V = st["Q"].double(), st["K"].double(), st["V"].double()
    B, Nq, Hq, d = Q.shape
    N, Hkv = K.shape[1], K.shape[2]
    G, W, S, off = Hq // Hkv, c["window"], c["sinks"], N - Nq
    lens = _lens(c) or [N] * B
    O, lse = torch.zeros_like(Q), torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device=Q.device)
    grads = "dO" in st
    if grads:
        dO = st["dO"].double()
        dQ, dK, dV = torch.zeros_like(Q), torch.zeros_like(K), torch.zeros_like(V)
    C = 1024
    for b in range(B):
        for i0 in range(0, Nq, C):
            i1 = min(i0 + C, Nq, lens[b] - off)
            if i1 <= i0:
                continue
            p = torch.arange(off + i0, off + i1, device=Q.device)
            lo = max(0, off + i0 - W + 1)
            j = torch.cat([torch.arange(min(S, lo), device=Q.device), torch.arange(lo, off + i1, device=Q.device)])
            see = (j[None] <= p[:, None]) & ((p[:, None] - j[None] < W) | (j[None] < S))
            for h in range(Hq):
                q, k, v = Q[b, i0:i1, h], K[b, j, h // G], V[b, j, h // G]
                s = (q @ k.T / math.sqrt(d)).masked_fill(~see, -math.inf)
                z = torch.logsumexp(s, 1)
                P = (s - z[:, None]).exp()
                O[b, i0:i1, h], lse[b, h, i0:i1] = P @ v, z
                if grads:
                    g = dO[b, i0:i1, h]
                    dP = g @ v.T
                    dS = P * (dP - (P * dP).sum(1, keepdim=True)) / math.sqrt(d)
                    dQ[b, i0:i1, h] = dS @ k
                    dK[b].index_put_((j, torch.tensor(h // G, device=Q.device)), dS.T @ q, accumulate=True)
                    dV[b].index_put_((j, torch.tensor(h // G, device=Q.device)), P.T @ g, accumulate=True)
    out = {"O": O, "lse": lse}
    return out | {"dQ": dQ, "dK": dK, "dV": dV} if grads else out


def _exact_decode(st, c):
    B, Hq, Hkv, d, W, S, cap = (c[k] for k in ("B", "Hq", "Hkv", "d", "window", "sinks", "Ncap"))
    o = torch.zeros(B, Hq, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(B, Hq, dtype=torch.float64, device=DEV)
    for b, p in enumerate(_positions(c)):
        slot = [x if x < S else S + (x - S) % (cap - S) for x in range(p + 1) if x < S or p - x < W]
        st["Kc"][b, slot[-1]], st["Vc"][b, slot[-1]] = st["k"][b], st["v"][b]
        k, v = st["Kc"][b, slot].double(), st["Vc"][b, slot].double()
        for h in range(Hq):
            s = k[:, h // (Hq // Hkv)] @ st["q"][b, h].double() / math.sqrt(d)
            lse[b, h] = torch.logsumexp(s, 0)
            o[b, h] = (s - lse[b, h]).exp() @ v[:, h // (Hq // Hkv)]
    return {"o": o, "lse": lse, "Kc": st["Kc"].double(), "Vc": st["Vc"].double()}


def _exact_rope(st, c):
    """The rotation as multiplication by unit complex numbers."""
    B, N, rot, d = c["B"], c["N"], c["rot"], c["d"]
    pos = st["pos"].double() if c["far"] else torch.arange(N, device=DEV).double().repeat(B, 1)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos[:, :, None, None] * st["inv_freq"].double())
    even = torch.arange(0, rot, 2, device=DEV) if c["interleaved"] else torch.arange(rot // 2, device=DEV)
    odd = even + 1 if c["interleaved"] else even + rot // 2

    def turned(x, by):
        y = x.clone()
        z = torch.complex(x[..., even], x[..., odd]) * by
        y[..., even], y[..., odd] = z.real, z.imag
        return y

    out = {}
    for n in ("Q", "K"):
        x = st[n].double()
        w = st["w" + n.lower()].double() if c["norm"] else torch.ones(d, dtype=torch.float64, device=DEV)
        root = torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS) if c["norm"] else torch.ones_like(x[..., :1])
        out[n + "r"] = turned(x / root * w, turn)
        if c["kind"] == "rope_train":
            g = turned(st["d" + n + "r"].double(), turn.conj())
            if c["norm"]:
                out["dw" + n.lower()] = (g * x / root).sum((0, 1, 2))
                g = g * w
                g = g / root - x * (g * x).sum(-1, keepdim=True) / (d * root ** 3)
            out["d" + n] = g
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "decode":
        return _exact_decode(st, case)
    if case["kind"] in ("rope", "rope_train"):
        return _exact_rope(st, case)
    w = work(case)
    return _exact_attn(st, case) if w["flops"] < 6e12 else None
