"""64-bit definitions of the attention over packed documents and over a paged cache, of the cache's 4-bit codes, and the
error bounds that the kernels' roundings allow. Dense: small sizes only. CPU or GPU tensors.

Roundings of the kernels: P and dS to bf16 (4-bit caches: P to fp16, which is less) before the second products, half a
step: 2^-8 of the value each; outputs to bf16 (2^-8); fp32 sums; O read back in bf16 by the backward. Scores: a sum of d products
in fp32 (at most (d + 8) 2^-24 of the sum of magnitudes), the cap's tanh within 2^-21 and the factor 1 - tanh^2 within
2^-19, the distance's share within 2^-22 of itself, the exponent of 2 within 2^-22 of itself."""
import math

import torch

from _window_ref import E, H

CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def head(q, k, v, see, scale, cap=0.0, slope=0.0, dist=None, g=None):
    """One head: q, g [n,d], k, v [m,d] float64, see [n,m]. Outputs and bounds, dK and dV before their bf16 rounding."""
    d = q.shape[1]
    x = scale * (q @ k.T)
    xe = scale * (q.abs() @ k.abs().T) * (d + 8) * E
    back = torch.ones_like(x)
    if cap:
        t = torch.tanh(x / cap)
        back = 1 - t * t
        x = cap * t
        xe = xe + cap * 2.0 ** -21
    if slope:
        x = x - slope * dist
        xe = xe + abs(slope) * dist * 2.0 ** -22
    xe = xe + x.abs() * 2.0 ** -22 + 2.0 ** -21
    rows = see.any(1)
    x = x.masked_fill(~see, -math.inf)
    z = torch.logsumexp(x, 1)
    P = torch.where(see, (x - torch.where(rows, z, 0.0)[:, None]).exp(), 0.0)
    ze = (P * xe).sum(1)                                               # the sum's relative error
    pe = xe + ze[:, None] + 2.0 ** -20                                 # P's, before its rounding
    o = P @ v
    out = {"O": o, "lse": z}
    tol = {"O": H * o.abs() + (P * (H + pe + 2.0 ** -12)) @ v.abs(),
           "lse": ze + 2.0 ** -21 * (1 + torch.where(rows, z, 0.0).abs())}
    if g is not None:
        acc = 2.0 ** -12                                               # fp32 sums of up to 4096 terms
        dP, D = g @ v.T, (g * o).sum(1, keepdim=True)
        dS = P * (dP - D) * back
        De = (g.abs() * tol["O"]).sum(1, keepdim=True) + (g.abs() * o.abs()).sum(1, keepdim=True) * d * E
        dPe = (g.abs() @ v.abs().T) * d * E
        # P (x + ex) (b + eb) with x = dP - D, b = 1 - tanh^2 is off by P (|b| ex + |x| eb + ex eb), ex = De + dPe, eb = 2^-19
        # (the last term is what remains where x and b are both 0)
        dSe = dS.abs() * (H + pe) + P * back.abs() * (De + dPe) * (1 + H) + P * ((dP - D).abs() + De + dPe) * 2.0 ** -19 * bool(cap)
        out |= {"dQ": scale * dS @ k, "dK": scale * dS.T @ q, "dV": P.T @ g}
        tol |= {"dQ": scale * (dSe + acc * dS.abs()) @ k.abs() + H * out["dQ"].abs(),
                "dK": scale * (dSe + acc * dS.abs()).T @ q.abs(), "dV": (P * (H + pe + acc)).T @ g.abs()}
    return out, tol


def doc_mask(T, starts, prefix, device="cpu"):
    """Which keys each of T rows sees."""
    see = torch.zeros(T, T, dtype=torch.bool, device=device)
    i = torch.arange(T, device=device)
    for m in range(len(starts) - 1):
        s, e = max(0, starts[m]), min(T, starts[m + 1])
        if s >= e:
            continue
        pre = s + (prefix[m] if prefix is not None else 0)
        own = (i >= s) & (i < e)
        see |= own[:, None] & own[None] & ((i[None] <= i[:, None]) | (i[None] < pre))
    return see


def doc_attention(Q, K, V, starts, prefix=None, slopes=None, cap=0.0, scale=0.0, dO=None):
    """Outputs and bounds, as dicts of float64 tensors: O, lse (, dQ, dK, dV)."""
    T, Hq, d = Q.shape
    Hkv = K.shape[1]
    G, scale, dev = Hq // Hkv, scale or 1 / math.sqrt(d), Q.device
    see = doc_mask(T, starts, prefix, dev)
    rows = see.any(1)
    i = torch.arange(T, device=dev)
    dist = (i[:, None] - i[None]).abs().double()
    clean = lambda x: torch.where(rows[:, None], x.double(), 0.0)      # noqa: E731 (a row sees itself or is padding)
    kinds = ["O", "lse"] + (["dQ", "dK", "dV"] if dO is not None else [])
    size = {"O": (T, Hq, d), "lse": (Hq, T), "dQ": (T, Hq, d), "dK": (T, Hkv, d), "dV": (T, Hkv, d)}
    out = {n: torch.zeros(size[n], dtype=torch.float64, device=dev) for n in kinds}
    tol = {n: torch.zeros_like(v) for n, v in out.items()}
    for h in range(Hq):
        kv = h // G
        o, t = head(clean(Q[:, h]), clean(K[:, kv]), clean(V[:, kv]), see, scale, cap, float(slopes[h]) if slopes is not None else 0.0,
                    dist, None if dO is None else clean(dO[:, h]))
        for n in kinds:
            at = h if n == "lse" else (slice(None), kv if n in ("dK", "dV") else h)
            out[n][at] += o[n]
            tol[n][at] += t[n]
    for n in ("dK", "dV"):
        if n in out:
            tol[n] += H * out[n].abs()
    return out, tol


def paged_attention(q, k, v, lens, slopes=None, cap=0.0, scale=0.0, hidden=None):
    """q [B,nq,Hq,d] against k, v: lists of [tokens,Hkv,d] float64 (a sequence's keys in order). hidden: per sequence a
    mask of keys that are not seen."""
    B, nq, Hq, d = q.shape
    G, scale, dev = Hq // k[0].shape[1], scale or 1 / math.sqrt(d), q.device
    out = {"O": torch.zeros(B, nq, Hq, d, dtype=torch.float64, device=dev),
           "lse": torch.full((B, nq, Hq), -math.inf, dtype=torch.float64, device=dev)}
    tol = {n: torch.zeros_like(x) for n, x in out.items()}
    for b, n in enumerate(lens):
        if n == 0:
            continue
        p = torch.arange(n - nq, n, device=dev)[:, None]
        j = torch.arange(n, device=dev)[None]
        see = j <= p
        if hidden is not None:
            see = see & ~hidden[b][None]
        for h in range(Hq):
            o, t = head(q[b, :, h].double(), k[b][:n, h // G], v[b][:n, h // G], see, scale, cap,
                        float(slopes[h]) if slopes is not None else 0.0, (p - j).abs().double())
            out["O"][b, :, h], out["lse"][b, :, h] = o["O"], o["lse"]
            tol["O"][b, :, h], tol["lse"][b, :, h] = t["O"], t["lse"]
    return out, tol


def quantise(x):
    """x [.., d] float64 (over the head's factor) -> codes [.., d] (0 .. 15) and scales [.., d/16] as float64: the scale the
    e4m3 value nearest to a sixth of the group's largest magnitude, each code the nearest one, ties to the even."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    bad = ~torch.isfinite(g).all(-1)
    g = torch.where(bad[..., None], 0.0, g)
    e4m3 = torch.tensor([(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1], dtype=torch.float64)
    e4m3 = torch.cat([torch.arange(8, dtype=torch.float64) * 2.0 ** -9, e4m3]).to(x.device)
    s = _nearest(g.abs().amax(-1) / 6, e4m3)
    s = e4m3[s]
    a = g.abs() / torch.where(s > 0, s, 1.0)[..., None]
    c = _nearest(a, torch.tensor(CODES, dtype=torch.float64, device=x.device))
    c = torch.where(s[..., None] > 0, c, 0) + 8 * torch.signbit(g)
    s = torch.where(bad, math.nan, s)
    return c.flatten(-2), s


def _nearest(a, grid):
    """Index of the grid's value nearest to a >= 0, ties to the even index."""
    hi = torch.searchsorted(grid, a.contiguous()).clamp_max(len(grid) - 1)
    lo = (hi - 1).clamp_min(0)
    dl, dh = a - grid[lo], grid[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0)) | (hi == lo)
    return torch.where(up, hi, lo)


def codes_of(pages):
    """[.., d/2] bytes -> [.., d] codes."""
    return torch.stack([pages & 15, pages >> 4], -1).flatten(-2).long()


def values_of(pages, scales, amp=None):
    """The float64 values of 4-bit pages [.., Hkv, page, d/2] with scales [.., Hkv, page, d/16]."""
    lut = torch.tensor([s * c for s in (1, -1) for c in CODES], dtype=torch.float64, device=pages.device)
    x = lut[codes_of(pages)] * scales.double().repeat_interleave(16, -1)
    return x if amp is None else x * amp.double()[:, None, None]
