"""64-bit definition of the window attention with sinks, its gradients, and the error bounds that
the kernels' roundings allow. Dense: small sizes only. CPU or GPU tensors.

Roundings of the kernels: P and dS to bf16 before the second products (half a step: 2^-8 of the
value each), outputs to bf16 (2^-8), fp32 sums (a term of a sum of n: at most n 2^-24 of the sum
of magnitudes), O read back in bf16 by the backward (2^-8 |O|, and O's own error)."""
import math

import torch

H = 2.0 ** -8          # half a bf16 step, relative
E = 2.0 ** -24         # half an fp32 step, relative


def visible(Nq, N, window, sinks, L, device="cpu"):
    p = torch.arange(N - Nq, N, device=device)[:, None]
    j = torch.arange(N, device=device)[None]
    return (j <= p) & (j < L) & (p < L) & ((p - j < window) | (j < sinks))


def attention(Q, K, V, window, sinks, lens=None, scale=0.0, dO=None):
    """Outputs and bounds, as dicts of float64 tensors: O, lse (, dQ, dK, dV)."""
    B, Nq, Hq, d = Q.shape
    N, Hkv = K.shape[1], K.shape[2]
    G, s, dev = Hq // Hkv, scale or 1 / math.sqrt(d), Q.device
    out = {"O": torch.zeros(B, Nq, Hq, d, dtype=torch.float64, device=dev),
           "lse": torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device=dev)}
    if dO is not None:
        out["dQ"] = torch.zeros_like(out["O"])
        out["dK"] = torch.zeros(B, N, Hkv, d, dtype=torch.float64, device=dev)
        out["dV"] = torch.zeros_like(out["dK"])
    tol = {k: torch.zeros_like(v) for k, v in out.items()}
    for b in range(B):
        L = N if lens is None else max(0, min(N, int(lens[b])))
        see = visible(Nq, N, window, sinks, L, dev)
        rows = see.any(1)
        keys = torch.arange(N, device=dev) < L
        for h in range(Hq):
            kv = h // G
            q = torch.where(rows[:, None], Q[b, :, h].double(), 0.0)      # what nothing sees is not used
            k = torch.where(keys[:, None], K[b, :, kv].double(), 0.0)
            v = torch.where(keys[:, None], V[b, :, kv].double(), 0.0)
            x = (s * (q @ k.T)).masked_fill(~see, -math.inf)
            z = torch.logsumexp(x, 1)
            P = torch.where(see, (x - torch.where(rows, z, 0.0)[:, None]).exp(), 0.0)
            o, oa = P @ v, P @ v.abs()
            xe = s * (q.abs() @ k.abs().T).masked_fill(~see, 0.0).amax(1) * (d + 8) * E + 2.0 ** -20   # a logit's error
            out["O"][b, :, h], out["lse"][b, h] = o, z
            tol["O"][b, :, h] = H * (o.abs() + oa) + oa * (2 * xe + 2.0 ** -12)[:, None]
            tol["lse"][b, h] = xe + 2.0 ** -21 * (1 + torch.where(rows, z, 0.0).abs())
            if dO is None:
                continue
            g = torch.where(rows[:, None], dO[b, :, h].double(), 0.0)
            dP, D = g @ v.T, (g * o).sum(1, keepdim=True)
            dS = P * (dP - D)
            De = (g.abs() * tol["O"][b, :, h]).sum(1, keepdim=True) + (g.abs() * o.abs()).sum(1, keepdim=True) * d * E
            dPe = (g.abs() @ v.abs().T) * d * E
            pe = (2 * xe + 2.0 ** -20)[:, None]                            # P's relative error before rounding
            dSe = dS.abs() * (H + pe) + P * (De + dPe) * (1 + H)
            acc = 2.0 ** -12                                               # fp32 sums of up to 4096 terms
            out["dQ"][b, :, h] = s * dS @ k
            tol["dQ"][b, :, h] = s * (dSe + acc * dS.abs()) @ k.abs() + H * out["dQ"][b, :, h].abs()
            out["dK"][b, :, kv] += s * dS.T @ q
            tol["dK"][b, :, kv] += s * (dSe + acc * dS.abs()).T @ q.abs()
            out["dV"][b, :, kv] += P.T @ g
            tol["dV"][b, :, kv] += (P * (H + pe + acc)).T @ g.abs()
    for n in ("dK", "dV"):
        if n in out:
            tol[n] += H * out[n].abs()
    return out, tol


def check(name, got, want, tol):
    got = got.double()
    fin = torch.isfinite(want)
    assert torch.equal(fin, torch.isfinite(got)), f"{name}: finite where it should not be, or the other way round"
    assert torch.equal(got[~fin], want[~fin]), f"{name}: infinities differ"
    over = (got - want)[fin].abs() - tol[fin] - 1e-30
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{name}: {int((over > 0).sum())} of {over.numel()} outside the bound, worst by {worst:.3g}"
