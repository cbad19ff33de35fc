"""Limits of the window attention and of the query/key norm without a GPU: sizes of workspaces,
refusals of calls that would read or write the wrong memory."""
import ctypes
import random

import pytest
import torch

import pyramid_top_selection_gb300 as pisa
from pyramid_top_selection_gb300 import _pisa

# ------------------------------------------------------------------------ workspace of the backward
# Partial sums: a key tile is cut into runs of at least a 912th of all the row tiles, and at least 16 of them,
# only where it has more than one run; so there are at most twice as many runs as shares, 17/16 for
# rounding a share down to a whole tile, for the tiles with sinks and for those without. (Small problems
# have shorter runs, one a CTA, and fewer.) A run holds dK and dV of 128 keys in fp32.
RUNS = 2 * (2 * 912 * 17 // 16 + 1)


def _backward_bytes(B, Nq, N, Hq, Hkv, d, window, sinks):
    return pisa.window_workspace_size(pisa.make_window_shape(B, Nq, N, Hq, Hkv, d, window, sinks), pisa.WINDOW_BWD)


def _most(B, Nq, Hq, d):
    return 256 + 4096 + 2 * (B * Hq * (Nq + 3) * 4 + 1024) + RUNS * 2 * 128 * d * 4


@pytest.mark.parametrize("B,N,Hq,Hkv,d,window,sinks", [
    (1, 32768, 32, 8, 128, 128, 1024), (4, 16384, 16, 4, 128, 128, 4), (4, 16384, 16, 4, 128, 1, 16384),
    (1, 32768, 8, 8, 128, 128, 32768), (1, 65536, 32, 8, 128, 256, 4096), (1, 1 << 20, 8, 8, 128, 128, 4),
    (1, 1 << 24, 1, 1, 128, 1, 4), (1, 32768, 8, 8, 128, 128, 32000), (2, 8192, 64, 1, 64, 16, 4000),
])
def test_backward_workspace_of_many_sinks_and_short_windows(B, N, Hq, Hkv, d, window, sinks):
    # no more than Q: in the last shape, the tightest, 2 x 912 shares of 64 KB are 120 MB, statistics 8 MB, Q 134 MB
    assert _backward_bytes(B, N, N, Hq, Hkv, d, window, sinks) <= B * N * Hq * d * 2


def test_backward_workspace_is_bounded():
    rng = random.Random(5)
    for _ in range(4000):
        Hkv, G, d, B = rng.randint(1, 16), rng.choice([1, 2, 3, 4, 8, 12, 16, 64]), rng.choice([64, 128]), rng.randint(1, 8)
        N = int(2 ** rng.uniform(0, 24))
        if B * N * Hkv * G >= 1 << 31:
            continue
        Nq = rng.choice([N, rng.randint(1, N)])
        window, sinks = int(2 ** rng.uniform(0, 24)), rng.choice([0, int(2 ** rng.uniform(0, 24))])
        assert _backward_bytes(B, Nq, N, Hkv * G, Hkv, d, window, sinks) <= _most(B, Nq, Hkv * G, d), (B, Nq, N, Hkv, G, d, window, sinks)


def test_sinks_that_meet_the_window_are_full_causal_attention():
    for N, window, sinks in ((32768, 128, 32768), (32768, 128, 32640), (5000, 4999, 1), (5000, 1, 4999), (1, 1, 1)):
        assert _backward_bytes(2, N, N, 8, 2, 128, window, sinks) == _backward_bytes(2, N, N, 8, 2, 128, N, 0)


# ------------------------------------------------------------------------------- overlapping buffers
A = 1 << 24        # fake, 16-byte aligned addresses: never dereferenced


def _overlaps(fn, shape, names, sizes, written, may_be, tail=(None,)):
    """Every buffer in `written` laid over every other one, at its first and its last 16 bytes, is refused by
    name; `may_be`: pairs (written, read) that may be the same buffer (or are refused in other words), but not lie askew."""
    far = {n: A + (k << 20) for k, n in enumerate(names)}
    for w in written:
        for r in names:
            if r == w:
                continue
            for at in (0, max(16, -(-sizes[r] // 16) * 16) - 16):
                if ((w, r) in may_be or (r, w) in may_be) and at == 0:
                    continue
                args = [far[r] + at if n == w else far[n] for n in names]
                rc = fn(ctypes.byref(shape), *args, *tail)
                msg = pisa.lib().pisa_last_error().decode()
                assert rc == _pisa.PISA_EINVAL and (f"{w} overlaps {r}" in msg or f"{r} overlaps {w}" in msg), (w, r, rc, msg)


def test_every_overlap_is_refused():
    # 100 tokens, 4 query heads over 4 KV heads of 64: 51200 bytes a tensor
    L, t = pisa.lib(), 100 * 4 * 64 * 2
    s = pisa.make_window_shape(1, 100, 100, 4, 4, 64, 10)
    need = pisa.window_workspace_size(s, pisa.WINDOW_BWD)
    fwd = ["Q", "K", "V", "len", "O", "lse", "workspace"]
    size = dict(Q=t, K=t, V=t, O=t, dO=t, dQ=t, dK=t, dV=t, len=4, lse=1600)
    _overlaps(L.pisa_window_attn_fwd, s, fwd, size | dict(workspace=256), ["O", "lse", "workspace"], [], (256, None))
    bwd = ["Q", "K", "V", "O", "lse", "dO", "len", "dQ", "dK", "dV", "workspace"]
    _overlaps(L.pisa_window_attn_bwd, s, bwd, size | dict(workspace=need), bwd[7:], [], (need, None))
    dec = ["pos", "Kcache", "Vcache", "q", "k_new", "v_new", "o", "lse", "status"]
    size = dict(pos=8, Kcache=2 * t, Vcache=2 * t, q=1024, k_new=1024, v_new=1024, o=1024, lse=32, status=4)
    _overlaps(L.pisa_window_decode_step, pisa.make_window_decode_shape(2, 100, 4, 4, 64, 10), dec, size,
              ["Kcache", "Vcache", "o", "lse", "status"], [("o", "q")])
    r = pisa.make_rope_shape(1, 100, 4, 4, 64, 64)
    size = dict(Q=t, K=t, Qr=t, Kr=t, dQr=t, dKr=t, dQ=t, dK=t, inv_freq=128, q_weight=256, k_weight=256, pos=400,
                dq_weight=256, dk_weight=256)
    _overlaps(L.pisa_qk_norm_rope, r, ["Q", "K", "inv_freq", "q_weight", "k_weight", "pos", "Qr", "Kr"], size,
              ["Qr", "Kr"], [("Qr", "Q"), ("Kr", "K")])
    b = ctypes.c_size_t()
    assert L.pisa_qk_norm_rope_workspace_size(ctypes.byref(r), ctypes.byref(b)) == 0
    bwd = ["Q", "K", "dQr", "dKr", "inv_freq", "q_weight", "k_weight", "pos", "dQ", "dK", "dq_weight", "dk_weight", "workspace"]
    _overlaps(L.pisa_qk_norm_rope_bwd, r, bwd, size | dict(workspace=b.value), bwd[8:], [("dQ", "dQr"), ("dK", "dKr"), ("dQ", "Q"), ("dK", "K")],
              (b.value, None))


# --------------------------------------------------------------------------------- token inputs of a step
def test_decode_step_refuses_token_slices():
    # a token's values as a slice of a fused projection lie H d apart, and the step reads them in a row: with
    # `rope`, q and k_new may be such slices (they pass through the norm), v_new may not
    B, Hq, Hkv, d = 2, 4, 2, 64
    x = torch.zeros(B, Hq + 2 * Hkv, d, dtype=torch.bfloat16)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    cache, pos = torch.zeros(B, 64, Hkv, d, dtype=torch.bfloat16), torch.zeros(B, dtype=torch.int32)
    shape = pisa.make_decode_shape(B, 64, Hq, Hkv, d, 64, 1)
    pyr = torch.zeros(B, Hkv, 1, d)
    for rope in (None, pisa.Rope(torch.zeros(32), d)):
        with pytest.raises(ValueError, match="v_new must be"):
            pisa.decode_step(shape, pos, cache, cache, pyr, q, k, v, rope=rope)


# ---------------------------------------------------------------------------------------------- sizes
@pytest.mark.parametrize("make,kw", [
    (pisa.make_window_shape, dict(B=1, Nq=8, N=8, Hq=2, Hkv=1, d=64, window=4, sinks=0, q_stride=0, k_stride=0, v_stride=0)),
    (pisa.make_window_decode_shape, dict(B=1, Ncap=8, Hq=2, Hkv=1, d=64, window=4, sinks=0)),
    (pisa.make_rope_shape, dict(B=1, N=8, Hq=2, Hkv=1, d=64, rot=64, q_stride=0, k_stride=0)),
])
def test_sizes_past_32_bits_are_refused(make, kw):
    # ctypes would keep the low 32 bits: a window of 2^32 + 4 "for no limit" would be one of 4 keys
    make(**kw)
    for n in kw:
        for bad in (2 ** 32 + kw[n], -2 ** 32 + kw[n], 2 ** 31):
            with pytest.raises(ValueError, match=n):
                make(**{**kw, n: bad})
    if "window" in kw:
        assert make(**{**kw, "window": 2 ** 31 - 1}).window == 2 ** 31 - 1
