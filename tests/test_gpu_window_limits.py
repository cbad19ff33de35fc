"""Window attention at its limits on the GPU, against the 64-bit definition (_window_ref.py)."""
import math

import pytest
import torch

import pyramid_top_selection_gb300 as pisa
from _window_ref import attention, check

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


def _inputs(B, Nq, N, Hq, Hkv, d, lens=None, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    Q, K, V, dO = (torch.randn(B, n, h, d, generator=g, device="cuda").to(bf16)
                   for n, h in ((Nq, Hq), (N, Hkv), (N, Hkv), (Nq, Hq)))
    for b, L in enumerate(lens or []):     # what lies past a sequence's tokens is never used
        K[b, L:], V[b, L:] = math.nan, math.inf
        r = max(0, L - (N - Nq))
        Q[b, r:], dO[b, r:] = math.nan, -math.inf
    return Q, K, V, dO


def _run(Q, K, V, dO, window, sinks, lens=None):
    s = pisa.window_shape_of(Q, K, V, window, sinks)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    O, lse = pisa.window_attn_fwd(Q, K, V, s, lens=ln)
    ws = pisa.window_workspace(s, pisa.WINDOW_BWD, Q.device).fill_(0xAB)
    grads = pisa.window_attn_bwd(Q, K, V, O, lse, dO, s, lens=ln, ws=ws)
    assert pisa.workspace_status(ws) == 0
    return dict(zip(("O", "lse", "dQ", "dK", "dV"), (O, lse, *grads)))


@pytest.mark.parametrize("B,Nq,N,Hq,Hkv,d,window,sinks,lens", [
    (1, 3000, 3000, 8, 2, 64, 16, 600, None),
    (2, 2500, 2500, 4, 4, 128, 5, 40, [2500, 1201]),
    (1, 700, 2600, 16, 1, 128, 1, 2000, None),
    (3, 900, 900, 24, 8, 64, 130, 300, [900, 17, 0]),
    (1, 2000, 2000, 6, 2, 128, 3, 1990, [1999]),
    (2, 4000, 4000, 2, 1, 64, 1, 129, None),
    (4, 2300, 2300, 8, 8, 64, 20, 1, None),
])
def test_many_sinks_and_short_windows(B, Nq, N, Hq, Hkv, d, window, sinks, lens):
    # the rows of a key tile with sinks are cut into runs of their own length
    Q, K, V, dO = _inputs(B, Nq, N, Hq, Hkv, d, lens, seed=N)
    got, again = (_run(Q, K, V, dO, window, sinks, lens) for _ in range(2))
    want, tol = attention(Q, K, V, window, sinks, lens, dO=dO)
    for n in want:
        check(n, got[n], want[n], tol[n])
        assert torch.equal(got[n], again[n]), n


@pytest.mark.parametrize("window,sinks", [(1, 700), (300, 400), (650, 50), (1, 5000)])
def test_sinks_that_meet_the_window_are_full_causal_attention(window, sinks):
    Q, K, V, dO = _inputs(2, 700, 700, 8, 2, 64, [700, 431], seed=3)
    a, b = _run(Q, K, V, dO, window, sinks, [700, 431]), _run(Q, K, V, dO, 700, 0, [700, 431])
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_decode_output_in_place_of_the_query():
    B, Ncap, Hq, Hkv, d = 3, 400, 32, 2, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(bf16)       # noqa: E731
    Kc, Vc, q, k, v = rnd(B, Ncap, Hkv, d), rnd(B, Ncap, Hkv, d), rnd(B, Hq, d), rnd(B, Hkv, d), rnd(B, Hkv, d)
    shape = pisa.make_window_decode_shape(B, Ncap, Hq, Hkv, d, 300, 4)
    pos = torch.tensor([399, 20, 5000], dtype=torch.int32, device="cuda")
    want = pisa.window_decode_step(shape, pos, Kc.clone(), Vc.clone(), q, k, v)
    got = pisa.window_decode_step(shape, pos, Kc, Vc, q, k, v, o=q)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(pisa.PisaError, match="Kcache overlaps lse"):
        pisa.window_decode_step(shape, pos, Kc, Vc, q, k, v, lse=Kc.view(torch.float32).reshape(-1)[:B * Hq].reshape(B, Hq))


def test_decode_steps_from_slices_of_a_projection():
    # with `rope`, q and k_new may be slices; a v_new that is one is refused by both steps, not misread
    B, Ncap, Hq, Hkv, d, L = 2, 512, 8, 2, 128, 200
    g = torch.Generator(device="cuda").manual_seed(6)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(bf16)       # noqa: E731
    Kc, Vc, x = rnd(B, Ncap, Hkv, d), rnd(B, Ncap, Hkv, d), rnd(B, Hq + 2 * Hkv, d)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    rope = pisa.Rope(pisa.rope_frequencies(d)[0].cuda(), d)
    pos = torch.tensor([L, L - 60], dtype=torch.int32, device="cuda")
    dshape, wshape = pisa.make_decode_shape(B, Ncap, Hq, Hkv, d, 64, 4), pisa.make_window_decode_shape(B, Ncap, Hq, Hkv, d, 64, 4)

    def selected(q, k, v):
        K, V = Kc.clone(), Vc.clone()
        return (*pisa.decode_step(dshape, pos, K, V, pisa.decode_build_pyramid(K, pos, dshape), q, k, v, rope=rope)[:2], K, V)

    def window(q, k, v):
        K, V = Kc.clone(), Vc.clone()
        return (*pisa.window_decode_step(wshape, pos, K, V, q, k, v, rope=rope)[:2], K, V)

    for step in (selected, window):
        for a, b in zip(step(q, k, v.contiguous()), step(q.contiguous(), k.contiguous(), v.contiguous())):
            assert torch.equal(a, b)
        with pytest.raises(ValueError, match="v_new must be"):
            step(q, k, v)
    with pytest.raises(ValueError, match="q must be"):
        pisa.decode_step(dshape, pos, Kc, Vc, pisa.decode_build_pyramid(Kc, pos, dshape), q, k.contiguous(), v.contiguous())


@pytest.mark.parametrize("first,end", [(0, 64), (16, 32), (0, 299), (100, 300), (0, 300)])
@pytest.mark.parametrize("Hq,d", [(6, 64), (32, 128)])
def test_logits_of_minus_infinity(first, end, Hq, d):
    # keys with scores of -inf weigh nothing, though they be all that one warp of the decode step, or one key tile
    # of the forward, has: as if these keys were not there; a row of nothing else is an empty one
    N, Hkv = 300, 2
    Q, K, V, _ = _inputs(1, N, N, Hq, Hkv, d, seed=12)
    Q[..., 0] = 1.0
    K[:, first:end, :, 0] = -math.inf
    O, lse = pisa.window_attn_fwd(Q, K, V, pisa.window_shape_of(Q, K, V, N))
    shape = pisa.make_window_decode_shape(1, N, Hq, Hkv, d, N)
    k, v = K[:, -1].clone(), V[:, -1].clone()
    o, l, _ = pisa.window_decode_step(shape, torch.tensor([N - 1], dtype=torch.int32, device="cuda"), K.clone(), V.clone(),
                                      Q[:, -1].contiguous(), k, v)
    seen = [j for j in range(N) if not first <= j < end]
    if not seen:
        want = {"O": torch.zeros(1, 1, Hq, d, device="cuda"), "lse": torch.full((1, Hq, 1), -math.inf, device="cuda")}
        tol = {n: torch.zeros_like(x) for n, x in want.items()}
    else:
        want, tol = attention(Q[:, -1:], K[:, seen], V[:, seen], len(seen), 0)
    check("O", O[:, -1:], want["O"], tol["O"])
    check("lse", lse[..., -1:], want["lse"], tol["lse"])
    check("o", o, want["O"][:, 0], tol["O"][:, 0])
    check("l", l, want["lse"][..., 0], tol["lse"][..., 0])


def _inv_2pi(bits):
    """1 / (2 pi) as an integer over 2^bits, by Machin's formula."""
    one = 1 << (bits + 64)

    def arctan_of_one_over(x):
        t = s = one // x
        n = 1
        while t:
            t //= -x * x
            n += 2
            s += t // n
        return s

    pi = 4 * (4 * arctan_of_one_over(5) - arctan_of_one_over(239))
    return (one << bits) // (2 * pi)


@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_of_any_frequency_and_position(interleaved):
    # pairs (1, 0) turned by pos * inv_freq, against integer arithmetic with 512 digits of 1 / (2 pi)
    f = torch.tensor([1.0, 0.1, 3.7e-5, 2.0 ** -40, 1e-38, 0.0, -0.75, 1000.5, 65536.25, -12345.678, 1e7, 2.0 ** 24 + 2, 1.7e12,
                      -3.1e19, 2.5e30, 3.4e38])
    pos = [0, 1, -1, 12345, 10**6 + 3, 2**24 + 1, 2**31 - 1, -2**31, -2**31 + 7, 1999999999]
    x = torch.zeros(1, len(pos), 1, 64, dtype=bf16, device="cuda")
    x[..., 0:32:2 if interleaved else 1] = 1.0
    if not interleaved:
        x[..., 16:32] = 0.0
    p = torch.tensor([pos], dtype=torch.int32, device="cuda")
    y, z = pisa.qk_norm_rope(x, x, f.cuda(), pisa.rope_shape_of(x, x, 32, interleaved, norm=False), pos=p)
    assert torch.equal(y, z)
    y = y[0, :, 0, :32].double().cpu()
    c, s = (y[:, 0::2], y[:, 1::2]) if interleaved else (y[:, :16], y[:, 16:])
    inv = _inv_2pi(512)
    want = torch.zeros(2, len(pos), 16, dtype=torch.float64)
    for i, q in enumerate(pos):
        for k, v in enumerate(f.tolist()):
            num, den = v.as_integer_ratio()
            turns = (q * num * inv // den) % (1 << 512) / (1 << 512)
            want[:, i, k] = torch.tensor([math.cos(2 * math.pi * turns), math.sin(2 * math.pi * turns)])
    # bf16's half step, and 2^-18 for the angle in fp32 (2^-24 of pi) and its cosine and sine (2^-21)
    for got, w in ((c, want[0]), (s, want[1])):
        assert float(((got - w).abs() - 2.0 ** -8 * w.abs()).max()) <= 2.0 ** -18
