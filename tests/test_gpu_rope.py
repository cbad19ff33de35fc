"""Per-head norm of queries and keys with the rotation by position, forward and backward, against
a 64-bit computation (rotation as multiplication by unit complex numbers); the operators run
together: projections -> norm and rotation -> window attention and pyramid selection -> decode."""
import math

import pytest
import torch

import pyramid_top_selection_gb300 as pisa
from _window_ref import E, H, attention, check

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


def _turn(x, pos, inv_freq, rot, interleaved, scale, back=False):
    y = x.clone()
    if rot:
        a = pos.double()[..., None, None] * inv_freq.double()
        t = torch.polar(torch.full_like(a, scale), -a if back else a)
        c = torch.arange(rot // 2, device=x.device)
        e, o = (2 * c, 2 * c + 1) if interleaved else (c, c + rot // 2)
        z = torch.complex(x[..., e], x[..., o]) * t
        y[..., e], y[..., o] = z.real, z.imag
    return y


def _reference(x, w, pos, inv_freq, rot, interleaved, norm, eps, scale, dy=None):
    """Output (and dx, dw) with bounds: bf16 outputs round by half a step; fp32 arithmetic and the
    angle's cosine and sine (absolute error under 2^-20) act on the pair's magnitudes."""
    x = x.double()
    d = x.shape[-1]
    w = torch.ones(d, dtype=torch.float64, device=x.device) if w is None else w.double()
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt() if norm else torch.ones_like(x[..., :1])
    h = x * r
    y = h * w if norm else h
    a = _turn(y, pos, inv_freq, rot, interleaved, scale)
    size = lambda v: v.square().amax(-1, keepdim=True).sqrt() * scale          # noqa: E731
    out = {"y": (a, H * a.abs() + 2.0 ** -18 * size(y) * (1 if norm or rot else 0))}
    if dy is not None:
        g = _turn(dy.double(), pos, inv_freq, rot, interleaved, scale, back=True)
        ge = 2.0 ** -18 * size(dy.double())
        if norm:
            dims = tuple(range(x.dim() - 1))
            rows = x[..., 0].numel()
            out["dw"] = ((g * h).sum(dims), (ge * h.abs() + (g * h).abs() * (2.0 ** -20 + math.sqrt(rows) * 4 * E)).sum(dims))
            gw = g * w
            dot = (gw * h).mean(-1, keepdim=True)
            dx = r * (gw - h * dot)
            e = r * ((ge + 2.0 ** -20 * g.abs()) * w.abs() + h.abs() * ((ge + 2.0 ** -18 * g.abs()) * (w * h).abs()).mean(-1, keepdim=True)
                     + 2.0 ** -20 * (h * dot).abs())
            out["dx"] = (dx, H * dx.abs() + e)
        else:
            out["dx"] = (g, H * g.abs() + ge * (1 if rot else 0))
    return out


CASES = {  # B, N, Hq, Hkv, d, rot, interleaved, norm, eps, rot_scale, weights, pos, fused
    "one token": (1, 1, 1, 1, 128, 128, False, True, 1e-6, 1.0, True, None, False),
    "half split": (2, 77, 8, 2, 128, 128, False, True, 1e-6, 1.0, True, None, False),
    "interleaved": (2, 77, 8, 2, 128, 128, True, True, 1e-6, 1.0, True, None, False),
    "d 64": (1, 300, 5, 3, 64, 64, False, True, 1e-5, 1.0, True, None, True),
    "d 64 interleaved": (3, 50, 4, 1, 64, 64, True, True, 1e-5, 1.0, False, None, True),
    "part of the head": (2, 33, 6, 2, 128, 48, False, True, 1e-6, 1.5, True, "far", True),
    "part, interleaved": (2, 33, 7, 1, 64, 16, True, True, 1e-6, 0.7, True, "far", False),
    "rotation only": (1, 129, 12, 4, 128, 32, False, False, 0.0, 1.25, False, "far", True),
    "rotation only, interleaved": (1, 129, 3, 3, 64, 64, True, False, 0.0, 1.0, False, "any", False),
    "norm only": (2, 40, 4, 2, 128, 0, False, True, 1e-6, 1.0, True, None, False),
    "many tokens": (1, 6000, 4, 2, 128, 128, False, True, 1e-6, 1.0, True, "any", False),
    "many tokens, d 64": (2, 5003, 3, 1, 64, 32, True, True, 1e-6, 1.0, True, None, False),
    "decode": (32, 1, 32, 8, 128, 128, False, True, 1e-6, 1.0, True, "any", False),
}


def _case(name):
    B, N, Hq, Hkv, d, rot, il, norm, eps, scale, weights, kind, fused = CASES[name]
    g = torch.Generator(device="cuda").manual_seed(len(name))
    x = torch.randn(B, N, Hq + 2 * Hkv, d, generator=g, device="cuda").to(bf16)
    Q, K = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
    if not fused:
        Q, K = Q.contiguous(), K.contiguous()
    inv = pisa.rope_frequencies(rot)[0].cuda() if rot else None
    wq, wk = (torch.randn(d, generator=g, device="cuda") + 1 for _ in range(2)) if weights else (None, None)
    pos, P = None, torch.arange(N, device="cuda").expand(B, N)
    if kind == "far":
        pos = (torch.arange(B * N, device="cuda", dtype=torch.int32) * 7 + 3_000_000).reshape(B, N)
    elif kind == "any":
        pos = torch.randint(0, 2**31 - 1, (B, N), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
        pos[0, 0] = 2**31 - 1
    shape = pisa.rope_shape_of(Q, K, rot, il, norm, eps, scale)
    return Q, K, inv, shape, wq, wk, pos, P if pos is None else pos, (rot, il, norm, eps, scale), g


@pytest.mark.parametrize("name", CASES)
def test_against_definition(name):
    Q, K, inv, shape, wq, wk, pos, P, how, g = _case(name)
    dQr, dKr = (torch.randn(t.shape, generator=g, device="cuda").to(bf16) for t in (Q, K))
    Qr, Kr = pisa.qk_norm_rope(Q, K, inv, shape, wq, wk, pos)
    ws = pisa.qk_norm_rope_workspace(shape, Q.device).fill_(0xEE)
    dQ, dK, dwq, dwk = pisa.qk_norm_rope_bwd(Q, K, dQr, dKr, inv, shape, wq, wk, pos, ws=ws)
    assert pisa.workspace_status(ws) == 0
    for n, x, w, y, dy, dx, dw in (("Q", Q, wq, Qr, dQr, dQ, dwq), ("K", K, wk, Kr, dKr, dK, dwk)):
        ref = _reference(x, w, P, inv, *how, dy=dy)
        check(n + "r", y, *ref["y"])
        check("d" + n, dx, *ref["dx"])
        if how[2]:
            check("dw" + n, dw, *ref["dw"])
        else:
            assert dw is None


def test_gradients_against_differences():
    # sum(dy . y) differenced in 64 bits on the reference, and the kernel's gradient inside the bounds of it
    Q, K, inv, shape, wq, wk, pos, P, how, g = _case("part of the head")
    dy = torch.randn(Q.shape, generator=g, device="cuda").to(bf16)
    _, _, dwq, _ = out = pisa.qk_norm_rope_bwd(Q, K, dy, torch.zeros(K.shape, dtype=bf16, device="cuda"), inv, shape, wq, wk, pos)
    f = lambda x, w: (_reference(x, w, P, inv, *how)["y"][0] * dy.double()).sum().item()       # noqa: E731
    x = Q.double()
    for b, n, h, e in ((0, 0, 0, 0), (1, 7, 5, 30), (0, 32, 3, 100), (1, 20, 2, 47)):
        v = x[b, n, h, e].item()
        x[b, n, h, e] = v + 1e-4
        up = f(x, wq)
        x[b, n, h, e] = v - 1e-4
        down = f(x, wq)
        x[b, n, h, e] = v
        num, scale = (up - down) / 2e-4, float(out[0][b, n, h].abs().max())
        assert abs(num - float(out[0][b, n, h, e])) <= H * abs(num) + 2.0 ** -16 * scale + 1e-4
    w = wq.double()
    for e in (0, 23, 24, 90):
        v = w[e].item()
        w[e] = v + 1e-4
        up = f(x, w)
        w[e] = v - 1e-4
        down = f(x, w)
        w[e] = v
        assert abs((up - down) / 2e-4 - float(dwq[e])) <= 1e-4 * float(dwq.abs().max())


def test_elements_that_do_not_turn_keep_infinities_and_zeros():
    Q = torch.zeros(1, 2, 1, 64, dtype=bf16, device="cuda")
    Q[0, 1, 0, 40], Q[0, 1, 0, 41] = math.inf, -math.inf
    for il in (False, True):
        shape = pisa.rope_shape_of(Q, Q, 32, il, norm=False)
        Qr, _ = pisa.qk_norm_rope(Q, Q, pisa.rope_frequencies(32)[0].cuda(), shape)
        assert torch.equal(Qr, Q)
    shape = pisa.rope_shape_of(Q[:, :1].contiguous(), Q[:, :1].contiguous(), 32, eps=1e-6)
    Qr, _ = pisa.qk_norm_rope(Q[:, :1].contiguous(), Q[:, :1].contiguous(), pisa.rope_frequencies(32)[0].cuda(), shape)
    assert torch.equal(Qr, torch.zeros_like(Qr))           # a row of zeros has a finite norm


def test_in_place_and_same_bits():
    Q, K, inv, shape, wq, wk, pos, *_ = _case("many tokens")
    Qr, Kr = pisa.qk_norm_rope(Q, K, inv, shape, wq, wk, pos)
    g = [pisa.qk_norm_rope_bwd(Q, K, Qr, Kr, inv, shape, wq, wk, pos) for _ in range(2)]
    for a, b in zip(*g):
        assert torch.equal(a, b)
    q, k = Q.clone(), K.clone()
    pisa.qk_norm_rope(q, k, inv, shape, wq, wk, pos, q_out=q, k_out=k)
    assert torch.equal(q, Qr) and torch.equal(k, Kr)


def test_captured_and_replayed():
    Q, K, inv, shape, wq, wk, pos, *_ = _case("decode")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    ws = pisa.qk_norm_rope_workspace(shape, Q.device)
    with torch.cuda.graph(graph, stream=side):
        Qr, Kr = pisa.qk_norm_rope(Q, K, inv, shape, wq, wk, pos)
        grads = pisa.qk_norm_rope_bwd(Q, K, Qr, Kr, inv, shape, wq, wk, pos, ws=ws)
    Q.copy_(torch.randn_like(Q, dtype=torch.float32))
    pos.add_(-77)
    graph.replay()
    torch.cuda.synchronize()
    want = pisa.qk_norm_rope(Q, K, inv, shape, wq, wk, pos)
    for a, b in zip((Qr, Kr, *grads), (*want, *pisa.qk_norm_rope_bwd(Q, K, *want, inv, shape, wq, wk, pos))):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------------ together
def test_layer_forward_and_backward_together():
    """Fused projection -> norm + rotation -> window attention, and back to the projection's gradient."""
    B, N, Hq, Hkv, d, window, sinks = 2, 400, 8, 2, 64, 90, 3
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(B, N, Hq + 2 * Hkv, d, generator=g, device="cuda").to(bf16)
    Q, K, V = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    wq, wk = (1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    dO = torch.randn(B, N, Hq, d, generator=g, device="cuda").to(bf16)
    inv, scale = pisa.rope_frequencies(d, scaling="yarn", factor=4.0, trained_len=128)
    inv = inv.cuda()
    rs = pisa.rope_shape_of(Q, K, d, rot_scale=scale)
    Qr, Kr = pisa.qk_norm_rope(Q, K, inv, rs, wq, wk)
    s = pisa.window_shape_of(Qr, Kr, V, window, sinks)
    O, lse = pisa.window_attn_fwd(Qr, Kr, V, s)
    dQr, dKr, dV = pisa.window_attn_bwd(Qr, Kr, V, O, lse, dO, s)
    dQ, dK, dwq, dwk = pisa.qk_norm_rope_bwd(Q, K, dQr, dKr, inv, rs, wq, wk)
    # the chain in 64 bits by autograd
    xs = [t.double().detach().requires_grad_() for t in (Q, K, V, wq, wk)]
    a = torch.arange(N, device="cuda").double()[:, None, None] * inv.double()
    c, sn = a.cos() * scale, a.sin() * scale

    def ready(t, w):
        y = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        u, v = y[..., :d // 2], y[..., d // 2:]
        return torch.cat([u * c - v * sn, u * sn + v * c], -1)

    q, k = ready(xs[0], xs[3]), ready(xs[1], xs[4])
    k, v = (t.repeat_interleave(Hq // Hkv, 2) for t in (k, xs[2]))
    p = torch.arange(N, device="cuda")
    see = (p[None] <= p[:, None]) & ((p[:, None] - p[None] < window) | (p[None] < sinks))
    z = (torch.einsum("bihd,bjhd->bhij", q, k) / math.sqrt(d)).masked_fill(~see, -math.inf)
    o = torch.einsum("bhij,bjhd->bihd", z.softmax(-1), v)
    want = torch.autograd.grad(o, xs, dO.double())
    # each of the four steps rounds its bf16 outputs (2^-8 at most, about 2^-9.8 in the mean square); the norms
    # of the results are compared, where such errors of single elements add up in quadrature: 2^-7 holds them
    for n, got, ref in (("O", O, o), *zip(("dQ", "dK", "dV", "dwq", "dwk"), (dQ, dK, dV, dwq, dwk), want)):
        err = float((got.double() - ref.detach()).norm() / ref.detach().norm())
        assert err < 2.0 ** -7, (n, err)


def test_decode_steps_take_raw_projections():
    """Both decode steps with `rope`: the selected blocks' step and the window's, from raw projections."""
    B, Ncap, Hq, Hkv, d, L = 2, 512, 8, 2, 128, 200
    g = torch.Generator(device="cuda").manual_seed(6)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(bf16)       # noqa: E731
    Kc, Vc, q, k, v = rnd(B, Ncap, Hkv, d), rnd(B, Ncap, Hkv, d), rnd(B, Hq, d), rnd(B, Hkv, d), rnd(B, Hkv, d)
    rope = pisa.Rope(pisa.rope_frequencies(d)[0].cuda(), d, q_weight=1 + 0.1 * torch.randn(d, device="cuda"))
    pos = torch.tensor([L, L - 60], dtype=torch.int32, device="cuda")
    rs = pisa.make_rope_shape(B, 1, Hq, Hkv, d, d)
    qr, kr = pisa.qk_norm_rope(q[:, None], k[:, None], rope.inv_freq, rs, rope.q_weight, None, pos[:, None])
    qr, kr = qr[:, 0], kr[:, 0]
    shape = pisa.make_window_decode_shape(B, Ncap, Hq, Hkv, d, 64, 4)
    Ka, Va, Kb, Vb = Kc.clone(), Vc.clone(), Kc.clone(), Vc.clone()
    a = pisa.window_decode_step(shape, pos, Ka, Va, q, k, v, rope=rope)
    b = pisa.window_decode_step(shape, pos, Kb, Vb, qr, kr, v)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(Ka, Kb) and not torch.equal(a[0], torch.zeros_like(a[0]))
    dshape = pisa.make_decode_shape(B, Ncap, Hq, Hkv, d, 64, 4)
    Ka, Kb, Va, Vb = Kc.clone(), Kc.clone(), Vc.clone(), Vc.clone()
    pa, pb = (pisa.decode_build_pyramid(t, pos, dshape) for t in (Ka, Kb))
    a = pisa.decode_step(dshape, pos, Ka, Va, pa, q, k, v, rope=rope)
    b = pisa.decode_step(dshape, pos, Kb, Vb, pb, qr, kr, v)
    for x, y in ((a[0], b[0]), (a[1], b[1]), (Ka, Kb), (pa, pb)):
        assert torch.equal(x, y)
    assert int(a[3][0]) == 0


def test_selection_and_window_agree_where_everything_is_visible():
    """Normed and rotated heads through the pyramid selection with every block kept, and through a window
    that spans the sequence: the two attentions are the same full causal attention."""
    B, N, Hq, Hkv, d, K = 1, 500, 8, 2, 128, 8
    g = torch.Generator(device="cuda").manual_seed(7)
    Q, Kt, V = (torch.randn(B, N, h, d, generator=g, device="cuda").to(bf16) for h in (Hq, Hkv, Hkv))
    inv = pisa.rope_frequencies(d)[0].cuda()
    Qr, Kr = pisa.qk_norm_rope(Q, Kt, inv, pisa.rope_shape_of(Q, Kt, d))
    shape = pisa.make_shape(B, N, Hq, Hkv, d, 64, K)
    idx, _, hl = pisa.select(Qr, Kr, pisa.build_pyramid(Kr, shape), shape, want_head_lse=True)
    O, lse = pisa.sparse_attn_fwd(Qr, Kr, V, idx, shape, head_lse=hl)
    want, tol = attention(Qr, Kr, V, N, 0)
    Ow, lw = pisa.window_attn_fwd(Qr, Kr, V, pisa.window_shape_of(Qr, Kr, V, N))
    check("window O", Ow, want["O"], tol["O"])
    check("window lse", lw, want["lse"], tol["lse"])
    # the selected blocks' O with the tolerances of its own tests
    torch.testing.assert_close(O.double(), want["O"], atol=2e-2, rtol=2e-2)
    torch.testing.assert_close(lse.double(), want["lse"], atol=1e-3, rtol=0)
