"""Sliding-window attention with sinks on the GPU against its 64-bit definition: forward,
backward and decode steps, with bounds that count the kernels' roundings (_window_ref.py)."""
import math

import pytest
import torch

import pyramid_top_selection_gb300 as pisa
from _window_ref import E, H, attention, check

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


def _inputs(B, Nq, N, Hq, Hkv, d, fused=False, lens=None, seed=0, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if fused:
        x = (torch.randn(B, N, Hq + 2 * Hkv, d, generator=g, device="cuda") * spread).to(bf16)
        Q, K, V = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    else:
        Q = (torch.randn(B, Nq, Hq, d, generator=g, device="cuda") * spread).to(bf16)
        K = (torch.randn(B, N, Hkv, d, generator=g, device="cuda") * spread).to(bf16)
        V = torch.randn(B, N, Hkv, d, generator=g, device="cuda").to(bf16)
    dO = torch.randn(B, Nq, Hq, d, generator=g, device="cuda").to(bf16)
    if lens is not None:                   # what lies past a sequence's tokens is never used
        for b, L in enumerate(lens):
            K[b, L:], V[b, L:] = math.nan, math.inf
            r = max(0, L - (N - Nq))
            Q[b, r:], dO[b, r:] = math.nan, -math.inf
    return Q, K, V, dO


def _run(Q, K, V, dO, window, sinks, lens=None, scale=0.0):
    s = pisa.window_shape_of(Q, K, V, window, sinks, scale)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    B, Nq, Hq, d = Q.shape
    out = torch.full((B, Nq, Hq, d), 7.0, dtype=bf16, device="cuda")     # every element is written
    lse = torch.full((B, Hq, Nq), 7.0, device="cuda")
    ws = pisa.window_workspace(s, pisa.WINDOW_FWD, Q.device)
    O, lse = pisa.window_attn_fwd(Q, K, V, s, lens=ln, ws=ws, out=out, lse=lse)
    assert pisa.workspace_status(ws) == 0
    got = {"O": O, "lse": lse}
    if dO is not None:
        ws = pisa.window_workspace(s, pisa.WINDOW_BWD, Q.device)
        ws.fill_(0xAB)
        got["dQ"], got["dK"], got["dV"] = pisa.window_attn_bwd(Q, K, V, O, lse, dO, s, lens=ln, ws=ws)
        assert pisa.workspace_status(ws) == 0
    return got


CASES = {  # B, Nq, N, Hq, Hkv, d, window, sinks, lens, fused
    "one token": (1, 1, 1, 1, 1, 64, 1, 0, None, False),
    "one query of many": (2, 1, 500, 8, 2, 128, 100, 4, [500, 77], False),
    "own key only": (1, 300, 300, 4, 2, 128, 1, 0, None, False),
    "padded": (2, 130, 130, 4, 2, 128, 17, 3, [130, 65], False),
    "chunk, three heads, an empty sequence": (3, 100, 357, 6, 2, 64, 64, 5, [357, 300, 0], False),
    "full causal": (1, 257, 257, 8, 1, 128, 1000, 0, None, False),
    "full causal with sinks": (1, 400, 400, 4, 4, 64, 400, 9, None, False),
    "many sinks, one head": (1, 513, 513, 5, 5, 64, 128, 128, None, False),
    "sinks past the window": (1, 700, 700, 2, 1, 128, 32, 300, None, False),
    "group of 16": (1, 300, 1000, 16, 1, 128, 256, 33, None, False),
    "group of 64": (1, 70, 70, 64, 1, 64, 20, 2, None, False),
    "group of 12": (2, 150, 150, 24, 2, 64, 40, 1, [150, 149], False),
    "projection slices": (2, 640, 640, 8, 2, 128, 200, 1, None, True),
    "projection slices, padded": (2, 333, 333, 4, 4, 64, 100, 7, [12, 333], True),
    "window of one tile": (1, 1025, 1025, 4, 1, 128, 128, 4, None, False),
    "wide window": (1, 1500, 1500, 4, 2, 64, 1024, 4, None, False),
    "padded, many tiles": (3, 1300, 1300, 4, 2, 64, 900, 4, [1300, 777, 1157], False),
    "padded, many tiles, wide heads": (2, 1100, 1100, 4, 4, 128, 2000, 0, [1001, 1099], False),
    "padded chunk with far sinks": (2, 400, 1500, 16, 2, 128, 128, 70, [1500, 1205], False),
    "many heads, whole key tiles": (3, 900, 900, 8, 8, 64, 100, 3, None, False),
    "many heads, whole key tiles, padded": (2, 1300, 1300, 16, 8, 128, 90, 0, [1300, 1001], True),
    "long chunk": (1, 129, 2000, 8, 2, 128, 700, 16, None, False),
}


@pytest.mark.parametrize("name", CASES)
def test_against_definition(name):
    B, Nq, N, Hq, Hkv, d, window, sinks, lens, fused = CASES[name]
    Q, K, V, dO = _inputs(B, Nq, N, Hq, Hkv, d, fused, lens, seed=len(name))
    got = _run(Q, K, V, dO, window, sinks, lens)
    want, tol = attention(Q, K, V, window, sinks, lens, dO=dO)
    for n in want:
        check(n, got[n], want[n], tol[n])


@pytest.mark.parametrize("scale,spread", [(0.5, 1.0), (0.0, 6.0), (0.01, 1.0)])
def test_peaked_and_flat_softmax(scale, spread):
    # logits up to several hundred: the running maximum moves and the sums must follow it
    Q, K, V, dO = _inputs(1, 520, 520, 4, 2, 128, seed=3, spread=spread)
    K[:, 100::90] *= 4
    got = _run(Q, K, V, dO, 300, 2, scale=scale)
    want, tol = attention(Q, K, V, 300, 2, scale=scale, dO=dO)
    for n in want:
        check(n, got[n], want[n], tol[n])


def test_rising_logits():
    # every later key beats all earlier ones by a wide margin, tile after tile
    Q, K, V, dO = _inputs(1, 600, 600, 2, 1, 64, seed=9)
    Q[..., 0] = 16.0
    K[..., 0] = torch.arange(600, device="cuda").reshape(1, 600, 1) / 4
    got = _run(Q, K, V, dO, 600, 0)
    want, tol = attention(Q, K, V, 600, 0, dO=dO)
    for n in want:
        check(n, got[n], want[n], tol[n])


@pytest.mark.parametrize("Hq,Hkv,d,window,sinks", [(16, 2, 128, 1024, 4), (4, 1, 64, 4096, 0), (8, 8, 128, 300, 64)])
def test_long_sequences_on_sampled_rows(Hq, Hkv, d, window, sinks):
    # 64-bit rows on the GPU for a sample of queries and keys of an 8192-token sequence
    N = 8192
    Q, K, V, dO = _inputs(1, N, N, Hq, Hkv, d, seed=5)
    got = _run(Q, K, V, dO, window, sinks)
    for lo in (0, 4000, N - 96):
        hi = lo + 96
        want, tol = attention(Q[:, lo:hi], K[:, :hi], V[:, :hi], window, sinks, dO=dO[:, lo:hi])
        for n, sl in (("O", (0, slice(lo, hi))), ("dQ", (0, slice(lo, hi))), ("lse", (0, slice(None), slice(lo, hi)))):
            check(n, got[n][sl], want[n][0], tol[n][0])
    # dK, dV of a block in the middle and (sinks) of the first keys: all the rows that see them
    G = Hq // Hkv
    for j0 in (0, 5000):
        j1 = j0 + 32
        for kv in (0, Hkv - 1):
            end = N if j0 < sinks else min(N, j1 + window)
            p = torch.arange(j0, end, device="cuda")[:, None]
            j = torch.arange(j0, j1, device="cuda")[None]
            see = (j <= p) & ((p - j < window) | (j < sinks))
            k, v = K[0, j0:j1, kv].double(), V[0, j0:j1, kv].double()
            dk = dv = dkt = dvt = 0
            for h in range(kv * G, kv * G + G):
                q, g = Q[0, j0:end, h].double(), dO[0, j0:end, h].double()
                z, o = got["lse"][0, h, j0:end].double()[:, None], got["O"][0, j0:end, h].double()
                P = torch.where(see, (q @ k.T / math.sqrt(d) - z).exp(), 0.0)
                dS = P * (g @ v.T - (g * o).sum(1, keepdim=True)) / math.sqrt(d)
                dk, dv = dk + dS.T @ q, dv + P.T @ g
                # O and lse are the forward's own here: what is left is P's and dS's rounding and fp32 sums
                e = H + 2.0 ** -11
                dkt = dkt + (dS.abs() * e + P * (g.abs() @ v.abs().T) * d * E).T @ q.abs()
                dvt = dvt + (P * e).T @ g.abs()
            check("dK", got["dK"][0, j0:j1, kv], dk, dkt + H * dk.abs())
            check("dV", got["dV"][0, j0:j1, kv], dv, dvt + H * dv.abs())


@pytest.mark.parametrize("B,Nq,N,Hq,Hkv,d,window,sinks,lens", [
    (1, 1, 9000, 16, 2, 128, 9000, 0, None),               # two items: sixteen CTAs each
    (1, 3, 5001, 5, 1, 64, 4000, 40, None),
    (3, 40, 4100, 4, 1, 128, 2500, 4, [4100, 0, 4071]),    # rows, and a whole sequence, that see nothing
    (2, 300, 2200, 8, 2, 64, 1500, 300, [2200, 2050]),     # sinks of several key tiles
    (1, 65, 700, 4, 2, 128, 640, 0, [650]),
    (1, 513, 1800, 8, 4, 64, 900, 1, None),
    (2, 1, 1300, 4, 4, 128, 1024, 200, [1300, 1299]),      # the only query of the second sequence is padding
    # padded batches: items with nothing to see among the split ones
    (3, 777, 5003, 12, 4, 128, 1500, 5, [5003, 3752, 0]),
    (4, 130, 3000, 8, 2, 64, 1200, 3, [3000, 2990, 2871, 100]),
    (5, 64, 2600, 4, 1, 128, 2600, 0, [2600, 2599, 2537, 2536, 0]),
    (2, 500, 2200, 8, 2, 128, 2000, 0, [2200, 2200]),
    (3, 300, 1500, 8, 4, 64, 1000, 40, [0, 0, 1201]),
    (2, 600, 2000, 12, 4, 128, 900, 1, [0, 1399]),         # no row at all
])
def test_few_rows_against_many_keys(B, Nq, N, Hq, Hkv, d, window, sinks, lens):
    # an item's keys are cut among a cluster's CTAs, whose sums are joined
    Q, K, V, _ = _inputs(B, Nq, N, Hq, Hkv, d, lens=lens, seed=N)
    K[:, N // 2] *= 3                                      # the runs' maxima differ
    got = _run(Q, K, V, None, window, sinks, lens)
    again = _run(Q, K, V, None, window, sinks, lens)
    want, tol = attention(Q, K, V, window, sinks, lens)
    for n in got:
        check(n, got[n], want[n], tol[n])
        assert torch.equal(got[n], again[n])


def test_split_item_keeps_nan_and_reports_waits(request):
    Q, K, V, _ = _inputs(1, 70, 4000, 2, 1, 128, seed=2)
    Q[0, 33, 1] = math.nan                                 # one row's own NaN, in every CTA's part
    got = _run(Q, K, V, None, 3500, 0)
    bad = got["O"].isnan().any(-1)[0]
    assert bool(bad[33, 1]) and int(bad.sum()) == 1 and bool(got["lse"][0, 1, 33].isnan())
    request.getfixturevalue("stalled")
    s = pisa.window_shape_of(Q, K, V, 3500, 0)
    ws = pisa.window_workspace(s, pisa.WINDOW_FWD, Q.device)
    O, lse = pisa.window_attn_fwd(Q, K, V, s, ws=ws)
    assert pisa.workspace_status(ws) & pisa.STATUS_TIMEOUT
    assert bool(O.isnan().all()) and bool(lse.isnan().all())


def test_split_items_of_a_padded_batch_report_waits(stalled):
    Q, K, V, _ = _inputs(3, 200, 3000, 8, 2, 64, lens=[3000, 2900, 50], seed=4)
    s = pisa.window_shape_of(Q, K, V, 2000, 4)
    ws = pisa.window_workspace(s, pisa.WINDOW_FWD, Q.device)
    ln = torch.tensor([3000, 2900, 50], dtype=torch.int32, device="cuda")
    O, lse = pisa.window_attn_fwd(Q, K, V, s, lens=ln, ws=ws)
    assert pisa.workspace_status(ws) & pisa.STATUS_TIMEOUT
    assert bool(O[0].isnan().all()) and bool(O[1, :100].isnan().all()) and bool(lse[0].isnan().all())
    assert float(O[2].abs().max()) == 0.0 and bool((lse[2] == -math.inf).all())


def test_split_item_captured():
    Q, K, V, _ = _inputs(1, 16, 6000, 8, 1, 64, seed=8)
    s = pisa.window_shape_of(Q, K, V, 6000, 0)
    want = [x.clone() for x in pisa.window_attn_fwd(Q, K, V, s)]
    O, lse = torch.empty_like(Q), torch.empty(1, 8, 16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pisa.window_attn_fwd(Q, K, V, s, out=O, lse=lse)
    for _ in range(3):
        O.zero_()
        g.replay()
        assert torch.equal(O, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("B,N,Hq,Hkv,d,window,sinks,lens", [
    (1, 400, 8, 2, 64, 2, 1, None), (2, 600, 4, 2, 128, 4, 0, [600, 391]), (1, 2000, 3, 1, 128, 17, 4, None),
    (1, 97, 5, 1, 128, 97, 0, None), (2, 300, 2, 2, 64, 60, 33, None),
])
def test_gradients_of_rows_with_few_keys_keep_their_precision(B, N, Hq, Hkv, d, window, sinks, lens):
    # dQ and dK carry two roundings to bf16 of the same size, dS's and their own: sqrt 2 of one's error (rms),
    # and 6 % for the sample. O's rounding, which D = dO . O would feel most here, is not to add to it.
    Q, K, V, dO = _inputs(B, N, N, Hq, Hkv, d, lens=lens, seed=N)
    got = _run(Q, K, V, dO, window, sinks, lens)
    want, _ = attention(Q, K, V, window, sinks, lens, dO=dO)
    for n in ("dQ", "dK", "dV"):
        w = want[n].double()
        one = (w.to(bf16).double() - w).norm()
        assert float((got[n].double() - w).norm() / one) < 1.5, n


def test_same_call_gives_same_bits():
    Q, K, V, dO = _inputs(2, 900, 900, 8, 2, 128, seed=1)
    a, b = _run(Q, K, V, dO, 250, 40), _run(Q, K, V, dO, 250, 40)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_captured_and_replayed_with_new_inputs():
    Q, K, V, dO = _inputs(1, 700, 700, 8, 2, 128, seed=2)
    s = pisa.window_shape_of(Q, K, V, 150, 5)
    lens = torch.tensor([700], dtype=torch.int32, device="cuda")
    wf, wb = (pisa.window_workspace(s, op, Q.device) for op in (pisa.WINDOW_FWD, pisa.WINDOW_BWD))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        O, lse = pisa.window_attn_fwd(Q, K, V, s, lens=lens, ws=wf)
        grads = pisa.window_attn_bwd(Q, K, V, O, lse, dO, s, lens=lens, ws=wb)
    for seed, L in ((11, 700), (12, 333)):
        Q2, K2, V2, dO2 = _inputs(1, 700, 700, 8, 2, 128, seed=seed)
        for t, u in ((Q, Q2), (K, K2), (V, V2), (dO, dO2)):
            t.copy_(u)
        lens.fill_(L)
        graph.replay()
        torch.cuda.synchronize()
        want = _run(Q2, K2, V2, dO2, 150, 5, [L])
        for n, t in zip(("O", "lse", "dQ", "dK", "dV"), (O, lse, *grads)):
            assert torch.equal(t, want[n]), (n, seed)


def test_two_streams_at_once():
    ins = [_inputs(1, 1200, 1200, 8, 2, 128, seed=20 + k) for k in range(2)]
    want = [_run(*x, 300, 4) for x in ins]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in ins], []
    for st, x in zip(streams, ins):
        with torch.cuda.stream(st):
            Q, K, V, dO = x
            s = pisa.window_shape_of(Q, K, V, 300, 4)
            O, lse = pisa.window_attn_fwd(Q, K, V, s)
            got.append((O, lse, *pisa.window_attn_bwd(Q, K, V, O, lse, dO, s)))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for n, t in zip(("O", "lse", "dQ", "dK", "dV"), g):
            assert torch.equal(t, w[n]), n


@pytest.fixture
def stalled():
    pisa.set_wait_limit(2_000_000)          # 2 ms
    pisa.set_test_stall(True)
    try:
        yield
    finally:
        pisa.set_test_stall(False)
        pisa.set_wait_limit(0)


@pytest.mark.parametrize("N,Hq,Hkv,d,window,sinks", [(700, 8, 2, 128, 150, 5), (20000, 4, 1, 64, 300, 0), (3000, 2, 2, 128, 3000, 0)])
def test_wait_that_runs_out_is_reported_and_poisons_outputs(stalled, N, Hq, Hkv, d, window, sinks):
    Q, K, V, dO = _inputs(1, N, N, Hq, Hkv, d, seed=6)
    s = pisa.window_shape_of(Q, K, V, window, sinks)
    wf, wb = (pisa.window_workspace(s, op, Q.device) for op in (pisa.WINDOW_FWD, pisa.WINDOW_BWD))
    O, lse = pisa.window_attn_fwd(Q, K, V, s, ws=wf)
    assert pisa.workspace_status(wf) & pisa.STATUS_TIMEOUT
    assert bool(O.isnan().all()) and bool(lse.isnan().all())
    with pytest.raises(pisa.PisaError):
        pisa.check_status(wf)
    assert bool(pisa.window_attn_fwd(Q, K, V, s)[0].isnan().all())       # without a workspace the outputs tell
    z = torch.zeros_like(O)
    grads = pisa.window_attn_bwd(Q, K, V, z, torch.zeros_like(lse), dO, s, ws=wb)
    assert pisa.workspace_status(wb) & pisa.STATUS_TIMEOUT
    for t in grads:
        assert bool(t.isnan().all())
    pisa.set_test_stall(False)                                           # and the next calls are sound again
    pisa.set_wait_limit(0)
    got = _run(Q, K, V, dO, window, sinks)
    for t in got.values():
        assert bool(t.isfinite().all())


# --------------------------------------------------------------------------------------- decode
def _slot(j, sinks, cap):
    return j if j < sinks else sinks + (j - sinks) % (cap - sinks)


@pytest.mark.parametrize("B,Ncap,Hq,Hkv,d,window,sinks,pos", [
    (1, 1, 1, 1, 64, 1, 0, [0]),
    (3, 64, 8, 2, 128, 16, 4, [0, 5, 63]),                 # below the capacity
    (4, 36, 6, 2, 64, 32, 4, [35, 36, 37, 10**6 + 3]),     # exactly sinks + window, rolled over
    (2, 1000, 16, 1, 128, 700, 33, [999, 40000]),
    (2, 5000, 8, 8, 128, 4096, 4, [4999, 2**31 - 1]),
    (2, 300, 64, 1, 128, 299, 1, [150, 299]),              # a group of 64
    (5, 700, 5, 1, 64, 600, 0, [0, 1, 63, 64, 699]),
    (2, 200, 4, 2, 64, 500, 3, [199, 100]),                # a window wider than the cache: positions below Ncap
    (33, 257, 4, 4, 128, 130, 100, list(range(90, 90 + 33 * 17, 17))),
    (1, 129, 3, 1, 128, 1, 0, [128]),
])
def test_decode_against_definition(B, Ncap, Hq, Hkv, d, window, sinks, pos):
    g = torch.Generator(device="cuda").manual_seed(Ncap)
    Kc, Vc = (torch.randn(B, Ncap, Hkv, d, generator=g, device="cuda").to(bf16) for _ in range(2))
    q = torch.randn(B, Hq, d, generator=g, device="cuda").to(bf16)
    kn, vn = (torch.randn(B, Hkv, d, generator=g, device="cuda").to(bf16) for _ in range(2))
    seen = []
    for b, p in enumerate(pos):            # slots that p does not see hold garbage
        j = list(range(min(sinks, max(0, p - window + 1)))) + list(range(max(0, p - window + 1), p + 1))
        seen.append([_slot(x, sinks, Ncap) for x in j])
        hide = torch.ones(Ncap, dtype=torch.bool, device="cuda")
        hide[seen[-1]] = False
        Kc[b, hide], Vc[b, hide] = math.nan, math.inf
    Kw, Vw = Kc.clone(), Vc.clone()
    for b, p in enumerate(pos):
        Kw[b, _slot(p, sinks, Ncap)], Vw[b, _slot(p, sinks, Ncap)] = kn[b], vn[b]
    shape = pisa.make_window_decode_shape(B, Ncap, Hq, Hkv, d, window, sinks)
    o, lse, status = pisa.window_decode_step(shape, torch.tensor(pos, dtype=torch.int32, device="cuda"), Kc, Vc, q, kn, vn)
    assert int(status[0]) == 0
    assert torch.equal(Kc.view(torch.int16), Kw.view(torch.int16)) and torch.equal(Vc.view(torch.int16), Vw.view(torch.int16))
    for b in range(B):
        n = len(seen[b])
        want, tol = attention(q[b:b + 1, None], Kw[b:b + 1, seen[b]], Vw[b:b + 1, seen[b]], n, 0)
        check(f"o {b}", o[b], want["O"][0, 0], tol["O"][0, 0])
        check(f"lse {b}", lse[b], want["lse"][0, :, 0], tol["lse"][0, :, 0])


def test_decode_positions_out_of_range_are_reported_and_left_alone():
    B, Ncap, Hq, Hkv, d = 4, 64, 4, 2, 64
    Kc, Vc = (torch.randn(B, Ncap, Hkv, d, device="cuda").to(bf16) for _ in range(2))
    q, kn = torch.randn(B, Hq, d, device="cuda").to(bf16), torch.randn(B, Hkv, d, device="cuda").to(bf16)
    K0, V0 = Kc.clone(), Vc.clone()
    o = torch.full_like(q, 3.0)
    shape = pisa.make_window_decode_shape(B, Ncap, Hq, Hkv, d, 62, 4)        # 62 + 4 > 64: no rolling
    pos = torch.tensor([-1, 64, 10, 2**31 - 1], dtype=torch.int32, device="cuda")
    o, lse, status = pisa.window_decode_step(shape, pos, Kc, Vc, q, kn, kn, o=o)
    assert int(status[0]) == pisa.STATUS_POS_RANGE
    assert torch.equal(o[[0, 1, 3]], torch.full_like(o[[0, 1, 3]], 3.0)) and not torch.equal(o[2], torch.full_like(o[2], 3.0))
    K0[2, 10], V0[2, 10] = kn[2], kn[2]
    assert torch.equal(Kc, K0) and torch.equal(Vc, V0)


def test_decode_steps_follow_the_prefill():
    # a prompt by the forward, then single tokens on a rolling cache that just holds sinks and window:
    # every step is the last row of a forward over the tokens so far
    B, N0, steps, Hq, Hkv, d, window, sinks = 2, 50, 120, 8, 2, 64, 48, 4
    T = N0 + steps
    Q, K, V, _ = _inputs(B, T, T, Hq, Hkv, d, seed=8)
    cap = sinks + window
    Kc, Vc = (torch.zeros(B, cap, Hkv, d, dtype=bf16, device="cuda") for _ in range(2))
    for j in range(N0):
        Kc[:, _slot(j, sinks, cap)], Vc[:, _slot(j, sinks, cap)] = K[:, j], V[:, j]
    shape = pisa.make_window_decode_shape(B, cap, Hq, Hkv, d, window, sinks)
    want, tol = attention(Q, K, V, window, sinks)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    for p in range(N0, T):
        pos = torch.full((B,), p, dtype=torch.int32, device="cuda")
        o, lse, _ = pisa.window_decode_step(shape, pos, Kc, Vc, Q[:, p].contiguous(), K[:, p].contiguous(),
                                            V[:, p].contiguous(), status=status)
        check(f"o at {p}", o, want["O"][:, p], tol["O"][:, p])
        check(f"lse at {p}", lse, want["lse"][:, :, p], tol["lse"][:, :, p])
    assert int(status[0]) == 0
