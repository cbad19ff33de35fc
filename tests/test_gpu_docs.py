"""Attention over packed documents on the GPU against its 64-bit definition: forward and backward, causal and prefix
masks, capped and distance-biased scores, with bounds that count the kernels' roundings (_docs_ref.py)."""
import math
import random

import pytest
import torch

import pyramid_top_selection_gb300 as pisa
from _docs_ref import doc_attention, doc_mask
from _window_ref import check

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _inputs(T, Hq, Hkv, d, fused=False, seed=0, spread=1.0, padding=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if fused:
        x = (torch.randn(T, Hq + 2 * Hkv, d, generator=g, device="cuda") * spread).to(bf16)
        Q, K, V = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        Q = (torch.randn(T, Hq, d, generator=g, device="cuda") * spread).to(bf16)
        K = (torch.randn(T, Hkv, d, generator=g, device="cuda") * spread).to(bf16)
        V = torch.randn(T, Hkv, d, generator=g, device="cuda").to(bf16)
    dO = torch.randn(T, Hq, d, generator=g, device="cuda").to(bf16)
    if padding is not None:                # what belongs to no document is never used
        Q[padding], K[padding], V[padding], dO[padding] = math.nan, math.nan, math.inf, -math.inf
    return Q, K, V, dO


def _run(Q, K, V, dO, starts, prefix=None, slopes=None, cap=0.0, scale=0.0, max_len=0):
    T, Hq, d = Q.shape
    s = pisa.doc_shape_of(Q, K, V, starts, max_len, scale, cap)
    out = torch.full((T, Hq, d), 7.0, dtype=bf16, device="cuda")       # every element is written
    lse = torch.full((Hq, T), 7.0, device="cuda")
    ws = pisa.doc_workspace(s, pisa.DOC_FWD, Q.device)
    ws.fill_(0xAB)
    O, lse = pisa.doc_attn_fwd(Q, K, V, starts, s, prefix, slopes, ws=ws, out=out, lse=lse)
    assert pisa.workspace_status(ws) == 0
    got = {"O": O, "lse": lse}
    if dO is not None:
        ws = pisa.doc_workspace(s, pisa.DOC_BWD, Q.device)
        ws.fill_(0xAB)
        got["dQ"], got["dK"], got["dV"] = pisa.doc_attn_bwd(Q, K, V, O, lse, dO, starts, s, prefix, slopes, ws=ws)
        assert pisa.workspace_status(ws) == 0
    return got


def _slopes(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")


CASES = {  # T, Hq, Hkv, d, starts, prefix, cap, slopes, fused
    "one token": (1, 1, 1, 64, [0, 1], None, 0.0, False, False),
    "one document": (257, 8, 1, 128, [0, 257], None, 0.0, False, False),
    "one key each": (40, 4, 2, 128, list(range(41)), None, 0.0, False, False),
    "no document at all": (70, 4, 2, 64, [0, 0, 0], None, 0.0, False, False),
    "documents and padding": (700, 4, 2, 128, [0, 130, 131, 131, 400, 650], None, 0.0, False, False),
    "tokens before the first document": (300, 6, 2, 64, [37, 200, 290], None, 0.0, False, True),
    "starts past the tokens": (200, 2, 2, 64, [0, 150, 400, 500], None, 0.0, False, False),
    "prefixes": (600, 8, 2, 128, [0, 300, 310, 555, 600], [100, 10, 0, 1], 0.0, False, False),
    "prefixes of whole documents": (500, 4, 4, 64, [0, 260, 500], [260, 900], 0.0, False, True),
    "prefix longer than a tile": (900, 4, 1, 128, [5, 900], [500], 0.0, False, False),
    "capped": (513, 8, 2, 128, [0, 513], None, 3.0, False, False),
    "capped, several": (777, 5, 5, 64, [0, 400, 500, 777], None, 20.0, False, True),
    "distance": (600, 8, 2, 128, [0, 411, 600], None, 0.0, True, False),
    "distance, three heads, prefixes": (650, 6, 2, 64, [0, 300, 610], [77, 300], 0.0, True, False),
    "capped and distance": (500, 4, 1, 128, [0, 490], None, 5.0, True, False),
    "all of it": (900, 12, 4, 64, [3, 100, 101, 600, 850], [50, 1, 200, 30], 10.0, True, True),
    "group of 64": (90, 64, 1, 64, [0, 50, 90], [7, 0], 15.0, True, False),
    "group of 16": (300, 16, 1, 128, [0, 299], None, 0.0, True, False),
    "many documents": (1500, 4, 2, 128, list(range(0, 1501, 23)), None, 0.0, False, False),
    "many short documents, capped": (1000, 16, 2, 64, list(range(0, 1000, 7)), None, 4.0, False, False),
    "long documents": (2300, 4, 4, 128, [0, 1100, 2300], None, 0.0, False, False),
    "long documents, capped": (2300, 4, 2, 64, [0, 1300, 2299], None, 8.0, False, False),
}


@pytest.mark.parametrize("name", CASES)
def test_against_definition(name):
    T, Hq, Hkv, d, starts, prefix, cap, biased, fused = CASES[name]
    pad = torch.ones(T, dtype=torch.bool, device="cuda")
    pad[starts[0]:starts[-1]] = False
    Q, K, V, dO = _inputs(T, Hq, Hkv, d, fused, len(name), padding=pad)
    slopes = _slopes(Hq) if biased else None
    got = _run(Q, K, V, dO, _ints(starts), None if prefix is None else _ints(prefix), slopes, cap)
    want, tol = doc_attention(Q, K, V, starts, prefix, slopes, cap, dO=dO)
    for n in want:
        check(n, got[n], want[n], tol[n])


@pytest.mark.parametrize("cap", [0.0, 1.0, 30.0])
@pytest.mark.parametrize("biased", [False, True])
def test_peaked_scores(cap, biased):
    # products up to several hundred: the cap's tanh from its linear part to 1, the running maximum moves
    Q, K, V, dO = _inputs(520, 4, 2, 128, seed=3, spread=6.0)
    K[100::90] *= 4
    Q[200:210] = 0
    starts, slopes = [0, 40, 500], _slopes(4) * 3 if biased else None
    Q[500:], K[500:], V[500:] = 0, 0, 0
    got = _run(Q, K, V, dO, _ints(starts), None, slopes, cap)
    want, tol = doc_attention(Q, K, V, starts, None, slopes, cap, dO=dO)
    for n in want:
        check(n, got[n], want[n], tol[n])


@pytest.mark.parametrize("biased", [False, True])
def test_the_smallest_cap(biased):
    # scale / cap at its limit: scores of 0 stay 0, all others are +-cap
    Q, K, V, dO = _inputs(300, 4, 2, 64, seed=15)
    Q[::3], K[::5] = 0, 0
    starts, slopes, cap = [0, 170, 300], _slopes(4) if biased else None, 2.0 ** -10
    got = _run(Q, K, V, dO, _ints(starts), None, slopes, cap, 1.0)
    want, tol = doc_attention(Q, K, V, starts, None, slopes, cap, 1.0, dO=dO)
    for n in want:
        check(n, got[n], want[n], tol[n])


def test_scores_that_grow_with_distance():
    # negative slopes: the farthest key wins, row by row
    Q, K, V, dO = _inputs(400, 2, 1, 64, seed=4)
    slopes = torch.tensor([-0.25, -1.0], device="cuda")
    got = _run(Q, K, V, dO, _ints([0, 180, 400]), None, slopes)
    want, tol = doc_attention(Q, K, V, [0, 180, 400], None, slopes, dO=dO)
    for n in want:
        check(n, got[n], want[n], tol[n])


def test_one_document_is_the_window_attention_of_all_keys():
    Q, K, V, dO = _inputs(1000, 8, 2, 128, seed=5)
    got = _run(Q, K, V, dO, _ints([0, 1000]))
    s = pisa.window_shape_of(Q[None], K[None], V[None], 1000)
    O, lse = pisa.window_attn_fwd(Q[None], K[None], V[None], s)
    want, tol = doc_attention(Q, K, V, [0, 1000])
    check("O", O[0], want["O"], tol["O"])
    check("O", got["O"], want["O"], tol["O"])
    check("lse", got["lse"], lse[0].double(), 2 * tol["lse"])


@pytest.mark.parametrize("max_len", [1, 100, 450, 1000])
def test_what_the_caller_says_of_the_longest_document_does_not_matter(max_len):
    Q, K, V, dO = _inputs(1000, 4, 1, 128, seed=6)
    starts = [0, 450, 900]
    got = _run(Q, K, V, dO, _ints(starts), max_len=max_len)
    Q[900:], K[900:], V[900:], dO[900:] = 0, 0, 0, 0
    want, tol = doc_attention(Q, K, V, starts, dO=dO)
    for n in want:
        check(n, got[n], want[n], tol[n])


@pytest.mark.parametrize("cap,biased,prefix", [(0.0, False, None), (6.0, False, None), (6.0, True, [90, 20])])
def test_gradients_against_differences(cap, biased, prefix):
    # the kernel's gradients along random directions against differences of the 64-bit loss sum(O dO)
    Q, K, V, dO = _inputs(220, 4, 2, 64, seed=7, spread=1.5)
    starts, slopes = [0, 120, 220], _slopes(4) if biased else None
    got = _run(Q, K, V, dO, _ints(starts), None if prefix is None else _ints(prefix), slopes, cap)
    _, tol = doc_attention(Q, K, V, starts, prefix, slopes, cap, dO=dO)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = {"dQ": Q.double(), "dK": K.double(), "dV": V.double()}

    def loss(y):
        out, _ = doc_attention(y["dQ"], y["dK"], y["dV"], starts, prefix, slopes, cap)
        return float((out["O"] * dO.double()).sum())

    for n in x:
        u = torch.randn(x[n].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4                           # the differences' own error: h^2 times third derivatives, and 2^-53 / h of the loss
        diff = (loss(x | {n: x[n] + h * u}) - loss(x | {n: x[n] - h * u})) / (2 * h)
        got_n = float((got[n].double() * u).sum())
        bound = float((tol[n] * u.abs()).sum())
        assert abs(got_n - diff) <= bound + 1e-3 * abs(diff), (n, got_n, diff, bound)


def test_the_same_call_gives_the_same_bits():
    Q, K, V, dO = _inputs(3000, 8, 2, 128, seed=8)
    starts, slopes = _ints([0, 10, 900, 2500, 2990]), _slopes(8)
    one, two = (_run(Q, K, V, dO, starts, None, slopes, 10.0) for _ in range(2))
    for n in one:
        assert torch.equal(one[n][torch.isfinite(one[n])], two[n][torch.isfinite(two[n])]), n


def test_captured_and_replayed_on_other_documents():
    # starts are read by the kernels: one graph serves every packing of the same size
    T, Hq, Hkv, d = 1200, 8, 2, 128
    Q, K, V, dO = _inputs(T, Hq, Hkv, d, seed=9)
    starts, pre, slopes = _ints([0, 600, 1200, 1200]), _ints([0, 50, 0]), _slopes(Hq)
    s = pisa.doc_shape_of(Q, K, V, starts, cap=12.0)
    ws, wb = (pisa.doc_workspace(s, op, Q.device) for op in (pisa.DOC_FWD, pisa.DOC_BWD))

    def step():
        O, lse = pisa.doc_attn_fwd(Q, K, V, starts, s, pre, slopes, ws=ws)
        return O, lse, *pisa.doc_attn_bwd(Q, K, V, O, lse, dO, starts, s, pre, slopes, ws=wb)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for new_starts, new_pre in (([0, 600, 1200, 1200], [0, 50, 0]), ([0, 1, 777, 1190], [1, 300, 0])):
        starts.copy_(_ints(new_starts))
        pre.copy_(_ints(new_pre))
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)
        assert pisa.workspace_status(ws) == 0 and pisa.workspace_status(wb) == 0


def test_two_streams_at_once():
    Q, K, V, dO = _inputs(2000, 4, 2, 64, seed=10)
    starts = _ints([0, 1500, 2000])
    want = _run(Q, K, V, dO, starts)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    s = pisa.doc_shape_of(Q, K, V, starts)
    got = []
    for st in streams:
        with torch.cuda.stream(st):
            O, lse = pisa.doc_attn_fwd(Q, K, V, starts, s)
            got.append((O, lse, *pisa.doc_attn_bwd(Q, K, V, O, lse, dO, starts, s)))
    torch.cuda.synchronize()
    for g in got:
        for a, n in zip(g, ("O", "lse", "dQ", "dK", "dV")):
            assert torch.equal(a, want[n]), n


@pytest.mark.parametrize("cap,biased", [(0.0, False), (9.0, True)])
def test_small_calls_need_no_workspace(cap, biased):
    # where nothing is laid out ahead the workspace is the status block alone, and may be left out
    Q, K, V, _ = _inputs(300, 8, 2, 64, fused=True, seed=11)
    starts, slopes = _ints([0, 120, 300]), _slopes(8) if biased else None
    s = pisa.doc_shape_of(Q, K, V, starts, cap=cap)
    assert pisa.doc_workspace_size(s, pisa.DOC_FWD) == 256
    want = _run(Q, K, V, None, starts, None, slopes, cap)
    O, lse = pisa.doc_attn_fwd(Q, K, V, starts, s, slopes=slopes)
    assert torch.equal(O, want["O"]) and torch.equal(lse, want["lse"])


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (40, 8)])
def test_more_documents_than_the_rows_kernel_holds(Hq, Hkv):
    # 6000 documents of 0, 1 or 2 tokens: searched for in the starts themselves; with one head by the attention's kernel, with 40
    # by the one before it. A token sees itself and, as its document's second, the first.
    lens = [(0, 1, 2, 1)[m % 4] for m in range(6000)]
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    T = starts[-1]
    Q, K, V, dO = _inputs(T, Hq, Hkv, 64, seed=12)
    got = _run(Q, K, V, dO, _ints(starts))
    first = torch.tensor([starts[m] for m in range(6000) for _ in range(lens[m])], device="cuda")
    second = torch.arange(T, device="cuda") > first
    G = Hq // Hkv
    q, k, v, g = Q.double(), K.double().repeat_interleave(G, 1), V.double().repeat_interleave(G, 1), dO.double()
    x0, x1 = ((q * kk).sum(-1) / 8 for kk in (k[first], k))
    p0 = torch.where(second[:, None], torch.sigmoid(x0 - x1), 0.0)[..., None]
    want = p0 * v[first] + (1 - p0) * v
    # P's error: the scores' (64 products, |q||k| up to 64 2^-24 of their sum) and the exponent's; its rounding; O's
    size = p0 * v[first].abs() + (1 - p0) * v.abs()
    xe = (q.abs() * torch.maximum(k.abs(), k[first].abs())).sum(-1)[..., None] / 8 * 72 * 2.0 ** -24 + 2.0 ** -19
    tol = 2.0 ** -8 * (want.abs() + size) + (2 * xe + 2.0 ** -11) * size
    check("O", got["O"], want, tol)
    # gradients: dS of the first key is -dS of the token itself
    dp0, dp1 = ((g * vv).sum(-1, keepdim=True) for vv in (v[first], v))
    ds = p0 * (1 - p0) * (dp0 - dp1)
    dq = ds * (k[first] - k) / 8
    # |ds| off by its rounding, P's error, and D's (O's error times dO) for either key
    De = (g.abs() * tol).sum(-1, keepdim=True) + (g.abs() * size).sum(-1, keepdim=True) * 64 * 2.0 ** -24
    dse = ds.abs() * (2.0 ** -8 + 4 * xe + 2.0 ** -11) + torch.maximum(p0, 1 - p0) * De * 1.01
    check("dQ", got["dQ"], dq, dse * (k[first].abs() + k.abs()) / 8 + 2.0 ** -8 * dq.abs())


@pytest.fixture
def stalled():
    pisa.set_wait_limit(2_000_000)          # 2 ms
    pisa.set_test_stall(True)
    try:
        yield
    finally:
        pisa.set_test_stall(False)
        pisa.set_wait_limit(0)


@pytest.mark.parametrize("T,Hq,Hkv,d,cap,biased", [(300, 4, 1, 64, 0.0, False), (700, 8, 2, 128, 10.0, False), (12000, 16, 2, 128, 0.0, True)])
def test_wait_that_runs_out_is_reported_and_poisons_outputs(stalled, T, Hq, Hkv, d, cap, biased):
    Q, K, V, dO = _inputs(T, Hq, Hkv, d, seed=13)
    starts, slopes = _ints([0, T // 3, T]), _slopes(Hq) if biased else None
    s = pisa.doc_shape_of(Q, K, V, starts, cap=cap)
    wf, wb = (pisa.doc_workspace(s, op, Q.device) for op in (pisa.DOC_FWD, pisa.DOC_BWD))
    O, lse = pisa.doc_attn_fwd(Q, K, V, starts, s, slopes=slopes, ws=wf)
    assert pisa.workspace_status(wf) & pisa.STATUS_TIMEOUT
    with pytest.raises(pisa.PisaError):
        pisa.check_status(wf)
    assert bool(O.isnan().all()) and bool(lse.isnan().all())
    assert bool(pisa.doc_attn_fwd(Q, K, V, starts, s, slopes=slopes)[0].isnan().all())    # without a workspace the outputs tell
    grads = pisa.doc_attn_bwd(Q, K, V, torch.zeros_like(O), torch.zeros_like(lse), dO, starts, s, slopes=slopes, ws=wb)
    assert pisa.workspace_status(wb) & pisa.STATUS_TIMEOUT
    for t in grads:
        assert bool(t.isnan().all())
    pisa.set_test_stall(False)                                           # and the next calls are sound again
    pisa.set_wait_limit(0)
    for t in _run(Q, K, V, dO, starts, None, slopes, cap).values():
        assert bool(t.isfinite().all())


def test_two_graphs_share_workspaces():
    # forwards and backwards of two packings, captured with the same workspaces, replayed in turn
    Q, K, V, dO = _inputs(2500, 16, 4, 64, seed=14)
    s = pisa.make_doc_shape(2500, 16, 4, 64, 2)
    ws, wb = (pisa.doc_workspace(s, op, Q.device) for op in (pisa.DOC_FWD, pisa.DOC_BWD))
    packs = [_ints([0, 2000, 2500]), _ints([0, 300, 2400])]

    def step(starts):
        O, lse = pisa.doc_attn_fwd(Q, K, V, starts, s, ws=ws)
        return O, lse, *pisa.doc_attn_bwd(Q, K, V, O, lse, dO, starts, s, ws=wb)

    want = [[t.clone() for t in step(p)] for p in packs]
    graphs, got = [torch.cuda.CUDAGraph() for _ in packs], []
    for g, p in zip(graphs, packs):
        with torch.cuda.graph(g):
            got.append(step(p))
    for k in (0, 1, 1, 0, 1):
        for t in got[k]:
            t.zero_()
        graphs[k].replay()
        torch.cuda.synchronize()
        for a, b in zip(got[k], want[k]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("fused", [False, True])
def test_tokens_past_32_bits(fused):
    # elements beyond 2^31 (bytes beyond 2^32): the last documents of many, against their definition
    T, Hq, Hkv, d, n = (1 << 18) + 300, 64, 1, 128, 300
    few = _inputs(n, Hq, Hkv, d, seed=16)
    if fused:
        x = torch.zeros(T, Hq + 2 * Hkv, d, dtype=bf16, device="cuda")
        Q, K, V = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        Q, K, V = (torch.zeros(T, h, d, dtype=bf16, device="cuda") for h in (Hq, Hkv, Hkv))
    dO = torch.zeros(T, Hq, d, dtype=bf16, device="cuda")
    for t, x in zip((Q, K, V, dO), few):
        t[-n:] = x
    starts = list(range(0, T - n, 1 << 12)) + [T - n, T - 120, T]
    got = _run(Q, K, V, dO, _ints(starts), max_len=1 << 12)
    want, tol = doc_attention(*few[:3], [0, 180, 300], dO=few[3])
    for name in want:
        check(name, got[name][:, -n:] if name == "lse" else got[name][-n:], want[name], tol[name])
    assert not bool(got["O"][:-n].any()) and not bool(got["dQ"][:-n].any())


@pytest.mark.parametrize("T,seed", [(500, 0), (500, 1), (6000, 2), (6000, 3)])
def test_starts_in_no_order_are_survived(T, seed):
    # what comes out is not defined, but the calls end, without a wait that gives up
    g = torch.Generator(device="cuda").manual_seed(seed)
    Q, K, V, dO = _inputs(T, 16, 2, 64, seed=17)
    starts = torch.randint(-T, 2 * T, (41,), generator=g, device="cuda").to(torch.int32)
    prefix = torch.randint(-T, 2 * T, (40,), generator=g, device="cuda").to(torch.int32)
    _run(Q, K, V, dO, starts, prefix, max_len=T // 8)
    Q, K, V, dO = _inputs(T, 16, 2, 64, seed=18)
    for t in _run(Q, K, V, dO, _ints([0, T]), None).values():
        assert bool(t.isfinite().all())


@pytest.mark.parametrize("cap", [0.0, 7.0])
@pytest.mark.parametrize("seed", [11, 42, 44, 45])
def test_starts_in_no_order_are_survived_with_biased_scores(seed, cap):
    # starts with a row tile whose first key lies before its item's (tokens in 16s, two row tiles an item)
    T, r = 6000, random.Random(seed)
    starts = [r.randint(-T, 2 * T) for _ in range(41)]
    prefix = [r.randint(-T, 2 * T) for _ in range(40)]
    Q, K, V, dO = _inputs(T, 64, 8, 64, seed=19)
    _run(Q, K, V, dO, _ints(starts), _ints(prefix), _slopes(64), cap, max_len=T // 8)
    for t in _run(Q, K, V, dO, _ints([0, T]), None, _slopes(64), cap).values():
        assert bool(t.isfinite().all())


def _reached(see, G, bad):
    """Where the definition's results are not finite, from where Q, K (NaN), V, dO (NaN or infinite) are not: a sum over visible
    pairs is not finite where one of its terms is not."""
    T, Hq, d = bad["Q"].shape
    Hkv = Hq // G
    some = lambda m, x: (m.double() @ x.double()) > 0                       # noqa: E731 (any over the inner dimension)
    out = {n: torch.zeros(T, h, d, dtype=torch.bool, device=see.device) for n, h in (("O", Hq), ("dQ", Hq), ("dK", Hkv), ("dV", Hkv))}
    out["lse"] = torch.zeros(Hq, T, dtype=torch.bool, device=see.device)
    for h in range(Hq):
        q, k, v, g = bad["Q"][:, h], bad["K"][:, h // G], bad["V"][:, h // G], bad["dO"][:, h]
        row = (see & (q.any(1)[:, None] | k.any(1)[None])).any(1)
        o = row[:, None] | some(see, v)
        D = (g | o).any(1)
        dP = g.any(1)[:, None] | v.any(1)[None]
        dS = see & (row[:, None] | D[:, None] | dP)
        out["lse"][h], out["O"][:, h] = row, o
        out["dQ"][:, h] = dS.any(1)[:, None] | some(see, k)
        out["dK"][:, h // G] |= dS.any(0)[:, None] | some(see.T, q)
        out["dV"][:, h // G] |= (see & row[:, None]).any(0)[:, None] | some(see.T, g)
    return out


SPOILED = {  # T, Hq, Hkv, d, starts, prefix, cap, slopes, fused, max_len
    "three documents": (420, 4, 2, 64, [0, 150, 290, 420], None, 0.0, False, True, 0),
    "short documents": (300, 8, 2, 128, [3, 40, 77, 130, 131, 180, 290], None, 0.0, False, False, 0),
    "long documents, prefixes": (900, 4, 1, 128, [0, 500, 890], [30, 200], 0.0, False, False, 0),
    "capped": (600, 4, 2, 64, [0, 310, 600], None, 5.0, False, False, 0),
    "biased": (600, 6, 2, 128, [0, 310, 600], None, 0.0, True, True, 0),
    "capped and biased, in runs": (700, 2, 2, 64, [0, 600, 700], None, 5.0, True, False, 0),
    "many items": (1300, 40, 20, 64, [0, 100, 700, 1290], None, 0.0, False, False, 0),
    "many items, capped": (1300, 40, 20, 128, [0, 100, 700, 1290], None, 5.0, False, False, 300),
    "many items, biased": (1500, 64, 32, 64, [7, 60, 800, 1100, 1500], [3, 0, 250, 9], 0.0, True, True, 200),
    "group of 64": (260, 64, 1, 64, [0, 100, 190, 260], [20, 0, 7], 0.0, True, False, 0),
}


@pytest.mark.parametrize("where", ["Q", "K", "V", "dO", "all"])
@pytest.mark.parametrize("name", SPOILED)
def test_what_is_not_finite_reaches_what_sees_it_and_nothing_else(name, where):
    T, Hq, Hkv, d, starts, prefix, cap, biased, fused, max_len = SPOILED[name]
    pad = torch.ones(T, dtype=torch.bool, device="cuda")
    pad[starts[0]:starts[-1]] = False
    x = dict(zip(("Q", "K", "V", "dO"), _inputs(T, Hq, Hkv, d, fused, len(name), padding=pad)))
    clean = {n: torch.where(pad[:, None, None], 0.0, t.double()).to(bf16) for n, t in x.items()}
    r = random.Random(len(name) + len(where))
    bad = {n: torch.zeros(t.shape, dtype=torch.bool, device="cuda") for n, t in x.items()}
    for n in (x if where == "all" else [where]):
        for _ in range(3):                                             # (the last document but one holds most of them)
            t = r.randrange(starts[-3], starts[-2])
            t, h, c = r.choice([t, starts[-3], starts[-2] - 1, starts[-2]]), r.randrange(x[n].shape[1]), r.randrange(d)
            value = math.nan if n in "QK" else r.choice([math.nan, math.inf, -math.inf])
            x[n][t, h, c], bad[n][t, h, c] = value, True
    slopes = _slopes(Hq) if biased else None
    got = _run(x["Q"], x["K"], x["V"], x["dO"], _ints(starts), None if prefix is None else _ints(prefix), slopes, cap, max_len=max_len)
    for n in x:
        clean[n][bad[n]] = 0.0
    want, tol = doc_attention(clean["Q"], clean["K"], clean["V"], starts, prefix, slopes, cap, dO=clean["dO"])
    reached = _reached(doc_mask(T, starts, prefix, "cuda"), Hq // Hkv, bad)
    for n in want:
        assert torch.equal(got[n].isfinite() | (got[n] == -math.inf) & (n == "lse"), ~reached[n]), n
        check(n, torch.where(reached[n], want[n], got[n].double()), want[n], tol[n])


def test_a_batch_of_nothing_but_nan_ends():
    # the most that can be taken pair by pair: every value but the first document's is NaN, and ends no later for it than in seconds
    T, d = 6000, 64
    Q, K, V, dO = _inputs(T, 16, 4, d, seed=21)
    clean = [t.clone() for t in (Q, K, V, dO)]
    for t in (Q, K, V, dO):
        t[100:] = math.nan
    got = _run(Q, K, V, dO, _ints([0, 100, 3000, T]))
    for n, t in got.items():
        t = t.T if n == "lse" else t
        assert bool(t[100:].isnan().all()), n
    want, tol = doc_attention(*(t[:100] for t in clean[:3]), [0, 100], dO=clean[3][:100])
    for n in want:
        check(n, got[n][:, :100] if n == "lse" else got[n][:100], want[n], tol[n])


def test_what_is_not_finite_in_a_graph():
    # the same bits in every call, captured or not, and nothing is left behind for finite values
    Q, K, V, dO = _inputs(1300, 40, 20, 64, seed=22)
    clean = [t.clone() for t in (Q, K, V, dO)]
    starts = _ints([0, 300, 900, 1300])
    s = pisa.doc_shape_of(Q, K, V, starts)
    ws, wb = (pisa.doc_workspace(s, op, Q.device) for op in (pisa.DOC_FWD, pisa.DOC_BWD))

    def step():
        O, lse = pisa.doc_attn_fwd(Q, K, V, starts, s, ws=ws)
        return O, lse, *pisa.doc_attn_bwd(Q, K, V, O, lse, dO, starts, s, ws=wb)

    want = [[t.clone() for t in step()]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t, at in ((Q, (310, 3)), (K, (500, 7)), (V, (880, 1)), (dO, (301, 39))):
        t[at][5] = math.nan
    want.append([t.clone() for t in step()])
    for k in (1, 1, 0, 1):
        for t, c in zip((Q, K, V, dO), clean):
            bad = [(310, 3), (500, 7), (880, 1), (301, 39)]
            for at in bad:
                if at[1] < t.shape[1]:
                    t[at] = c[at]
        if k:
            for t, at in ((Q, (310, 3)), (K, (500, 7)), (V, (880, 1)), (dO, (301, 39))):
                t[at][5] = math.nan
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[k]):
            assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(nan=9e9), b.nan_to_num(nan=9e9))
    assert pisa.workspace_status(ws) == 0 and pisa.workspace_status(wb) == 0
