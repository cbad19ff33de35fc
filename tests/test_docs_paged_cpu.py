"""The documents' attention and the paged cache without a GPU: refusals before any CUDA call, sizes of workspaces, and the
64-bit definitions that the GPU tests go by against plainer ones."""
import ctypes
import math

import pytest
import torch

import pyramid_top_selection_gb300 as pisa
from _docs_ref import CODES, doc_attention, doc_mask, paged_attention, quantise
from pyramid_top_selection_gb300 import _pisa
from _window_ref import attention

A = 1 << 24        # fake, 16-byte aligned addresses: never dereferenced
EINVAL, EUNSUP, EWS = _pisa.PISA_EINVAL, _pisa.PISA_EUNSUPPORTED, _pisa.PISA_EWORKSPACE


def _said(rc, code, text):
    msg = pisa.lib().pisa_last_error().decode()
    assert rc == code and text in msg, (rc, msg)


# ---------------------------------------------------------------------------------------- shapes
DOC = dict(T=100, Hq=4, Hkv=2, d=64, n_docs=3)
PAGED = dict(B=2, Hq=4, Hkv=2, d=64, n_pages=8, page=16, max_pages=4)


@pytest.mark.parametrize("change,code,text", [
    (dict(T=0), EINVAL, "positive"), (dict(n_docs=0), EINVAL, "positive"), (dict(Hq=5), EINVAL, "multiple"),
    (dict(d=96), EUNSUP, "head dim"), (dict(Hq=130), EUNSUP, "GQA group"), (dict(T=(1 << 24) + 1), EUNSUP, "2^24"),
    (dict(T=1 << 24, Hq=128, Hkv=128), EUNSUP, "2^31"), (dict(cap=-1.0), EINVAL, "cap"), (dict(cap=1e-9), EINVAL, "cap"),
    (dict(cap=math.nan), EINVAL, "cap"), (dict(cap=math.inf), EINVAL, "cap"),
    (dict(cap=2.0 ** -10, scale=1.5), EUNSUP, "1024"), (dict(scale=math.inf), EINVAL, "scale"),
    (dict(scale=-1.0), EINVAL, "scale"), (dict(q_stride=255), EINVAL, "q_stride"), (dict(k_stride=64), EINVAL, "k_stride"),
    (dict(v_stride=132), EINVAL, "v_stride"),
])
def test_document_shapes_are_checked(change, code, text):
    n = ctypes.c_size_t()
    s = pisa.make_doc_shape(**(DOC | change))
    for op in (pisa.DOC_FWD, pisa.DOC_BWD):
        _said(pisa.lib().pisa_doc_workspace_size(ctypes.byref(s), op, ctypes.byref(n)), code, text)


@pytest.mark.parametrize("change,code,text", [
    (dict(B=0), EINVAL, "positive"), (dict(n_pages=0), EINVAL, "positive"), (dict(max_pages=0), EINVAL, "positive"),
    (dict(Hkv=3), EINVAL, "multiple"), (dict(d=32), EUNSUP, "head dim"), (dict(Hq=130), EUNSUP, "GQA group"),
    (dict(bits=8), EUNSUP, "bits"), (dict(page=8), EUNSUP, "page"), (dict(page=48), EUNSUP, "page"), (dict(page=2048), EUNSUP, "page"),
    (dict(max_pages=(1 << 20) + 1), EUNSUP, "2^24"), (dict(nq=0), EUNSUP, "nq"), (dict(nq=17), EUNSUP, "nq"),
    (dict(B=1 << 23), EUNSUP, "2^24"), (dict(n_pages=(1 << 31) - 1, page=1024), EUNSUP, "2^39"), (dict(Hq=1 << 16, Hkv=1 << 16, page=1024), EUNSUP, "2^30"),
    (dict(B=1 << 12, Hq=1 << 10, Hkv=1 << 8, max_pages=1 << 20), EUNSUP, "2^44"), (dict(cap=2e6), EINVAL, "cap"), (dict(cap=0.5, scale=1e4), EUNSUP, "1024"),
    (dict(scale=math.nan), EINVAL, "scale"),
])
def test_paged_shapes_are_checked(change, code, text):
    n = ctypes.c_size_t()
    s = pisa.make_paged_shape(**(PAGED | change))
    _said(pisa.lib().pisa_paged_workspace_size(ctypes.byref(s), ctypes.byref(n)), code, text)


def test_sizes_that_do_not_fit_32_bits_are_refused():
    with pytest.raises(ValueError, match="T="):
        pisa.make_doc_shape(**(DOC | dict(T=(1 << 32) + 4)))
    with pytest.raises(ValueError, match="max_len"):
        pisa.make_doc_shape(**DOC, max_len=1 << 31)
    with pytest.raises(ValueError, match="n_pages"):
        pisa.make_paged_shape(**(PAGED | dict(n_pages=1 << 31)))
    with pytest.raises(pisa.PisaError, match="negative"):
        pisa.doc_workspace_size(pisa.make_doc_shape(**DOC, max_len=-1), pisa.DOC_FWD)
    with pytest.raises(pisa.PisaError, match="unknown op"):
        pisa.doc_workspace_size(pisa.make_doc_shape(**DOC), 2)


# -------------------------------------------------------------------------------------- buffers
def _overlaps(call, names, sizes, written, may_be=()):
    """Every buffer in `written` laid over every other one, at its first and its last 16 bytes, is refused by name."""
    far = {n: A + (k << 28) for k, n in enumerate(names)}
    for w in written:
        for r in names:
            if r == w:
                continue
            for at in (0, max(16, -(-sizes[r] // 16) * 16) - 16):
                if ((w, r) in may_be or (r, w) in may_be) and at == 0:
                    continue
                rc = call({n: far[r] + at if n == w else far[n] for n in names})
                msg = pisa.lib().pisa_last_error().decode()
                assert rc == EINVAL and (f"{w} overlaps {r}" in msg or f"{r} overlaps {w}" in msg), (w, r, rc, msg)


def _doc_calls():
    # 4 heads of 12000 tokens: more items than the GPU has SMs, so that the forward has a workspace of its own
    L, s = pisa.lib(), pisa.make_doc_shape(T=12000, Hq=4, Hkv=4, d=64, n_docs=300)
    nf, nb = (pisa.doc_workspace_size(s, op) for op in (pisa.DOC_FWD, pisa.DOC_BWD))
    fwd = ["Q", "K", "V", "starts", "prefix", "slopes", "O", "lse", "workspace"]
    bwd = ["Q", "K", "V", "O", "lse", "dO", "starts", "prefix", "slopes", "dQ", "dK", "dV", "workspace"]
    return (fwd, lambda a, n=nf: L.pisa_doc_attn_fwd(ctypes.byref(s), *(a[x] for x in fwd), n, None), nf,
            bwd, lambda a, n=nb: L.pisa_doc_attn_bwd(ctypes.byref(s), *(a[x] for x in bwd), n, None), nb)


def test_overlaps_of_the_documents_calls_are_refused():
    fwd, call_f, nf, bwd, call_b, nb = _doc_calls()
    t = 12000 * 4 * 64 * 2
    size = dict(Q=t, K=t, V=t, O=t, dO=t, dQ=t, dK=t, dV=t, lse=192000, starts=1204, prefix=1200, slopes=16)
    _overlaps(call_f, fwd, size | dict(workspace=nf), ["O", "lse", "workspace"])
    _overlaps(call_b, bwd, size | dict(workspace=nb), ["dQ", "dK", "dV", "workspace"])


def test_missing_and_misaligned_buffers_of_the_documents_calls_are_refused():
    fwd, call_f, nf, bwd, call_b, nb = _doc_calls()
    for names, call, need in ((fwd, call_f, nf), (bwd, call_b, nb)):
        far = {n: A + (k << 28) for k, n in enumerate(names)}
        for n in names:
            if n not in ("prefix", "slopes"):
                _said(call(far | {n: None}), EWS if n == "workspace" else EINVAL, f"{n} is NULL")
            _said(call(far | {n: far[n] + 4}), EINVAL, f"{n} is not 16-byte aligned")
        _said(call(far, need - 1), EWS, "workspace")


def _paged_calls(bits):
    L, s = pisa.lib(), pisa.make_paged_shape(B=2, Hq=4, Hkv=4, d=64, n_pages=8, page=16, max_pages=4, bits=bits)
    t = pisa.make_rope_shape(2, 50, 4, 4, 64, 64)
    need = ctypes.c_size_t()
    assert L.pisa_paged_workspace_size(ctypes.byref(s), ctypes.byref(need)) == 0
    tensors = ["k", "v"] + (["k_scale", "v_scale", "k_amp", "v_amp"] if bits == 4 else [])
    rest = ["Q", "K", "V", "inv_freq", "q_weight", "k_weight", "table", "seq", "pos", "Qr", "status"]
    att = ["table", "len", "q", "slopes", "o", "lse", "workspace"]

    def cache(a):
        return _pisa._PagedCache(*(a.get(n) for n in ("k", "v", "k_scale", "v_scale", "k_amp", "v_amp")))

    def append(a, tokens=t, v_stride=0):
        c = cache(a)
        return L.pisa_paged_append(ctypes.byref(s), ctypes.byref(c), ctypes.byref(tokens), a["Q"], a["K"], a["V"], v_stride,
                                   *(a[n] for n in rest[3:]), None)

    def attn(a, n=need.value):
        c = cache(a)
        return L.pisa_paged_attn(ctypes.byref(s), ctypes.byref(c), *(a[x] for x in att), n, None)

    rows = 8 * 16 * 4
    size = dict(k=rows * (128 if bits == 16 else 32), v=rows * (128 if bits == 16 else 32), k_scale=rows * 4, v_scale=rows * 4,
                k_amp=16, v_amp=16, Q=51200, K=51200, V=51200, Qr=51200, inv_freq=128, q_weight=256, k_weight=256, table=32, seq=400,
                pos=400, status=4, len=8, q=1024, o=1024, lse=32, slopes=16, workspace=need.value)
    return tensors, rest, att, append, attn, size, need.value


@pytest.mark.parametrize("bits", [16, 4])
def test_overlaps_of_the_paged_calls_are_refused(bits):
    tensors, rest, att, append, attn, size, _ = _paged_calls(bits)
    _overlaps(append, tensors + rest, size, [t for t in tensors if "amp" not in t] + ["Qr", "status"], [("Qr", "Q")])
    _overlaps(attn, tensors + att, size, ["o", "lse", "workspace"])


@pytest.mark.parametrize("bits", [16, 4])
def test_missing_and_misaligned_buffers_of_the_paged_calls_are_refused(bits):
    tensors, rest, att, append, attn, _, need = _paged_calls(bits)
    for names, call, may in ((tensors + rest, append, ("q_weight", "k_weight", "seq", "k_amp", "v_amp")),
                             (tensors + att, attn, ("slopes", "lse", "k_amp", "v_amp"))):
        far = {n: A + (k << 28) for k, n in enumerate(names)}
        for n in names:
            if n not in may:
                text = "both" if n in ("Q", "Qr") else f"{n} is NULL"
                _said(call(far | {n: None}), EWS if n == "workspace" else EINVAL, text)
            _said(call(far | {n: far[n] + 8}), EINVAL, f"{n} is not 16-byte aligned")
    far = {n: A + (k << 28) for k, n in enumerate(tensors + att)}
    _said(attn(far, need - 1), EWS, "workspace")
    if bits == 16:
        _said(attn(far | dict(k_scale=A >> 1)), EINVAL, "no scales")


def test_append_checks_its_tokens_against_the_cache():
    tensors, rest, _, append, _, _, _ = _paged_calls(16)
    far = {n: A + (k << 28) for k, n in enumerate(tensors + rest)}
    _said(append(far, pisa.make_rope_shape(2, 50, 4, 2, 64, 64)), EINVAL, "the cache")
    _said(append(far, pisa.make_rope_shape(2, 50, 4, 4, 128, 64)), EINVAL, "the cache")
    _said(append(far | dict(seq=None), pisa.make_rope_shape(1, 100, 4, 4, 64, 64)), EINVAL, "without seq")
    _said(append(far, pisa.make_rope_shape(2, 50, 4, 4, 64, 65)), EINVAL, "rot")
    _said(append(far, v_stride=100), EINVAL, "v_stride")
    _said(append(far | dict(Qr=far["Q"]), pisa.make_rope_shape(2, 50, 4, 4, 64, 64, q_stride=512)), EINVAL, "in place")


def test_the_binding_checks_tensors():
    Q, K = torch.zeros(10, 4, 64, dtype=torch.bfloat16), torch.zeros(10, 2, 64, dtype=torch.bfloat16)
    starts = torch.tensor([0, 10], dtype=torch.int32)
    s = pisa.doc_shape_of(Q, K, K, starts)
    assert (s.T, s.Hq, s.Hkv, s.d, s.n_docs) == (10, 4, 2, 64, 1)
    with pytest.raises(ValueError, match="CUDA"):
        pisa.doc_attn_fwd(Q, K, K, starts, s)
    with pytest.raises(ValueError, match="starts"):
        pisa.doc_attn_fwd(Q, K, K, starts.long(), s)
    with pytest.raises(ValueError, match="prefix"):
        pisa.doc_attn_fwd(Q, K, K, starts, s, prefix=starts)
    with pytest.raises(ValueError, match="slopes"):
        pisa.doc_attn_fwd(Q, K, K, starts, s, slopes=torch.zeros(2))
    with pytest.raises(ValueError, match="V must"):
        pisa.doc_attn_fwd(Q, K, K.float(), starts, s)
    with pytest.raises(ValueError, match="evenly spaced"):
        pisa.doc_shape_of(Q.transpose(0, 1).contiguous().transpose(0, 1), K, K, starts)
    x = torch.zeros(10, 8, 64, dtype=torch.bfloat16)
    s = pisa.doc_shape_of(x[:, :4], x[:, 4:6], x[:, 6:], starts)
    assert (s.q_stride, s.k_stride, s.v_stride) == (512, 512, 512)
    with pytest.raises(ValueError, match="strides"):
        pisa.doc_attn_fwd(Q, x[:, 4:6], x[:, 6:], starts, s)

    table = torch.zeros(2, 4, dtype=torch.int32)
    for bits in (16, 4):
        shape = pisa.make_paged_shape(**PAGED, bits=bits)
        cache = pisa.paged_cache(shape, "cpu")
        again = pisa.paged_shape_of(cache, table, 4)
        assert bytes(again) == bytes(shape)
        q, lens = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
        with pytest.raises(ValueError, match="CUDA"):
            pisa.paged_attn(shape, cache, table, lens, q)
        with pytest.raises(ValueError, match="table"):
            pisa.paged_attn(shape, cache, table[:, :3], lens, q)
        with pytest.raises(ValueError, match="lens"):
            pisa.paged_attn(shape, cache, table, lens.long(), q)
        with pytest.raises(ValueError, match="q must"):
            pisa.paged_attn(shape, cache, table, lens, q[:, 0])
        with pytest.raises(ValueError, match="k must"):
            pisa.paged_attn(shape, cache._replace(k=cache.k[1:]), table, lens, q)
        with pytest.raises(ValueError, match="scale"):
            pisa.paged_attn(shape, cache._replace(k_scale=None if bits == 4 else lens), table, lens, q)
        pos = torch.zeros(10, dtype=torch.int32)
        with pytest.raises(ValueError, match="CUDA"):
            pisa.paged_append(shape, cache, table, pos, K, K)
        with pytest.raises(ValueError, match="needs rope"):
            pisa.paged_append(shape, cache, table, pos, K, K, Q=Q)
        with pytest.raises(ValueError, match="without seq"):
            pisa.paged_append(shape, cache, table, pos[:9], K[:9], K[:9])
        with pytest.raises(ValueError, match="no tokens"):
            pisa.paged_append(shape, cache, table, pos[:0], K[:0], K[:0])
        with pytest.raises(ValueError, match="pos"):
            pisa.paged_append(shape, cache, table, pos[:8], K, K)
        with pytest.raises(ValueError, match="q_out"):
            pisa.paged_append(shape, cache, table, pos, K, K, q_out=Q)
        with pytest.raises(ValueError, match="inv_freq"):
            pisa.paged_append(shape, cache, table, pos, K, K, rope=pisa.Rope(torch.zeros(3), 16))


# ---------------------------------------------------------------------------------- definitions
def test_the_mask_pair_by_pair():
    starts, prefix, T = [2, 5, 5, 11, 40], [1, 0, 4, 9], 14
    see = doc_mask(T, starts, prefix)
    for t in range(T):
        for j in range(T):
            m = [x for x in range(4) if starts[x] <= t < starts[x + 1]]
            want = bool(m) and starts[m[0]] <= j < min(T, starts[m[0] + 1]) and (j <= t or j < starts[m[0]] + prefix[m[0]])
            assert bool(see[t, j]) == want, (t, j)


def test_one_document_without_extras_is_full_causal_attention():
    g = torch.Generator().manual_seed(0)
    Q, K, V, dO = (torch.randn(50, h, 64, generator=g).double() for h in (4, 2, 2, 4))
    a, _ = doc_attention(Q, K, V, [0, 50], dO=dO)
    b, _ = attention(Q[None], K[None], V[None], 50, 0, dO=dO[None])
    for n in a:
        assert torch.allclose(a[n], b[n][0], rtol=1e-12, atol=1e-12), n


def test_gradients_of_the_definition_by_autograd():
    g = torch.Generator().manual_seed(1)
    Q, K, V, dO = (torch.randn(40, h, 64, generator=g).double() for h in (4, 2, 2, 4))
    slopes, cap, starts, prefix = torch.tensor([.5, .1, .02, 0.]), 3.0, [0, 25, 40], [7, 0]
    out, _ = doc_attention(Q, K, V, starts, prefix, slopes, cap, dO=dO)
    q, k, v = (x.clone().requires_grad_() for x in (Q, K, V))
    see, i = doc_mask(40, starts, prefix), torch.arange(40)
    rep = lambda x: x.repeat_interleave(2, 1)                          # noqa: E731
    x = torch.einsum("ihd,jhd->hij", q, rep(k)) / 8
    x = cap * torch.tanh(x / cap) - slopes[:, None, None].double() * (i[:, None] - i).abs()
    o = torch.einsum("hij,jhd->ihd", x.masked_fill(~see, -math.inf).softmax(-1), rep(v))
    (o * dO).sum().backward()
    assert torch.allclose(o, out["O"])
    for n, t in (("dQ", q), ("dK", k), ("dV", v)):
        assert torch.allclose(out[n], t.grad, rtol=1e-10, atol=1e-12), n


def test_the_paged_definition_is_the_documents_last_rows():
    g = torch.Generator().manual_seed(2)
    lens, Hq, Hkv = [30, 1, 17], 4, 2
    Q, K, V = (torch.randn(sum(lens), h, 64, generator=g).double() for h in (Hq, Hkv, Hkv))
    starts = [0, 30, 31, 48]
    slopes = torch.tensor([.5, .1, .02, 0.])
    want, _ = doc_attention(Q, K, V, starts, None, slopes, 3.0)
    parts = [(x[:30], x[30:31], x[31:]) for x in (K, V)]
    last = torch.stack([Q[[s - 1]] for s in starts[1:]])
    got, _ = paged_attention(last, parts[0], parts[1], lens, slopes, 3.0)
    for b, s in enumerate(starts[1:]):
        assert torch.allclose(got["O"][b, 0], want["O"][s - 1]) and torch.allclose(got["lse"][b, 0], want["lse"][:, s - 1])


def test_codes_by_comparing_with_every_one():
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(500, 64, generator=g) * 2).to(torch.bfloat16).double()
    codes, scales = quantise(x)
    assert torch.equal(scales.float(), (x.reshape(500, 4, 16).abs().amax(-1) / 6).float().to(torch.float8_e4m3fn).float())
    grid = torch.tensor(CODES, dtype=torch.float64)
    q = x.abs().reshape(500, 4, 16) / scales[..., None]
    off = (q[..., None] - grid).abs()
    got = codes.reshape(500, 4, 16) % 8
    assert torch.equal(off.gather(-1, got[..., None])[..., 0], off.amin(-1))
    tied = (off == off.amin(-1, keepdim=True)).sum(-1) > 1
    assert int(tied.sum()) > 50 and bool((got[tied] % 2 == 0).all())
    assert torch.equal(codes >= 8, torch.signbit(x))


def test_append_of_more_rows_than_32_bits_is_refused():
    # queries, keys and values of all tokens together: 180M tokens of 4 + 2 x 4 heads, which the norm and rotation would take (4 + 4)
    tensors, rest, _, append, _, _, _ = _paged_calls(16)
    far = {n: A + (k << 28) for k, n in enumerate(tensors + rest)}
    _said(append(far, pisa.make_rope_shape(1, 180_000_000, 4, 4, 64, 64)), pisa._pisa.PISA_EUNSUPPORTED, "2Hkv")
