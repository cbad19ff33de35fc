"""Window attention, query/key norm and rotation without a GPU: the 64-bit reference against
differences, the refusals of the C ABI and of the binding, the host helpers."""
import ctypes
import math

import pytest
import torch

import pyramid_top_selection_gb300 as pisa
from pyramid_top_selection_gb300 import _pisa
from _window_ref import attention, visible

A = 1 << 20        # fake, 16-byte aligned address: never dereferenced


def _refused(fn, code, text, *args):
    rc = fn(*args)
    msg = pisa.lib().pisa_last_error().decode()
    assert rc == code and text in msg, (rc, msg)


def test_visible_keys_by_hand():
    see = visible(3, 6, 2, 1, 5)          # rows at 3, 4, 5; tokens 0..4 valid
    assert see.int().tolist() == [[1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0], [0, 0, 0, 0, 0, 0]]
    assert visible(4, 4, 9, 0, 4).int().tolist() == torch.tril(torch.ones(4, 4)).int().tolist()


def test_reference_gradients_match_differences():
    g = torch.Generator().manual_seed(0)
    B, Nq, N, Hq, Hkv, d = 1, 7, 9, 2, 1, 4
    Q, dO = (torch.randn(B, Nq, Hq, d, generator=g, dtype=torch.float64) for _ in range(2))
    K, V = (torch.randn(B, N, Hkv, d, generator=g, dtype=torch.float64) for _ in range(2))
    args = dict(window=3, sinks=2, lens=[8])
    out, _ = attention(Q, K, V, dO=dO, **args)
    for name, t in (("dQ", Q), ("dK", K), ("dV", V)):
        num = torch.zeros_like(t)
        for i in range(t.numel()):
            f = []
            for e in (1e-5, -1e-5):
                x = t.reshape(-1)[i].item()
                t.reshape(-1)[i] = x + e
                f.append((attention(Q, K, V, **args)[0]["O"] * dO).sum().item())
                t.reshape(-1)[i] = x
            num.reshape(-1)[i] = (f[0] - f[1]) / 2e-5
        torch.testing.assert_close(out[name], num, atol=1e-8, rtol=1e-6)


WIN = dict(B=2, Nq=100, N=300, Hq=8, Hkv=2, d=128, window=64, sinks=4)


@pytest.mark.parametrize("change,code,text", [
    (dict(B=0), _pisa.PISA_EINVAL, "positive"), (dict(window=0), _pisa.PISA_EINVAL, "positive"),
    (dict(sinks=-1), _pisa.PISA_EINVAL, "sinks"), (dict(Nq=301), _pisa.PISA_EINVAL, "exceeds N"),
    (dict(Hkv=3), _pisa.PISA_EINVAL, "multiple"), (dict(d=96), _pisa.PISA_EUNSUPPORTED, "head dim"),
    (dict(Hq=130, Hkv=2), _pisa.PISA_EUNSUPPORTED, "GQA group"), (dict(N=(1 << 24) + 1), _pisa.PISA_EUNSUPPORTED, "2^24"),
    (dict(B=1 << 12, N=1 << 20), _pisa.PISA_EUNSUPPORTED, "2^31"), (dict(scale=-1.0), _pisa.PISA_EINVAL, "scale"),
    (dict(scale=math.inf), _pisa.PISA_EINVAL, "scale"), (dict(scale=math.nan), _pisa.PISA_EINVAL, "scale"),
    (dict(q_stride=1000), _pisa.PISA_EINVAL, "q_stride"), (dict(k_stride=260), _pisa.PISA_EINVAL, "k_stride"),
    (dict(v_stride=-256), _pisa.PISA_EINVAL, "v_stride"),
])
def test_window_shapes_refused(change, code, text):
    L = pisa.lib()
    s = pisa.make_window_shape(**{**WIN, **change})
    _refused(L.pisa_window_attn_fwd, code, text, ctypes.byref(s), A, A, A, None, A, A, A, 1 << 40, None)
    _refused(L.pisa_window_attn_bwd, code, text, ctypes.byref(s), *[A] * 6, None, A, A, A, A, 1 << 40, None)
    _refused(L.pisa_window_workspace_size, code, text, ctypes.byref(s), 0, ctypes.byref(ctypes.c_size_t()))


def test_window_pointers_and_workspaces_refused():
    L = pisa.lib()
    s = pisa.make_window_shape(**WIN)
    fwd = [A, A, A, None, A, A, A, 1 << 40, None]
    names = ["Q", "K", "V", "len", "O", "lse"]
    for k, n in enumerate(names):
        for bad, text in ((A + 4, "aligned"), (None, "NULL")):
            if n == "len" and bad is None:
                continue
            _refused(L.pisa_window_attn_fwd, _pisa.PISA_EINVAL, f"{n} is {'NULL' if bad is None else 'not'}",
                     ctypes.byref(s), *fwd[:k], bad, *fwd[k + 1:])
    for op, fn, n in ((pisa.WINDOW_FWD, L.pisa_window_attn_fwd, 6), (pisa.WINDOW_BWD, L.pisa_window_attn_bwd, 10)):
        need = pisa.window_workspace_size(s, op)
        assert need >= 256
        _refused(fn, _pisa.PISA_EWORKSPACE, "workspace", ctypes.byref(s), *[A] * n, A, need - 1, None)
        _refused(fn, _pisa.PISA_EWORKSPACE, "NULL", ctypes.byref(s), *[A] * n, None, need, None)
        _refused(fn, _pisa.PISA_EINVAL, "aligned", ctypes.byref(s), *[A] * n, A + 8, need, None)
        _refused(fn, _pisa.PISA_EINVAL, "shape is NULL", None, *[A] * n, A, need, None)
    _refused(L.pisa_window_workspace_size, _pisa.PISA_EINVAL, "op", ctypes.byref(s), 2, ctypes.byref(ctypes.c_size_t()))


@pytest.mark.parametrize("change,code,text", [
    (dict(Ncap=0), _pisa.PISA_EINVAL, "positive"), (dict(Ncap=4), _pisa.PISA_EINVAL, "exceed sinks"),
    (dict(sinks=-2), _pisa.PISA_EINVAL, "sinks"), (dict(d=32), _pisa.PISA_EUNSUPPORTED, "head dim"),
    (dict(Hq=9), _pisa.PISA_EINVAL, "multiple"), (dict(B=65536), _pisa.PISA_EUNSUPPORTED, "65535"),
    (dict(Ncap=(1 << 24) + 1), _pisa.PISA_EUNSUPPORTED, "2^24"), (dict(scale=-2.0), _pisa.PISA_EINVAL, "scale"),
])
def test_window_decode_refused(change, code, text):
    s = pisa.make_window_decode_shape(**{**dict(B=2, Ncap=100, Hq=8, Hkv=2, d=64, window=32, sinks=4), **change})
    _refused(pisa.lib().pisa_window_decode_step, code, text, ctypes.byref(s), *[A] * 9, None)


def test_window_decode_pointers_refused():
    L = pisa.lib()
    s = pisa.make_window_decode_shape(2, 100, 8, 2, 64, 32, 4)
    names = ["pos", "Kcache", "Vcache", "q", "k_new", "v_new", "o", "lse", "status"]
    for k, n in enumerate(names):
        args = [A] * 9
        if n != "lse":
            _refused(L.pisa_window_decode_step, _pisa.PISA_EINVAL, f"{n} is NULL", ctypes.byref(s), *args[:k], None,
                     *args[k + 1:], None)
        _refused(L.pisa_window_decode_step, _pisa.PISA_EINVAL, f"{n} is not", ctypes.byref(s), *args[:k], A + 8,
                 *args[k + 1:], None)


@pytest.mark.parametrize("change,code,text", [
    (dict(N=0), _pisa.PISA_EINVAL, "positive"), (dict(d=80), _pisa.PISA_EUNSUPPORTED, "head dim"),
    (dict(rot=144), _pisa.PISA_EINVAL, "rot"), (dict(rot=-16), _pisa.PISA_EINVAL, "rot"),
    (dict(rot=24), _pisa.PISA_EUNSUPPORTED, "multiples of 16"), (dict(eps=-1.0), _pisa.PISA_EINVAL, "eps"),
    (dict(rot_scale=math.nan), _pisa.PISA_EINVAL, "rot_scale"), (dict(q_stride=512), _pisa.PISA_EINVAL, "q_stride"),
    (dict(k_stride=1028), _pisa.PISA_EINVAL, "k_stride"), (dict(B=1 << 16, N=1 << 16), _pisa.PISA_EUNSUPPORTED, "2^31"),
])
def test_rope_shapes_refused(change, code, text):
    L = pisa.lib()
    s = pisa.make_rope_shape(**{**dict(B=2, N=50, Hq=8, Hkv=2, d=128, rot=64), **change})
    _refused(L.pisa_qk_norm_rope, code, text, ctypes.byref(s), *[A] * 8, None)
    _refused(L.pisa_qk_norm_rope_bwd, code, text, ctypes.byref(s), *[A] * 12, A, 1 << 40, None)


def test_rope_arguments_refused():
    L = pisa.lib()
    s = pisa.make_rope_shape(2, 50, 8, 2, 128, 64, q_stride=2048)
    _refused(L.pisa_qk_norm_rope, _pisa.PISA_EINVAL, "inv_freq is NULL", ctypes.byref(s), A, A, None, A, A, A, A, A, None)
    _refused(L.pisa_qk_norm_rope, _pisa.PISA_EINVAL, "in place", ctypes.byref(s), A, 2 * A, A, A, A, A, A, 3 * A, None)
    plain = pisa.make_rope_shape(2, 50, 8, 2, 128, 64, norm=False)
    _refused(L.pisa_qk_norm_rope_bwd, _pisa.PISA_EINVAL, "weight gradients", ctypes.byref(plain), A, A, A, A, A, None,
             None, None, 2 * A, 2 * A, A, None, A, 1 << 40, None)
    _refused(L.pisa_qk_norm_rope_bwd, _pisa.PISA_EINVAL, "must not be Q", ctypes.byref(s), *[A] * 12, A, 1 << 40, None)
    b = ctypes.c_size_t()
    assert L.pisa_qk_norm_rope_workspace_size(ctypes.byref(s), ctypes.byref(b)) == 0 and b.value > 256
    _refused(L.pisa_qk_norm_rope_bwd, _pisa.PISA_EWORKSPACE, "workspace", ctypes.byref(s), *[A] * 8, 2 * A, 2 * A, A, A,
             A, b.value - 1, None)


def test_overlapping_buffers_refused():
    # 100 tokens of 2 x 64 and 1 x 64 bf16: 25600 and 12800 bytes; a fused projection interleaves its slices
    L = pisa.lib()
    q, k = 25600, 12800
    s = ctypes.byref(pisa.make_window_shape(1, 100, 100, 2, 1, 64, 10))
    far = [A + n * (1 << 20) for n in range(12)]
    for out in (far[0], far[0] + q - 16, far[1] + k - 16, far[2] - q + 16):
        _refused(L.pisa_window_attn_fwd, _pisa.PISA_EINVAL, "O overlaps", s, *far[:3], None, out, far[5], None, 0, None)
    _refused(L.pisa_window_attn_fwd, _pisa.PISA_EINVAL, "lse overlaps K", s, *far[:3], None, far[4], far[1], None, 0, None)
    for j, n in enumerate(["dQ", "dK", "dV", "workspace"]):
        out = far[6:10]
        for i, m in enumerate(["Q", "K", "V", "O", "lse", "dO"]):
            _refused(L.pisa_window_attn_bwd, _pisa.PISA_EINVAL, f"{n} overlaps {m}", s, *far[:6], None,
                     *out[:j], far[i], *out[j + 1:], 1 << 19, None)
    fused = ctypes.byref(pisa.make_window_shape(1, 100, 100, 2, 1, 64, 10, q_stride=256, k_stride=256, v_stride=256))
    _refused(L.pisa_window_attn_fwd, _pisa.PISA_EINVAL, "O overlaps", fused, A, A + 256, A + 384, None, A + 99 * 512, far[5],
             None, 0, None)
    r = ctypes.byref(pisa.make_rope_shape(1, 100, 2, 1, 64, 64))
    _refused(L.pisa_qk_norm_rope, _pisa.PISA_EINVAL, "Kr overlaps Q", r, far[0], far[1], far[2], None, None, None, far[3],
             far[0], None)
    _refused(L.pisa_qk_norm_rope, _pisa.PISA_EINVAL, "Qr overlaps Q", r, far[0], far[1], far[2], None, None, None, far[0] + 16,
             far[4], None)
    _refused(L.pisa_qk_norm_rope_bwd, _pisa.PISA_EINVAL, "dK overlaps dQr", r, *far[:5], None, None, None, far[6], far[2],
             None, None, far[8], 1 << 19, None)


def test_binding_refuses_expanded_and_far_apart_tokens():
    # tokens that share memory, or lie 2^31 elements apart, have no stride the shape can hold
    z = torch.zeros(2, 8, 4, 64, dtype=torch.bfloat16)
    s = pisa.window_shape_of(z, z, z, 4, 1)
    for bad in (z[:, :1].expand(2, 8, 4, 64), z[:1].expand(2, 8, 4, 64), z[:, :, :1].expand(2, 8, 4, 64),
                z[:1, :1].expand(2, 1, 4, 64), z.as_strided((2, 8, 4, 64), (8 * 128, 128, 64, 1)),
                z[:, :, :, :1].expand(2, 8, 4, 64),
                torch.empty(1 << 33, dtype=torch.bfloat16, device="meta").as_strided((2, 1, 4, 64), (1 << 32, 256, 64, 1))):
        with pytest.raises(ValueError, match="evenly spaced"):
            pisa.window_shape_of(z, bad, z, 4)
    with pytest.raises(ValueError, match="evenly spaced"):
        pisa.window_attn_fwd(z, z[:, :1].expand(2, 8, 4, 64), z, s)
    one = torch.zeros(1, 1, 4, 128, dtype=torch.bfloat16)[..., :64]          # a single token with gaps between its heads
    with pytest.raises(ValueError, match="evenly spaced"):
        pisa.window_attn_fwd(one, one, one, pisa.make_window_shape(1, 1, 1, 4, 4, 64, 1))


def test_binding_refuses_workspaces_and_status_words_elsewhere():
    z = torch.zeros(2, 8, 4, 64, dtype=torch.bfloat16)
    s = pisa.window_shape_of(z, z, z, 4, 1)
    lse = torch.zeros(2, 4, 8)
    for ws in (torch.zeros(1 << 16, dtype=torch.float32), torch.zeros(1 << 16, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match="ws must"):
            pisa.window_attn_fwd(z, z, z, s, ws=ws)
        with pytest.raises(ValueError, match="ws must"):
            pisa.window_attn_bwd(z, z, z, z, lse, z, s, ws=ws)
        with pytest.raises(ValueError, match="ws must"):
            pisa.qk_norm_rope_bwd(z, z, z, z, torch.zeros(32), pisa.rope_shape_of(z, z, 64), ws=ws)
    with pytest.raises(ValueError, match="status must"):
        pisa.window_decode_step(pisa.make_window_decode_shape(2, 8, 4, 4, 64, 4), torch.zeros(2, dtype=torch.int32), z, z,
                                z[:, 0].contiguous(), z[:, 0].contiguous(), z[:, 0].contiguous(),
                                status=torch.zeros(4))


def test_binding_refuses_tensors_that_do_not_fit():
    z = torch.zeros(2, 8, 4, 64, dtype=torch.bfloat16)
    s = pisa.window_shape_of(z, z, z, 4, 1)
    assert (s.q_stride, s.k_stride, s.v_stride) == (0, 0, 0)
    with pytest.raises(ValueError, match="CUDA"):
        pisa.window_attn_fwd(z, z, z, s)
    with pytest.raises(ValueError, match="CUDA"):
        pisa.qk_norm_rope(z, z, torch.zeros(32), pisa.rope_shape_of(z, z, 64))
    for bad in (z.float(), z[:, :7], z.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(ValueError, match="V "):
            pisa.window_attn_fwd(z, z, bad, s)
    with pytest.raises(ValueError, match="lens"):
        pisa.window_attn_fwd(z, z, z, s, lens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="out"):
        pisa.window_attn_fwd(z, z, z, s, out=z[:1])
    with pytest.raises(ValueError, match="dO"):
        pisa.window_attn_bwd(z, z, z, z, torch.zeros(2, 4, 8), z[:, :, :2], s)
    with pytest.raises(ValueError, match="inv_freq"):
        pisa.qk_norm_rope(z, z, torch.zeros(16), pisa.rope_shape_of(z, z, 64))
    with pytest.raises(ValueError, match="pos"):
        pisa.window_decode_step(pisa.make_window_decode_shape(2, 8, 4, 4, 64, 4), torch.zeros(2), z, z, z[:, 0],
                                z[:, 0], z[:, 0])
    with pytest.raises(ValueError, match="evenly spaced"):
        pisa.window_shape_of(z.transpose(1, 2), z, z, 4)
    with pytest.raises(ValueError, match="evenly spaced"):
        pisa.rope_shape_of(z[:, ::2, :, :].expand(2, 4, 4, 64)[:, :3], z, 64)


def test_strides_of_projection_slices():
    x = torch.zeros(3, 5, 8, 64, dtype=torch.bfloat16)
    s = pisa.window_shape_of(x[:, :, :4], x[:, :, 4:6], x[:, :, 6:], 4)
    assert (s.q_stride, s.k_stride, s.v_stride) == (512, 512, 512)
    assert pisa.rope_shape_of(x[:, :1, :4], x[:, :1, 4:5], 64).q_stride == 5 * 512       # one token a sequence
    assert pisa.rope_shape_of(x[:1, :1, :4], x[:1, :1, 4:5], 64).q_stride == 0           # a single token


def test_rope_frequencies():
    f, m = pisa.rope_frequencies(64)
    want = torch.tensor([10000.0 ** (-2 * c / 64) for c in range(32)])
    torch.testing.assert_close(f, want, rtol=2 ** -23, atol=0)
    assert m == 1.0 and f.dtype == torch.float32
    lin, m = pisa.rope_frequencies(64, scaling="linear", factor=4)
    torch.testing.assert_close(lin, want / 4, rtol=2 ** -23, atol=0)
    ntk, m = pisa.rope_frequencies(64, scaling="ntk", factor=4)
    assert m == 1.0 and ntk[0] == 1
    torch.testing.assert_close(ntk[-1], want[-1] / 4, rtol=1e-5, atol=0)
    yarn, m = pisa.rope_frequencies(64, scaling="yarn", factor=4, trained_len=4096)
    turns = 4096 * want / (2 * math.pi)
    assert math.isclose(m, 0.1 * math.log(4) + 1)
    torch.testing.assert_close(yarn[turns > 32], want[turns > 32], rtol=1e-6, atol=0)
    torch.testing.assert_close(yarn[turns < 1], want[turns < 1] / 4, rtol=1e-6, atol=0)
    mid = (turns > 1) & (turns < 32)
    assert bool(mid.any()) and bool(((yarn < want) & (yarn > want / 4))[mid].all())
    for bad in (dict(rot=7), dict(rot=0), dict(rot=64, factor=0.5), dict(rot=64, scaling="yarn", factor=2),
                dict(rot=64, scaling="other"), dict(rot=2, scaling="ntk", factor=2)):
        with pytest.raises(ValueError):
            pisa.rope_frequencies(**bad)
