"""The paged key/value cache on the GPU: appends (norm, rotation, 16- and 4-bit pages) and the attention of the last tokens
over it, against 64-bit definitions with bounds that count the kernels' roundings (_docs_ref.py); prompts, appends and
decode steps run together."""
import math

import pytest
import torch

import pyramid_top_selection_gb300 as pisa
from _docs_ref import codes_of, doc_attention, paged_attention, quantise, values_of
from _window_ref import check

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *size, scale=1.0):
    return (torch.randn(*size, generator=g, device="cuda") * scale).to(bf16)


def _slopes(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")


def _table(g, lens, page, spare=2, width=0):
    """A page table in random order; entries behind a sequence's pages hold what nothing may read."""
    need = [-(-n // page) for n in lens]
    pool = max(1, sum(need) + spare)
    ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, width, *need)), 0x7fffffff, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, pool


def _keys(cache, table, lens, page):
    """Every sequence's keys and values in order, float64 [tokens,Hkv,d]."""
    out = []
    for t, sc, amp in ((cache.k, cache.k_scale, cache.k_amp), (cache.v, cache.v_scale, cache.v_amp)):
        x = t.double() if sc is None else values_of(t, sc, amp)
        out.append([x[table[b, :max(1, -(-n // page))].long().clamp(0, len(x) - 1)].transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[:n]
                    for b, n in enumerate(lens)])
    return out


def _filled(g, shape, amps=True):
    """A cache full of values (all slots, so that what lies behind a sequence's end is not zero)."""
    size = (shape.n_pages, shape.Hkv, shape.page, shape.d)
    if shape.bits == 16:
        return pisa.PagedCache(_randn(g, *size), _randn(g, *size))
    parts = []
    for _ in range(2):
        c, s = quantise(torch.randn(*size, generator=g, device="cuda").double())
        c = c.to(torch.uint8).reshape(*size[:3], -1, 2)
        parts.append(((c[..., 0] | c[..., 1] << 4).contiguous(), s.float().to(torch.float8_e4m3fn)))
    amp = [0.5 + torch.rand(shape.Hkv, generator=g, device="cuda") if amps else None for _ in range(2)]
    return pisa.PagedCache(parts[0][0], parts[1][0], parts[0][1], parts[1][1], *amp)


# ------------------------------------------------------------------------------------- attention
CASES = {  # B, nq, Hq, Hkv, d, page, lens, cap, slopes
    "one key": (1, 1, 1, 1, 64, 16, [1], 0.0, False),
    "nothing in the cache": (2, 1, 4, 2, 128, 16, [0, 0], 0.0, False),
    "lengths around pages and chunks": (9, 1, 8, 1, 128, 16, [0, 1, 15, 16, 17, 31, 32, 33, 100], 0.0, False),
    "one long sequence": (1, 1, 16, 2, 128, 64, [5000], 0.0, False),
    "one long sequence, capped": (1, 1, 8, 1, 64, 128, [7001], 5.0, False),
    "several heads, d 64": (3, 1, 12, 4, 64, 32, [777, 1, 300], 0.0, True),
    "drafts": (4, 4, 8, 2, 128, 16, [500, 3, 0, 65], 0.0, False),
    "drafts, three heads a group": (3, 5, 9, 3, 64, 16, [130, 4, 1000], 20.0, True),
    "sixteen drafts": (2, 16, 4, 2, 128, 64, [300, 9], 0.0, True),
    "group of 64": (1, 1, 64, 1, 64, 64, [333], 0.0, False),
    "group of 64, drafts": (1, 3, 64, 1, 128, 32, [200], 30.0, False),
    "group of 12": (2, 2, 24, 2, 128, 256, [600, 257], 0.0, False),
    "many sequences": (40, 1, 4, 2, 64, 16, [(37 * b) % 211 for b in range(40)], 0.0, False),
    "whole pages of 1024": (2, 1, 8, 8, 64, 1024, [1024, 2049], 0.0, True),
    "uneven": (3, 1, 32, 8, 128, 64, [3000, 1, 700], 0.0, False),
}


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("name", CASES)
def test_attention_against_definition(name, bits):
    B, nq, Hq, Hkv, d, page, lens, cap, biased = CASES[name]
    g = _gen(len(name))
    table, pool = _table(g, lens, page)
    shape = pisa.make_paged_shape(B, Hq, Hkv, d, pool, page, table.shape[1], bits, nq, cap=cap)
    cache = _filled(g, shape)
    q = _randn(g, B, nq, Hq, d, scale=2.0 if cap else 1.0)
    slopes = _slopes(Hq) if biased else None
    ws = pisa.paged_workspace(shape, "cuda")
    ws.fill_(0xAB)
    o = torch.full((B, nq, Hq, d), 7.0, dtype=bf16, device="cuda")
    lse = torch.full((B, nq, Hq), 7.0, device="cuda")
    pisa.paged_attn(shape, cache, table, _ints(lens), q, slopes, ws=ws, o=o, lse=lse)
    assert pisa.workspace_status(ws) == 0
    k, v = _keys(cache, table, lens, page)
    want, tol = paged_attention(q, k, v, lens, slopes, cap)
    check("o", o, want["O"], tol["O"])
    check("lse", lse, want["lse"], tol["lse"])


@pytest.mark.parametrize("bits", [16, 4])
def test_what_lies_behind_a_sequence_is_not_used(bits):
    g = _gen(1)
    lens, page = [5, 40, 16, 0], 16
    table, pool = _table(g, lens, page)
    shape = pisa.make_paged_shape(4, 8, 2, 128, pool, page, table.shape[1], bits, 2)
    cache = _filled(g, shape)
    q = _randn(g, 4, 2, 8, 128)
    o0, lse0 = pisa.paged_attn(shape, cache, table, _ints(lens), q)
    used = torch.zeros(pool, page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for p in range(n):
            used[table[b, p // page], p % page] = True
    dark = ~used[:, None, :, None]
    if bits == 16:
        cache.k.masked_fill_(dark, math.nan)
        cache.v.masked_fill_(dark, math.inf)
    else:
        cache.k_scale.view(torch.uint8).masked_fill_(dark, 0x7f)
        cache.v_scale.view(torch.uint8).masked_fill_(dark, 0x7f)
    o1, lse1 = pisa.paged_attn(shape, cache, table, _ints(lens), q)
    assert torch.equal(o0, o1) and torch.equal(lse0, lse1)
    assert bool(torch.isfinite(o1).all())


@pytest.mark.parametrize("bits", [16, 4])
def test_pages_in_another_order_give_the_same_bits(bits):
    g = _gen(2)
    lens, page = [900, 333], 32
    table, pool = _table(g, lens, page)
    shape = pisa.make_paged_shape(2, 8, 2, 64, pool, page, table.shape[1], bits)
    cache = _filled(g, shape)
    q = _randn(g, 2, 1, 8, 64)
    o0, lse0 = pisa.paged_attn(shape, cache, table, _ints(lens), q)
    perm = torch.randperm(pool, generator=g, device="cuda")
    moved = pisa.PagedCache(*(t if t is None or i > 3 else t.view(torch.uint8)[perm].view(t.dtype) if t.dtype == torch.float8_e4m3fn else t[perm]
                              for i, t in enumerate(cache)))
    back = torch.empty_like(perm)
    back[perm] = torch.arange(pool, device="cuda")
    table2 = table.clone()
    for b, n in enumerate(lens):
        m = -(-n // page)
        table2[b, :m] = back[table[b, :m].long()].to(torch.int32)
    o1, lse1 = pisa.paged_attn(shape, moved, table2, _ints(lens), q)
    assert torch.equal(o0, o1) and torch.equal(lse0, lse1)


def test_a_page_used_by_two_sequences():
    # a shared prompt: the same pages at the head of both
    g = _gen(3)
    shape = pisa.make_paged_shape(2, 4, 2, 128, 6, 16, 4)
    cache = _filled(g, shape)
    table = _ints([[0, 1, 2, 3], [0, 1, 4, 5]])
    lens = [60, 50]
    q = _randn(g, 2, 1, 4, 128)
    o, lse = pisa.paged_attn(shape, cache, table, _ints(lens), q)
    k, v = _keys(cache, table, lens, 16)
    want, tol = paged_attention(q, k, v, lens)
    check("o", o, want["O"], tol["O"])
    check("lse", lse, want["lse"], tol["lse"])


@pytest.mark.parametrize("bits", [16, 4])
def test_pages_and_lengths_out_of_range_are_reported(bits):
    g = _gen(4)
    page, lens = 16, [100, 100, 50]
    table, pool = _table(g, lens, page)
    shape = pisa.make_paged_shape(3, 4, 2, 64, pool, page, table.shape[1], bits)
    cache = _filled(g, shape)
    q = _randn(g, 3, 1, 4, 64)
    table[0, 2], table[0, 5], table[1, :] = -1, pool, -7               # holes, and a sequence without any page
    ws = pisa.paged_workspace(shape, "cuda")
    o, lse = pisa.paged_attn(shape, cache, table, _ints(lens), q, ws=ws)
    assert pisa.workspace_status(ws) == pisa.STATUS_POS_RANGE
    k, v = _keys(cache, table, lens, page)
    hole = [torch.zeros(n, dtype=torch.bool, device="cuda") for n in lens]
    hole[0][32:48], hole[0][80:96], hole[1][:] = True, True, True
    want, tol = paged_attention(q, k, v, lens, hidden=hole)
    check("o", o, want["O"], tol["O"])
    check("lse", lse, want["lse"], tol["lse"])
    # lengths outside [0, max_pages * page]
    table, pool = _table(_gen(4), [112, 112, 112], page)
    shape = pisa.make_paged_shape(3, 4, 2, 64, pool, page, 7, bits)
    cache = _filled(g, shape)
    o, lse = pisa.paged_attn(shape, cache, table, _ints([-3, 113, 112]), q, ws=ws)
    assert pisa.workspace_status(ws) == pisa.STATUS_POS_RANGE
    clamped = [0, 112, 112]
    k, v = _keys(cache, table, clamped, page)
    want, tol = paged_attention(q, k, v, clamped)
    check("o", o, want["O"], tol["O"])
    check("lse", lse, want["lse"], tol["lse"])


# ---------------------------------------------------------------------------------------- append
APPENDS = {  # B, lens, first positions, Hq, Hkv, d, page, rot, interleaved, norm, with Q, fused, padding
    "one token": (1, [1], [0], 4, 2, 128, 16, 128, False, True, True, False, 0),
    "prompts": (3, [100, 7, 33], [0, 0, 0], 8, 2, 128, 16, 128, False, True, True, False, 3),
    "chunks behind what is there": (2, [40, 50], [13, 1000], 4, 4, 64, 32, 64, True, True, True, True, 0),
    "decode": (16, [1] * 16, [17 * b for b in range(16)], 32, 8, 128, 16, 128, False, True, True, False, 0),
    "no queries": (2, [20, 3], [5, 0], 4, 1, 128, 64, 32, False, False, False, False, 1),
    "as they are": (2, [70, 64], [0, 0], 4, 2, 64, 16, 0, False, False, False, True, 0),
    "part of the head": (1, [333], [70000], 6, 3, 128, 128, 48, False, True, True, True, 0),
    "many tokens": (4, [1500, 1700, 900, 1], [0, 3, 0, 16], 4, 2, 64, 64, 64, False, True, True, False, 9),
    "many tokens, wide": (2, [2500, 1501], [0, 0], 8, 2, 128, 64, 128, True, True, True, True, 0),
}


def _append(name, bits, seed=0):
    B, lens, first, Hq, Hkv, d, page, rot, il, norm, with_q, fused, pad = APPENDS[name]
    g = _gen(seed + len(name))
    T = sum(lens) + pad
    x = _randn(g, T, Hq + 2 * Hkv, d)
    Q, K, V = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if not fused:
        Q, K, V = Q.contiguous(), K.contiguous(), V.contiguous()
    table, pool = _table(g, [f + n for f, n in zip(first, lens)], page)
    shape = pisa.make_paged_shape(B, Hq, Hkv, d, pool, page, table.shape[1], bits)
    cache = _filled(g, shape)
    seq = [b for b, n in enumerate(lens) for _ in range(n)] + [-1] * pad
    pos = [f + i for f, n in zip(first, lens) for i in range(n)] + [-5] * pad
    inv, _ = pisa.rope_frequencies(rot) if rot else (None, 1.0)
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") if norm else None for _ in range(2))
    rope = pisa.Rope(inv.cuda() if rot else None, rot, il, norm, 1e-6, 1.0, wq, wk)
    return shape, cache, table, seq, pos, Q if with_q else None, K, V, rope


def _slots(table, seq, pos, page):
    s, p = torch.tensor(seq, device="cuda"), torch.tensor(pos, device="cuda")
    return table[s, p // page].long(), p % page


@pytest.mark.parametrize("name", APPENDS)
def test_append_in_16_bits_is_the_norm_and_rotation_put_into_slots(name):
    shape, cache, table, seq, pos, Q, K, V, rope = _append(name, 16)
    n = sum(s >= 0 for s in seq)
    want_k, want_v = cache.k.clone(), cache.v.clone()
    s = pisa.rope_shape_of((Q if Q is not None else K)[None, :n], K[None, :n], rope.rot, rope.interleaved, rope.norm, rope.eps)
    Qr, Kr = pisa.qk_norm_rope((Q if Q is not None else K)[None, :n], K[None, :n], rope.inv_freq, s, rope.q_weight, rope.k_weight,
                               _ints(pos[:n])[None])
    page, slot = _slots(table, seq[:n], pos[:n], shape.page)
    want_k[page, :, slot], want_v[page, :, slot] = Kr[0], V[:n]
    q_out = None if Q is None else torch.full(Q.shape, 7.0, dtype=bf16, device="cuda")
    got, status = pisa.paged_append(shape, cache, table, _ints(pos), K, V, Q=Q, seq=_ints(seq), rope=rope, q_out=q_out)
    assert int(status[0]) == 0
    assert torch.equal(cache.k, want_k) and torch.equal(cache.v, want_v)
    if Q is not None:
        assert torch.equal(got[:n], Qr[0])
        assert bool((got[n:] == 7.0).all())                            # padding's rows stay as they were


@pytest.mark.parametrize("name", APPENDS)
def test_append_in_4_bits_holds_the_codes_of_the_same_keys(name):
    shape16, c16, table16, seq, pos, Q, K, V, rope = _append(name, 16)
    shape, cache, table, _, _, _, _, _, _ = _append(name, 4)
    n = sum(s >= 0 for s in seq)
    pisa.paged_append(shape16, c16, table16, _ints(pos), K, V, Q=Q, seq=_ints(seq), rope=rope)
    before = [t.clone() for t in cache[:4]]
    _, status = pisa.paged_append(shape, cache, table, _ints(pos), K, V, Q=Q, seq=_ints(seq), rope=rope)
    assert int(status[0]) == 0
    p16, p4 = _slots(table16, seq[:n], pos[:n], shape.page), _slots(table, seq[:n], pos[:n], shape.page)
    for k, sc, amp, src, old, old_s in ((cache.k, cache.k_scale, cache.k_amp, c16.k, before[0], before[2]),
                                        (cache.v, cache.v_scale, cache.v_amp, c16.v, before[1], before[3])):
        x = src[p16[0], :, p16[1]].float() / amp[:, None]              # the quotient is rounded to fp32 by definition
        codes, scales = quantise(x.double())
        assert torch.equal(sc[p4[0], :, p4[1]].double(), scales)
        assert torch.equal(codes_of(k[p4[0], :, p4[1]]), codes)
        rest = torch.ones(shape.n_pages, shape.page, dtype=torch.bool, device="cuda")
        rest[p4[0], p4[1]] = False
        keep = rest[:, None, :, None].expand(-1, shape.Hkv, -1, 1)[..., 0]
        assert torch.equal(k[keep], old[keep]) and torch.equal(sc.view(torch.uint8)[keep], old_s.view(torch.uint8)[keep])


def test_codes_at_ties_and_extremes():
    # group by group: every tie, the scale's own ties and ends, zeros, tiny and huge values, infinities and NaN
    rows = [[6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6],
            [0.0] * 16, [-0.0] * 16, [2688.0] + [1344.0] * 15, [60000.0] + [2688.0, 5.0] * 7 + [0.0], [2.0 ** -12] * 16,
            [6 * 2.0 ** -9, 2.0 ** -9] * 8, [6 * 2.0 ** -10, 2.0 ** -11] * 8, [6 * 2.0 ** -10 * 1.5] + [2.0 ** -9] * 15,
            [math.inf] + [1.0] * 15, [1.0] * 15 + [math.nan], [-math.inf, math.nan] * 8, [6.375] + [1.0625] * 15, [6.75, 1.125] * 8,
            [1e38] * 16, [1e-40] * 16]
    V = torch.tensor(rows, device="cuda").reshape(len(rows) // 4, 1, 64).to(bf16)
    T = V.shape[0]
    shape = pisa.make_paged_shape(1, 1, 1, 64, 1, 16, 1, bits=4)
    cache = pisa.paged_cache(shape, "cuda")
    pisa.paged_append(shape, cache, _ints([[0]]), _ints(list(range(T))), torch.zeros_like(V), V)
    codes, scales = quantise(V[:, 0].double())
    got, got_s = codes_of(cache.v[0, 0, :T]), cache.v_scale[0, 0, :T].double()
    assert torch.equal(got_s.isnan(), scales.isnan()) and torch.equal(got_s.nan_to_num(), scales.nan_to_num())
    fine = ~scales.isnan().repeat_interleave(16, -1)
    assert torch.equal(got[fine], codes[fine])
    assert bool((values_of(cache.v, cache.v_scale)[0, 0, :T][~fine]).isnan().all())


@pytest.mark.parametrize("bits", [16, 4])
def test_append_without_seq_and_queries_in_place(bits):
    g = _gen(11)
    B, n, Hq, Hkv, d, page = 3, 4, 4, 2, 128, 16
    table, pool = _table(g, [40] * B, page)
    shape = pisa.make_paged_shape(B, Hq, Hkv, d, pool, page, table.shape[1], bits)
    a, b = pisa.paged_cache(shape, "cuda"), pisa.paged_cache(shape, "cuda")
    Q, K, V = _randn(g, B * n, Hq, d), _randn(g, B * n, Hkv, d), _randn(g, B * n, Hkv, d)
    pos = _ints([30 + i for _ in range(B) for i in range(n)])
    rope = pisa.Rope(pisa.rope_frequencies(d)[0].cuda(), d)
    q1, _ = pisa.paged_append(shape, a, table, pos, K, V, Q=Q, seq=_ints([x for x in range(B) for _ in range(n)]), rope=rope)
    Q2 = Q.clone()
    q2, _ = pisa.paged_append(shape, b, table, pos, K, V, Q=Q2, rope=rope, q_out=Q2)
    assert q2 is Q2 and torch.equal(q1, q2)
    for x, y in zip(a[:4], b[:4]):
        assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("bits", [16, 4])
def test_tokens_out_of_range_are_skipped_and_reported(bits):
    g = _gen(12)
    shape = pisa.make_paged_shape(2, 4, 2, 64, 4, 16, 3, bits)
    cache = _filled(g, shape)
    table = _ints([[0, -1, 4], [2, 3, 1]])
    seq, pos = [0, 0, 0, 1, 1, 1, 2, -1, 1], [3, 20, 40, -1, 48, 17, 0, 5, 1 << 30]
    good = [0, 5]
    K, V, Q = _randn(g, 9, 2, 64), _randn(g, 9, 2, 64), _randn(g, 9, 4, 64)
    before = [None if t is None else t.clone() for t in cache[:4]]
    q_out = torch.full_like(Q, 7.0)
    rope = pisa.Rope(None, 0)
    status = _ints([0, 0, 0, 0])
    pisa.paged_append(shape, cache, table, _ints(pos), K, V, Q=Q, seq=_ints(seq), rope=rope, q_out=q_out, status=status)
    assert int(status[0]) == pisa.STATUS_POS_RANGE
    left = [t for t in range(9) if t not in good]
    assert bool((q_out[left] == 7.0).all()) and not bool((q_out[good] == 7.0).any())
    same = torch.ones(4, 16, dtype=torch.bool, device="cuda")
    same[0, 3] = same[3, 1] = False
    keep = same[:, None].expand(-1, 2, -1)
    for t, old in zip(cache[:4], before):
        if t is not None:
            assert torch.equal(t.view(torch.uint8)[keep], old.view(torch.uint8)[keep])
            assert not torch.equal(t.view(torch.uint8)[~keep], old.view(torch.uint8)[~keep])


# --------------------------------------------------------------------------------- run together
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("cap,biased", [(0.0, False), (8.0, True)])
def test_prompts_then_steps(bits, cap, biased):
    """A serving run: packed prompts through norm, rotation and the documents' attention, their keys into pages, then decode
    steps captured in a graph whose positions advance on the device."""
    g = _gen(20)
    lens, Hq, Hkv, d, page, steps = [70, 33, 128], 8, 2, 128, 16, 5
    B, T = len(lens), sum(lens)
    x = _randn(g, T, Hq + 2 * Hkv, d)
    Q, K, V = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    rope = pisa.Rope(pisa.rope_frequencies(d)[0].cuda(), d, q_weight=torch.ones(d, device="cuda"), k_weight=torch.ones(d, device="cuda"))
    slopes = _slopes(Hq) if biased else None
    table, pool = _table(g, [n + steps for n in lens], page)
    shape = pisa.make_paged_shape(B, Hq, Hkv, d, pool, page, table.shape[1], bits, cap=cap)
    cache = pisa.paged_cache(shape, "cuda")
    seq = [b for b, n in enumerate(lens) for _ in range(n)]
    pos = [i for n in lens for i in range(n)]
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    # prompts: the queries come back from the append, the rotated keys from the norm and rotation
    s = pisa.rope_shape_of(Q[None], K[None], d)
    Qr, Kr = pisa.qk_norm_rope(Q[None], K[None], rope.inv_freq, s, rope.q_weight, rope.k_weight, _ints(pos)[None])
    q2, status = pisa.paged_append(shape, cache, table, _ints(pos), K, V, Q=Q, seq=_ints(seq), rope=rope)
    assert torch.equal(q2, Qr[0])
    ds = pisa.doc_shape_of(Qr[0], Kr[0], V, _ints(starts), cap=cap)
    O, lse = pisa.doc_attn_fwd(Qr[0], Kr[0], V, _ints(starts), ds, slopes=slopes)
    want, tol = doc_attention(Qr[0], Kr[0], V, starts, None, slopes, cap)
    check("O", O, want["O"], tol["O"])
    # the prompts' last rows are what a decode step over the pages gives
    last = [e - 1 for e in starts[1:]]
    o, l1 = pisa.paged_attn(shape, cache, table, _ints(lens), Qr[0][last][:, None].contiguous(), slopes)
    if bits == 16:
        check("o", o[:, 0], want["O"][last], tol["O"][last])
        check("lse", l1[:, 0], want["lse"].T[last], tol["lse"].T[last])
    # steps
    new = _randn(g, steps, B, Hq + 2 * Hkv, d)
    now, at, length = new[0].clone(), _ints(lens), _ints([n + 1 for n in lens])
    ws = pisa.paged_workspace(shape, "cuda")

    def step():
        q, _ = pisa.paged_append(shape, cache, table, at, now[:, Hq:Hq + Hkv], now[:, Hq + Hkv:], Q=now[:, :Hq], rope=rope, status=status)
        o, lse = pisa.paged_attn(shape, cache, table, length, q[:, None], slopes, ws=ws)
        at.add_(1)
        length.add_(1)
        return q, o, lse

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    at.copy_(_ints(lens))
    length.copy_(_ints([n + 1 for n in lens]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, o, lse = step()
    for t in range(steps):
        now.copy_(new[t])
        graph.replay()
        n = [x + t + 1 for x in lens]
        k, v = _keys(cache, table, n, page)
        want, tol = paged_attention(q[:, None], k, v, n, slopes, cap)
        check("o", o, want["O"], tol["O"])
        check("lse", lse, want["lse"], tol["lse"])
    assert int(status[0]) == 0 and pisa.workspace_status(ws) == 0


def test_4_bit_values_are_near_the_16_bit_ones():
    # a code is within half the widest gap (1 of 6) of the group's largest magnitude, and the scale within 1 / 16 of itself
    g = _gen(21)
    shape = pisa.make_paged_shape(1, 4, 4, 128, 8, 64, 8, bits=4)
    cache = pisa.paged_cache(shape, "cuda", k_amp=torch.full((4,), 0.3, device="cuda"))
    K, V = _randn(g, 500, 4, 128), _randn(g, 500, 4, 128, scale=0.05)
    pisa.paged_append(shape, cache, _ints([list(range(8))]), _ints(list(range(500))), K, V)
    k, v = _keys(cache, _ints([list(range(8))]), [500], 64)
    for got, x in ((k[0], K), (v[0], V)):
        top = x.double().reshape(500, 4, 8, 16).abs().amax(-1, keepdim=True)
        off = (got - x.double()).reshape(500, 4, 8, 16).abs()
        assert bool((off <= top * (1 / 6) * (1 + 2.0 ** -4) + 2.0 ** -9).all())


@pytest.mark.parametrize("bits", [16, 4])
def test_pages_past_32_bits(bits):
    # pages whose bytes (and, in 16 bits, elements) lie past 2^32 (2^31): the same as in a small cache, to the bit
    g = _gen(22)
    Hq, Hkv, d, page = 8, 4, 128, 1024
    row = d * 2 if bits == 16 else d // 2
    pool = (9 << 29) // (Hkv * page * row)                               # 4.5 GiB of codes or values
    lens = [3000, 1500]
    small = pisa.make_paged_shape(2, Hq, Hkv, d, 5, page, 3, bits)
    large = pisa.make_paged_shape(2, Hq, Hkv, d, pool, page, 3, bits)
    few = _filled(g, small)
    ids = torch.tensor([pool - 1, 0, pool - 2, pool // 2, pool - 5], device="cuda")
    many = []
    for x in few[:4]:
        if x is None:
            many.append(None)
            continue
        y = torch.empty(pool, *x.shape[1:], dtype=x.dtype, device="cuda")
        y.view(torch.uint8)[ids] = x.view(torch.uint8)
        many.append(y)
    many = pisa.PagedCache(*many, *few[4:])
    t0 = torch.tensor([[0, 1, 2], [3, 4, 0]], device="cuda")
    t1 = ids[t0].to(torch.int32)
    t0 = t0.to(torch.int32)
    K, V, Q = _randn(g, 100, Hkv, d), _randn(g, 100, Hkv, d), _randn(g, 100, Hq, d)
    seq = _ints([0] * 60 + [1] * 40)
    pos = _ints(list(range(2940, 3000)) + list(range(1460, 1500)))
    rope = pisa.Rope(pisa.rope_frequencies(d)[0].cuda(), d, norm=False)
    q = _randn(g, 2, 1, Hq, d)
    outs = []
    for shape, cache, table in ((small, few, t0), (large, many, t1)):
        Qr, status = pisa.paged_append(shape, cache, table, pos, K, V, Q=Q, seq=seq, rope=rope)
        assert int(status[0]) == 0
        outs.append((Qr, *pisa.paged_attn(shape, cache, table, _ints(lens), q)))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    for x, y in zip(few[:4], many[:4]):
        assert x is None or torch.equal(y.view(torch.uint8)[ids], x.view(torch.uint8))


@pytest.mark.parametrize("bits", [16, 4])
def test_two_graphs_share_a_workspace(bits):
    g = _gen(23)
    page = 16
    lens = [[700, 30, 0, 5], [1, 650, 64, 222]]
    table, pool = _table(g, [700, 650, 64, 222], page)
    shape = pisa.make_paged_shape(4, 16, 2, 128, pool, page, table.shape[1], bits, 2)
    cache = _filled(g, shape)
    q, ws = _randn(g, 4, 2, 16, 128), pisa.paged_workspace(shape, "cuda")
    lens = [_ints(n) for n in lens]
    want = [[t.clone() for t in pisa.paged_attn(shape, cache, table, n, q, ws=ws)] for n in lens]
    graphs, got = [torch.cuda.CUDAGraph() for _ in lens], []
    for graph, n in zip(graphs, lens):
        with torch.cuda.graph(graph):
            got.append(pisa.paged_attn(shape, cache, table, n, q, ws=ws))
    for k in (0, 1, 1, 0, 1):
        for t in got[k]:
            t.zero_()
        graphs[k].replay()
        torch.cuda.synchronize()
        for a, b in zip(got[k], want[k]):
            assert torch.equal(a, b)
    # and at once on streams of their own, with workspaces of their own
    streams, out = [torch.cuda.Stream() for _ in lens], []
    for st, n in zip(streams, lens):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            out.append(pisa.paged_attn(shape, cache, table, n, q))
    torch.cuda.synchronize()
    for x, y in zip(out, want):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("bits", [16, 4])
def test_captured_behind_two_streams(bits):
    # the calls' inputs come from two streams that meet right before them, in a graph and outside
    g = _gen(24)
    B, Hq, Hkv, d, page, n = 3, 8, 2, 128, 16, 90
    table, pool = _table(g, [n + 1] * B, page)
    shape = pisa.make_paged_shape(B, Hq, Hkv, d, pool, page, table.shape[1], bits)
    cache = _filled(g, shape)
    K, V, Q = (_randn(g, B, h, d) for h in (Hkv, Hkv, Hq))
    pos, lens = _ints([n] * B), _ints([n + 1] * B)
    rope = pisa.Rope(pisa.rope_frequencies(d)[0].cuda(), d, norm=False)
    starts = _ints([0, 2, 3])
    out = [torch.empty(B, Hq, d, dtype=bf16, device="cuda"), torch.empty(B, 1, Hq, d, dtype=bf16, device="cuda"),
           torch.empty(B, Hq, d, dtype=bf16, device="cuda")]
    status, ws = _ints([0, 0, 0, 0]), pisa.paged_workspace(shape, "cuda")
    lse, dlse = torch.empty(B, 1, Hq, device="cuda"), torch.empty(Hq, B, device="cuda")
    k, v, q = (torch.empty_like(x) for x in (K, V, Q))
    other = torch.cuda.Stream()

    def meet(work):
        here = torch.cuda.current_stream()
        other.wait_stream(here)
        with torch.cuda.stream(other):
            k.copy_(K * 1)
            v.copy_(V * 1)
        q.copy_(Q * 1)
        here.wait_stream(other)
        work()

    def run():
        meet(lambda: pisa.paged_append(shape, cache, table, pos, k, v, Q=q, rope=rope, q_out=out[0], status=status))
        meet(lambda: pisa.paged_attn(shape, cache, table, lens, out[0][:, None], ws=ws, o=out[1], lse=lse))
        meet(lambda: pisa.doc_attn_fwd(q, k, v, starts, pisa.doc_shape_of(q, k, v, starts), out=out[2], lse=dlse))

    run()
    torch.cuda.synchronize()
    want = [t.clone() for t in (*out, lse, dlse)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for t in (k, v, q, *out, lse, dlse):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*out, lse, dlse), want):
            assert torch.equal(a, b)
    assert int(status[0]) == 0 and pisa.workspace_status(ws) == 0


# ------------------------------------------------------------------- visible values that are not finite
SPREADS = {  # B, nq, Hq, Hkv, d, lens: a unit over all CTAs, units over several, more units than CTAs with one over several
    "one sequence": (1, 1, 8, 1, 128, [9000]),
    "a few": (6, 2, 8, 2, 64, [3000, 10, 0, 700, 1234, 5]),
    "sixteen rows": (2, 4, 8, 2, 128, [4000, 900]),
    "many": (130, 1, 8, 4, 64, [20000] + [(97 * b) % 500 for b in range(1, 130)]),
    "within a CTA": (300, 1, 8, 4, 64, [60] * 300),
}


def _spread_case(name, bits, seed):
    B, nq, Hq, Hkv, d, lens = SPREADS[name]
    g, page = _gen(seed), 16
    table, pool = _table(g, lens, page)
    shape = pisa.make_paged_shape(B, Hq, Hkv, d, pool, page, table.shape[1], bits, nq)
    return g, shape, _filled(g, shape), table, lens, _randn(g, B, nq, Hq, d)


def _put(shape, cache, table, seq, pos, K, V):
    """Tokens of sequence seq written over those at pos."""
    _, status = pisa.paged_append(shape, cache, table, _ints(pos), K, V, seq=_ints([seq] * len(pos)))
    assert int(status[0]) == 0


def _same(a, b):
    return torch.equal(a.nan_to_num(nan=9e9), b.nan_to_num(nan=9e9)) and torch.equal(a.isnan(), b.isnan())


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("name", SPREADS)
def test_a_query_with_a_nan_gives_nan(name, bits):
    g, shape, cache, table, lens, q = _spread_case(name, bits, 30)
    o0, lse0 = pisa.paged_attn(shape, cache, table, _ints(lens), q)
    q[0, 0, 1, 5] = math.nan
    o, lse = pisa.paged_attn(shape, cache, table, _ints(lens), q)
    o0[0, 0, 1], lse0[0, 0, 1] = math.nan, math.nan
    assert _same(o, o0) and _same(lse, lse0)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("name", SPREADS)
def test_keys_of_nan_give_nan(name, bits):
    # a third of a sequence's keys, or two CTAs' part of a long one, in one KV head: parts of a unit see nothing else
    g, shape, cache, table, lens, q = _spread_case(name, bits, 31)
    o0, lse0 = pisa.paged_attn(shape, cache, table, _ints(lens), q)
    n = lens[0]
    pos = list(range(n // 3, 2 * n // 3)) if n != 9000 else list(range(2560, 2688))
    k, v = ([x[0][pos] for x in _keys(cache, table, lens[:1], shape.page)])
    if bits == 16:
        k[:, 0] = math.nan
        _put(shape, cache, table, 0, pos, k.to(bf16), v.to(bf16))
    else:                                                              # (the codes of the others stay as they are)
        page, slot = _slots(table, [0] * len(pos), pos, shape.page)
        cache.k_scale.view(torch.uint8)[page, 0, slot] = 0x7f
    o, lse = pisa.paged_attn(shape, cache, table, _ints(lens), q)
    G = shape.Hq // shape.Hkv
    o0[0, :, :G], lse0[0, :, :G] = math.nan, math.nan
    assert _same(o, o0) and _same(lse, lse0)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("name", SPREADS)
def test_a_value_of_nan_reaches_its_channels_however_small_its_weight(name, bits):
    # the first key has all the weight: the others' parts are taken times factors that underflow
    g, shape, cache, table, lens, q = _spread_case(name, bits, 32)
    n, d = lens[0], shape.d
    q[0] = q[0, :1, :1].clone()
    V = _randn(g, 1, shape.Hkv, d)
    _put(shape, cache, table, 0, [0], (40 * q[0, :1, :1]).expand(1, shape.Hkv, d).contiguous(), V)
    low, bad = (-40 * q[0, :1, :1]).expand(1, shape.Hkv, d).contiguous(), V.clone()
    bad[..., 16:32] = math.nan
    for p in range(n // 9, n - n // 9, n // 9):
        _put(shape, cache, table, 0, [p], low, V)
        o0, lse0 = pisa.paged_attn(shape, cache, table, _ints(lens), q)
        assert bool(torch.isfinite(o0).all())
        _put(shape, cache, table, 0, [p], low, bad)
        o, lse = pisa.paged_attn(shape, cache, table, _ints(lens), q)
        o0[0, ..., 16:32] = math.nan
        assert _same(o, o0) and _same(lse, lse0)
        _put(shape, cache, table, 0, [p], low, V)


@pytest.mark.parametrize("cap,biased", [(0.0, False), (4.0, True)])
@pytest.mark.parametrize("amp", [1e-8, 1e-19, 2.0 ** -64])
def test_queries_of_zeros_with_small_factors(amp, cap, biased):
    # what a score is multiplied by may leave 32 bits: a query of zeros, or of tiny values, has equal weights all the same
    g = _gen(33)
    lens, page = [33, 1, 70, 4001], 16
    table, pool = _table(g, lens, page)
    shape = pisa.make_paged_shape(4, 8, 2, 64, pool, page, table.shape[1], 4, cap=cap)
    cache = _filled(g, shape)
    cache = cache._replace(k_amp=torch.tensor([amp, 0.7], device="cuda"))
    q = _randn(g, 4, 1, 8, 64)
    q[:, :, ::2] = 0
    q[:, :, 1] *= 2.0 ** -100
    slopes = _slopes(8) if biased else None
    o, lse = pisa.paged_attn(shape, cache, table, _ints(lens), q, slopes)
    k, v = _keys(cache, table, lens, page)
    want, tol = paged_attention(q, k, v, lens, slopes, cap)
    check("o", o, want["O"], tol["O"])
    check("lse", lse, want["lse"], tol["lse"])


@pytest.mark.parametrize("amp", [0.1, 1.0 / 3, 1e-3, 3e-12, 2.0 ** -64, 7e8, 2.0 ** 64])
def test_codes_of_extremes_over_a_factor(amp):
    # quotients past the largest code and scale, and past 32 bits: the scale stays 448, the codes 6, their signs what they were
    rows = [[1e38] * 16, [-1e38, 1e38] * 8, [3.38e38, 1.0] * 8, [-3.38e38] + [0.0] * 15, [2688.0 * amp] * 16, [-5376.0 * amp, amp] * 8,
            [4096.0 * amp, 4097.0 * amp] * 8, [amp, -2 * amp] * 8, [1e30, -1e-30] * 8, [1e-30] * 16, [-0.0, 0.0] * 8, [1e-40] * 16,
            [math.inf, 1e38] * 8, [math.nan, 1e38] * 8, [6 * amp, 0.25 * amp] * 8, [1e38, -2.0 ** -100] * 8]
    X = torch.tensor(rows, dtype=torch.float64, device="cuda").reshape(len(rows) // 4, 1, 64).to(bf16)
    T = X.shape[0]
    shape = pisa.make_paged_shape(1, 1, 1, 64, 1, 16, 1, bits=4)
    factor = torch.tensor([amp], device="cuda")
    cache = pisa.paged_cache(shape, "cuda", factor, factor)
    pisa.paged_append(shape, cache, _ints([[0]]), _ints(list(range(T))), X, X)
    x = X[:, 0].double() / factor.double()
    near = x.float().double()                                          # the quotient in 32 bits, where it has a place there
    codes, scales = quantise(torch.where(torch.isfinite(X[:, 0]) & torch.isinf(near), x, near))
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        got, got_s = codes_of(t[0, 0, :T]), s[0, 0, :T].double()
        assert torch.equal(got_s.isnan(), scales.isnan()) and torch.equal(got_s.nan_to_num(), scales.nan_to_num())
        fine = ~scales.isnan().repeat_interleave(16, -1)
        assert torch.equal(got[fine], codes[fine])


# -------------------------------------------------------------------------------------- many of everything
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("name", ["many", "many, sixteen rows", "equal", "equal, sixteen rows", "a thousand", "rows in sets", "rows in sets, drafts"])
def test_attention_of_many(name, bits):
    # more units than CTAs (a unit that crosses into the next CTA is found by its place), units that end where a CTA's run does, more
    # sequences than a few look-ups, and rows in several sets of 16
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    mixed = [30000] + [(b * b * 131) % 2001 for b in range(1, 129)] + [3000]
    B, nq, Hq, Hkv, d, page, lens = {
        "many": (130, 1, 8, 4, 64, 16, mixed), "many, sixteen rows": (130, 4, 12, 4, 128, 64, mixed),
        "equal": (3 * sms // 2, 1, 4, 4, 128, 64, [320] * (3 * sms // 2)),
        "equal, sixteen rows": (3 * sms // 2, 4, 12, 4, 64, 32, [160] * (3 * sms // 2)),
        "a thousand": (1003, 1, 2, 1, 64, 16, [(b * b * 17) % 301 for b in range(1003)]),
        "rows in sets": (3, 1, 48, 1, 128, 64, [5000, 2000, 17]), "rows in sets, drafts": (2, 16, 64, 1, 64, 16, [3000, 40]),
    }[name]
    g = _gen(40 + len(name))
    table, pool = _table(g, lens, page)
    shape = pisa.make_paged_shape(B, Hq, Hkv, d, pool, page, table.shape[1], bits, nq)
    cache = _filled(g, shape)
    q = _randn(g, B, nq, Hq, d)
    ws = pisa.paged_workspace(shape, "cuda")
    ws.fill_(0xAB)
    o, lse = torch.full_like(q, 7.0), torch.full((B, nq, Hq), 7.0, device="cuda")
    pisa.paged_attn(shape, cache, table, _ints(lens), q, ws=ws, o=o, lse=lse)
    assert pisa.workspace_status(ws) == 0
    k, v = _keys(cache, table, lens, page)
    want, tol = paged_attention(q, k, v, lens)
    check("o", o, want["O"], tol["O"])
    check("lse", lse, want["lse"], tol["lse"])


@pytest.mark.parametrize("bits", [16, 4])
def test_append_of_more_tokens_than_one_look_up(bits):
    # every warp looks 32 units up at a time: some 117K tokens on 152 SMs, here more, and behind those padding, tokens out of
    # range and pages that are none
    g = _gen(41)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B, Hq, Hkv, d, page = 3, 1, 1, 64, 128
    T = sms * 24 * 32 + 33333
    n = T // B
    lens = [n, n, T - 2 * n]
    table, pool = _table(g, lens, page)
    table[2, 30] = pool
    shape = pisa.make_paged_shape(B, Hq, Hkv, d, pool, page, table.shape[1], bits)
    cache = _filled(g, shape)
    x = _randn(g, T, Hq + 2 * Hkv, d)
    Q, K, V = x[:, :1], x[:, 1:2], x[:, 2:]
    seq = torch.arange(B, device="cuda").repeat_interleave(torch.tensor(lens, device="cuda"))
    pos = torch.cat([torch.arange(m, device="cuda") for m in lens])
    late = torch.arange(T, device="cuda") > T - 20000
    skip = late & (torch.randint(0, 4, (T,), generator=g, device="cuda") == 0)
    off = late & ~skip & (torch.randint(0, 5, (T,), generator=g, device="cuda") == 0)
    none = (seq == 2) & (pos // page == 30)
    inv = pisa.rope_frequencies(d)[0].cuda()
    rope = pisa.Rope(inv, d, q_weight=1 + 0.1 * torch.randn(d, generator=g, device="cuda"), k_weight=torch.ones(d, device="cuda"))
    s = pisa.rope_shape_of(Q[None], K[None], d)
    Qr, Kr = pisa.qk_norm_rope(Q[None], K[None], inv, s, rope.q_weight, rope.k_weight, pos.to(torch.int32)[None])
    before = [None if t is None else t.clone() for t in cache[:4]]
    given = torch.where(off, pos + (1 << 24), pos)
    q_out = torch.full(Q.shape, 7.0, dtype=bf16, device="cuda")
    got, status = pisa.paged_append(shape, cache, table, given.to(torch.int32), K, V, Q=Q, seq=torch.where(skip, -1, seq).to(torch.int32),
                                    rope=rope, q_out=q_out)
    assert int(status[0]) == pisa.STATUS_POS_RANGE
    kept = ~(skip | off | none)
    assert bool((got[~kept] == 7.0).all()) and torch.equal(got[kept], Qr[0][kept])
    page_of, slot = table[seq[kept], pos[kept] // page].long(), pos[kept] % page
    for t, sc, amp, src, old, old_s in ((cache.k, cache.k_scale, cache.k_amp, Kr[0], before[0], before[2]),
                                        (cache.v, cache.v_scale, cache.v_amp, V, before[1], before[3])):
        if bits == 16:
            old[page_of, :, slot] = src[kept]
            assert torch.equal(t, old)
            continue
        codes, scales = quantise((src[kept].float() / amp[:, None]).double())
        c = codes.to(torch.uint8).reshape(*codes.shape[:2], -1, 2)
        old[page_of, :, slot] = c[..., 0] | c[..., 1] << 4
        old_s.view(torch.uint8)[page_of, :, slot] = scales.float().to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(t, old) and torch.equal(sc.view(torch.uint8), old_s.view(torch.uint8))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("B,nq,Hq,Hkv,d,page", [(5, 4, 8, 2, 128, 16), (4, 16, 4, 2, 64, 32), (3, 2, 12, 2, 64, 16), (2, 9, 8, 2, 128, 64), (60, 3, 20, 4, 128, 16)])
def test_drafted_tokens_that_are_not_finite_reach_the_queries_that_see_them(B, nq, Hq, Hkv, d, page, bits):
    g = _gen(34 + nq)
    lens = [(700, 33, nq, 48 + nq, 2)[b % 5] + b for b in range(B)]
    table, pool = _table(g, lens, page)
    shape = pisa.make_paged_shape(B, Hq, Hkv, d, pool, page, table.shape[1], bits, nq)
    cache = _filled(g, shape)
    q = _randn(g, B, nq, Hq, d)
    k, v = _keys(cache, table, lens, page)
    want, tol = paged_attention(q, k, v, lens)                         # (what is reached is left out of the comparison)
    reached = torch.zeros(B, nq, Hq, d, dtype=torch.bool, device="cuda")
    lost = torch.zeros(B, nq, Hq, dtype=torch.bool, device="cuda")
    G = Hq // Hkv
    for b, n in enumerate(lens):
        for back in range(min(n, nq)):
            if (b + back) % 3 == 2:
                continue
            p, kv, c = n - 1 - back, (b + back) % Hkv, (5 * b + 11 * back) % d
            pg, slot = table[b, p // page].long(), p % page
            sees = torch.arange(nq, device="cuda") >= nq - 1 - back
            if (b + back) % 4 == 3:                                    # a key: every query that sees it
                if bits == 16:
                    cache.k[pg, kv, slot, c] = math.nan
                else:
                    cache.k_scale.view(torch.uint8)[pg, kv, slot, c // 16] = 0x7f
                lost[b, :, kv * G:(kv + 1) * G] |= sees[:, None]
            elif bits == 16:
                cache.v[pg, kv, slot, c] = (math.inf, -math.inf, math.nan)[back % 3]
                reached[b, :, kv * G:(kv + 1) * G, c] |= sees[:, None]
            else:
                cache.v_scale.view(torch.uint8)[pg, kv, slot, c // 16] = 0x7f if back % 2 else 0xff
                reached[b, :, kv * G:(kv + 1) * G, c // 16 * 16:c // 16 * 16 + 16] |= sees[:, None, None]
    o, lse = pisa.paged_attn(shape, cache, table, _ints(lens), q)
    reached |= lost[..., None]
    assert torch.equal(~o.isfinite(), reached) and torch.equal(lse.isnan(), lost)
    check("o", torch.where(reached, want["O"], o.double()), want["O"], tol["O"])
    check("lse", torch.where(lost, want["lse"], lse.double()), want["lse"], tol["lse"])
