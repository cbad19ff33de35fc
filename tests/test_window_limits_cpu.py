"""Limits of the window attention and of the query/key norm without a GPU: sizes of workspaces,
refusals of calls that would read or write the wrong memory."""
import random

import pytest

import pyramid_top_selection_gb300 as pisa

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
