"""Workspaces made for the largest call fit every smaller one: their sizes never fall as a call grows."""
import itertools
import os

import pytest

import lossless_bit_weight_w12_amd as w12

BEAM_N = [1, 2, 3, 4, 8, 13, 25, 26, 27, 28, 52, 53, 54, 55, 96, 107, 108, 512, 1023, 1024, 1025, 4096]
BEAM_VOCAB = [64, 4096, 4097, 8192, 8193, 16384, 16385, 50257, 128259, 151936, 1 << 19, (1 << 19) + 1, 1 << 20, 1 << 21]
BEAM_K = [1, 2, 8, 15, 16, 17, 18, 32, 33, 63, 64]


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(w12.lib_path()):
        from lossless_bit_weight_w12_amd import build
        build.build()
    return w12.lib()


def grows(size, *axes):
    """Pairs of neighbours along an axis where size falls."""
    falls = []
    for at in itertools.product(*(range(len(a)) for a in axes)):
        for i, a in enumerate(axes):
            if at[i] + 1 < len(a):
                here = [x[j] for x, j in zip(axes, at)]
                more = list(here)
                more[i] = a[at[i] + 1]
                if size(*more) < size(*here):
                    falls.append((here, more))
    return falls


def test_beam_workspace_never_falls(L):
    assert grows(L.w12_beam_ws_bytes, BEAM_N, BEAM_VOCAB, BEAM_K) == []
    assert L.w12_beam_ws_bytes(0, 1, 1) == 16384


def test_beam_workspace_holds_the_parts(L):
    """A maximum, a sum and k pairs per row and part, for each share that the call may take."""
    for n, vocab, k in itertools.product(BEAM_N, BEAM_VOCAB, BEAM_K):
        values = 64 if k > 16 or vocab > 1 << 19 else next(
            (v for v in (16, 32) if n * -(-vocab // (256 * v)) <= 1024), 64)
        assert L.w12_beam_ws_bytes(n, vocab, k) >= 16384 + n * -(-vocab // (256 * values)) * (16 + 8 * k)


def test_shared_attention_workspace_never_falls(L):
    f = lambda d, m, n: L.w12_attn_shared_ws_bytes(m, n, d)
    assert grows(f, [64, 128, 256], [0, 1, 4, 10, 11, 42, 43, 44, 96, 128], [1, 2, 8, 40, 128, 1023, 1024]) == []
    assert f(256, 4, 8) >= f(128, 4, 8) > f(64, 4, 8) > 0
