"""Block-cache prefills on values at the ends of their ranges: V blocks of zeros or of far smaller scales, scores that
vanish beside masked ones, scales far out of range whose products are not, windows up to the largest."""

import numpy as np
import pytest

from grouped_query_attention_gb300 import capi
from test_gpu_block_cache import NP, check, make, regime, run_gpu

pytestmark = pytest.mark.gpu

# One query tile (128 rows a KV head) and several; eight 16-token blocks.
TILES = {"one_tile": (8, 16), "two_tiles": (60, 16)}


@pytest.mark.parametrize("softcap", [0.0, 5.0])
@pytest.mark.parametrize("tiles", list(TILES))
@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("which", ["one_zero", "seven_zero", "far_apart", "near_border"])
def test_value_blocks_of_far_smaller_scales(dtype, which, tiles, softcap):
    """Their probabilities stay in the denominator, whatever of them the product with V can hold."""
    S, G = TILES[tiles]
    d = make((dtype, 2, S, 4 * G, 4, 128, 128, 16, (128, 125), None, -1, softcap, 0, 1, 0), seed=70)
    d["cache"][2][:] = 0.01          # equal K scales: no block is without weight
    vs = d["cache"][3]
    vs[:] = 0.02
    if which == "one_zero":
        vs[:, :, 3] = 0
    elif which == "seven_zero":
        vs[:, :, [0, 1, 2, 4, 5, 6, 7]] = 0
    elif which == "far_apart":
        vs[:, :, ::2] *= np.float32(2.0 ** -35)
    else:                            # about where fp16 probabilities run out of bits
        vs *= np.float32(2.0) ** -np.array([0, 7, 8, 9, 10, 11, 20, 26], np.float32)
    got = run_gpu(d)
    assert regime(got[3]) == capi.GQA_REGIME_PREFILL
    check(d, got)


def test_appended_zero_values():
    """The same through the append: a prompt whose middle rows have values of zero."""
    d = make(("f16", 2, 60, 16, 4, 128, 128, 16, (60, 60), None, -1, 0, 0, 1, 1), seed=71)
    d["v"][:, 16:48] = 0
    d["k"] *= np.float16(0.25)
    got = run_gpu(d)
    assert regime(got[3]) == capi.GQA_REGIME_PREFILL
    check(d, got)


@pytest.mark.parametrize("softcap", [0.0, 0.5, 30.0])
@pytest.mark.parametrize("tiles", list(TILES))
@pytest.mark.parametrize("dtype,tiny", [("f32", 1e-20), ("f32", 1e-36), ("f16", 1.0)])
def test_vanishing_scores_beside_masked_ones(dtype, tiny, tiles, softcap):
    """Rows of tiny queries on key blocks of zeros: every masked key stays without weight, padding rows are zeros."""
    S, G = TILES[tiles]
    d = make((dtype, 3, S, 4 * G, 4, 128, 256, 16, (200, S, 131), (S, S - 3, S // 2), 90, softcap, 0, 1, 0), seed=72)
    d["cache"][2][:] = 0.01
    d["cache"][2][:, :, ::2] = 0
    d["cache"][2][:, :, (200 - S) // 16:] = 0      # the diagonal of the first sequence
    d["q"][:, ::3] *= NP[dtype](tiny)
    d["q"][2, S // 2:] *= NP[dtype](tiny)     # padding rows
    got = run_gpu(d)
    assert regime(got[3]) == capi.GQA_REGIME_PREFILL
    check(d, got)


@pytest.mark.parametrize("softcap", [0.0, 2.0])
@pytest.mark.parametrize("tiles", list(TILES) + ["split"])
@pytest.mark.parametrize("factor", [1e30, 1e-30, 1e-35, 1e35])
def test_scales_far_out_of_range(factor, tiles, softcap):
    """Large queries on keys as much smaller, and the other way round: the scores are ordinary ones."""
    S, G = TILES.get(tiles, (2, 8))
    d = make(("f32", 2, S, 4 * G, 4, 128, 256, 16, (200, S + 7), (S, S - 1), -1, softcap, 0, 1, 0), seed=73)
    d["q"] *= np.float32(factor)
    d["cache"][2][:] /= np.float32(factor)
    got = run_gpu(d)
    assert (regime(got[3]) == capi.GQA_REGIME_PREFILL) == (tiles != "split")
    check(d, got)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 200, 2 ** 30, 301, 300, 299, 298])
@pytest.mark.parametrize("dtype,N,Nkv,S,total", [("f16", 16, 4, 150, 150), ("f16", 16, 16, 150, 150), ("f32", 16, 4, 150, 150),
                                                 ("f32", 4, 4, 150, 150), ("f16", 16, 4, 100, 300), ("f32", 16, 4, 100, 300),
                                                 ("f16", 4, 2, 1, 300), ("f32", 4, 2, 3, 300), ("f32", 6, 2, 9, 300)])
def test_windows_that_reach_every_row(dtype, N, Nkv, S, total, window):
    """Output and weights at windows beside the length and at the attribute's largest values."""
    d = make((dtype, 2, S, N, Nkv, 128, 320, 64, (total, S), None, window, 0, 1, 1, 1), seed=74)
    check(d, run_gpu(d))


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_the_largest_window_is_none(dtype):
    case = (dtype, 2, 150, 16, 4, 128, 320, 64, (150, 300), None, 2 ** 31 - 1, 4.0, 1, 1, 1)
    a, b = (run_gpu(make(case[:10] + (w,) + case[11:], seed=75)) for w in (2 ** 31 - 1, -1))
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[2], b[2])
