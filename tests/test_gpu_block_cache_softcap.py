"""Attention over the block-scaled cache under softcaps far above and below the scores (oracle/block_cache.py). The
tolerance takes 2^-20 of the largest |score| for c tanh(s / c), whatever c is: its quotient and product, the tangent's
fit, two or three steps of 2^-24 each."""

import numpy as np
import pytest

from grouped_query_attention_gb300 import GroupQueryAttention, capi
from oracle import block_cache as ob
from test_gpu_block_cache import make, output_tolerance, regime, run_gpu, smallest_step

pytestmark = pytest.mark.gpu

FORMS = {"one_tile": (8, 16), "two_tiles": (60, 16), "split": (2, 8)}


def softcap_check(dtype, form, softcap, change=None):
    S, G = FORMS[form]
    d = make((dtype, 2, S, 4 * G, 4, 128, 256, 16, (200, S + 7), (S, S - 1), -1, softcap, 0, 0, 1), seed=80)
    if change:
        change(d)
    cache = [x.copy() for x in d["cache"]]
    out, mag, reach = ob.step(d["q"], d["k"], d["v"], d["totals"] - 1, d["news"], cache, d["bs"], d["N"], d["Nkv"],
                              softcap=softcap, window=-1, sink=None, past_weights=None, weights=None)
    op = GroupQueryAttention(d["N"], d["Nkv"], softcap=softcap)
    got = run_gpu(d, op)
    assert op.block_status() == 0
    assert (regime(op) == capi.GQA_REGIME_PREFILL) == (form != "split" and 2.0 ** -40 <= softcap <= 2.0 ** 19)
    more = 2 * 2.0 ** -20 * np.minimum(softcap, reach).repeat(d["H"], -1).reshape(out.shape) * mag
    tol = output_tolerance(out, mag, reach, dtype, d["H"]) + more + smallest_step(d, cache)
    bad = ~(np.abs(got[0] - out) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), np.nanmax(np.abs(got[0] - out)))


@pytest.mark.parametrize("softcap", [1e4, 5e5, 1e6, 3e7, 1e8, 1e10, 1e30])
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_softcaps_far_above_the_scores(dtype, form, softcap):
    softcap_check(dtype, form, softcap)


@pytest.mark.parametrize("softcap", [1e-3, 1e-10, 1e-38, 1e-45])
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_softcaps_far_below_the_scores(dtype, form, softcap):
    """Every score is c, -c or (of a zero product) 0: all visible rows weigh the same."""
    def zeros(d):
        d["k"][:, 0] = 0
    softcap_check(dtype, form, softcap, zeros)


@pytest.mark.parametrize("softcap", [1e38, 2.4e38, 3.4e38])
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_the_largest_softcaps(dtype, form, softcap):
    """c log2(e) is no float any more."""
    softcap_check(dtype, form, softcap)
