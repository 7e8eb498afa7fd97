"""Block-cache prompts past 1024 keys and past one query tile, with and without softcap and weights, and prompts of head
sizes above 128: the instantiations that long prompts and chunks run, against the fp64 definitions."""

import pytest

from grouped_query_attention_gb300 import capi
from test_gpu_block_cache import check, make, regime, run_gpu

pytestmark = pytest.mark.gpu

PREFILL = {
    # dtype, B, S, N, Nkv, H, C, bs, totals, news, window, softcap, sink, weights, key given
    "two_tiles": ("f16", 1, 150, 32, 4, 128, 1280, 64, (1200,), None, -1, 0, 0, 1, 1),
    "two_tiles_softcap": ("f16", 1, 150, 32, 4, 128, 1280, 64, (1200,), None, -1, 20.0, 1, 1, 1),
    "two_tiles_window": ("f16", 1, 200, 32, 4, 128, 1600, 16, (1577,), None, 1100, 0, 1, 1, 1),
    "two_tiles_window_softcap": ("f16", 1, 200, 32, 4, 96, 1600, 128, (1577,), (199,), 1100, 50.0, 1, 1, 1),
    "fresh_prompt": ("f16", 1, 1100, 8, 4, 128, 1152, 64, (1100,), None, -1, 0, 0, 1, 1),
    "fresh_prompt_softcap": ("f16", 1, 1100, 8, 4, 64, 1152, 64, (1100,), None, -1, 3.0, 0, 1, 1),
    "fresh_ragged": ("f16", 2, 1100, 2, 1, 128, 1152, 32, (1100, 300), (1100, 300), -1, 0, 0, 1, 1),
    "one_tile": ("f16", 8, 16, 32, 4, 128, 1152, 64, (1100, 1152, 1025, 16, 1024, 700, 1100, 900), None, -1, 0, 0, 1, 1),
    "one_tile_softcap": ("f16", 8, 16, 32, 4, 128, 1152, 64, (1100, 1152, 1025, 16, 1024, 700, 1100, 900), None, -1, 9.0,
                         1, 1, 1),
    "one_tile_softcap_short": ("f16", 4, 16, 32, 4, 128, 448, 64, (400, 300, 16, 444), None, -1, 9.0, 0, 1, 1),
}


@pytest.mark.parametrize("name", list(PREFILL))
def test_prefill(name):
    d = make(PREFILL[name], seed=80)
    got = run_gpu(d)
    assert regime(got[3]) == capi.GQA_REGIME_PREFILL
    check(d, got)


@pytest.mark.parametrize("softcap", [0.0, 10.0])
@pytest.mark.parametrize("dtype,H,S,total,window", [("f16", 256, 130, 250, -1), ("f16", 144, 90, 90, 40),
                                                    ("f32", 192, 100, 300, -1), ("f32", 256, 64, 640, 200)])
def test_prompts_of_wide_heads(dtype, H, S, total, window, softcap):
    """The split over the keys in row tiles of 8."""
    d = make((dtype, 2, S, 6, 2, H, 640, 32, (total, S), (S, S - 5), window, softcap, 1, 1, 1), seed=81)
    got = run_gpu(d)
    assert regime(got[3]) == capi.GQA_REGIME_DECODE
    check(d, got)
