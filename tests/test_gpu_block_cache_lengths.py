"""Block-cache steps whose total_sequence_length is only an upper bound of the lengths (a captured graph's capacity,
slots that are empty): the split over the keys then has fewer units of work than the grid has workers. Every call runs
on a workspace of NaN bytes, so that a piece no worker wrote shows."""

import numpy as np
import pytest
import torch

from grouped_query_attention_gb300 import GroupQueryAttention, capi
from grouped_query_attention_gb300.block_cache import _raw_stream
from test_gpu_block_cache import check, dev, from_gpu_cache, make, regime, run_gpu, to_gpu_cache

pytestmark = pytest.mark.gpu

ONE_OF_32 = tuple(100 if b == 17 else 0 for b in range(32))

CASES = {
    # dtype, B, S, N, Nkv, H, C, bs, totals, news, window, softcap, sink, weights, key given; T = C
    "decode": ("f16", 8, 1, 16, 8, 128, 2048, 64, (40, 33, 300, 64, 1, 100, 200, 257), None, -1, 0, 1, 0, 1),
    "decode_weights": ("f16", 8, 1, 8, 2, 128, 4096, 64, (40,) * 8, None, -1, 0, 0, 1, 1),
    "decode_f32": ("f32", 8, 1, 8, 2, 64, 4096, 32, (40, 33, 300, 64, 1, 100, 200, 257), None, -1, 0, 1, 0, 1),
    "decode_weights_f32": ("f32", 8, 1, 32, 8, 128, 2048, 16, (200,) * 8, None, -1, 0, 0, 1, 1),
    "one_live_slot": ("f16", 32, 1, 8, 8, 128, 1024, 64, ONE_OF_32, tuple(min(t, 1) for t in ONE_OF_32), -1, 0, 0, 1, 1),
    "one_live_slot_f32": ("f32", 32, 2, 4, 2, 96, 1024, 64, ONE_OF_32, tuple(min(t, 2) for t in ONE_OF_32), -1, 0, 0, 1, 1),
    "h256": ("f16", 4, 1, 8, 4, 256, 2048, 64, (90, 33, 300, 0), (1, 1, 1, 0), -1, 0, 0, 1, 1),
    "row_tiles_f32": ("f32", 3, 9, 8, 2, 192, 2048, 32, (90, 9, 300), (9, 9, 4), -1, 0, 0, 1, 1),
    "window_softcap": ("f16", 6, 2, 8, 2, 80, 4096, 16, (90, 33, 300, 700, 2, 64), None, 70, 6.0, 1, 1, 1),
    "attend_only": ("f16", 4, 1, 8, 2, 64, 4096, 32, (50, 3, 129, 64), None, -1, 0, 0, 0, 0),
    "drafts": ("f16", 8, 4, 12, 3, 112, 3000, 128, (50, 4, 129, 64, 65, 31, 33, 500), (4, 4, 1, 2, 0, 3, 4, 4), -1, 0, 0, 1, 1),
}


def poisoned(d):
    """An operator whose eager workspace holds NaN bytes."""
    op = GroupQueryAttention(d["N"], d["Nkv"], softcap=float(d["softcap"]), local_window_size=d["window"])
    op._block_ws[(0, _raw_stream(0))] = torch.full((1 << 28,), 0xFF, dtype=torch.uint8, device="cuda")
    return op


@pytest.mark.parametrize("name", list(CASES))
def test_total_sequence_length_above_the_lengths(name):
    d = make(CASES[name], seed=60)
    got = run_gpu(d, poisoned(d), total=d["C"])
    assert regime(got[3]) == capi.GQA_REGIME_DECODE
    check(d, got)


@pytest.mark.parametrize("total", [41, 64, 300, 1000, 2111, 4096])
def test_the_bound_does_not_change_the_result(total):
    """From a tight bound to a loose one the outputs stay within the tolerance of the same definition."""
    d = make(("f16", 3, 1, 8, 2, 128, 4096, 64, (40, 1, 33), None, -1, 0, 0, 1, 1), seed=61)
    check(d, run_gpu(d, poisoned(d), total=total))


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_captured_step_whose_lengths_change(dtype):
    """One graph for the cache's whole capacity, replayed at lengths that shrink and grow; what the workspace holds
    from the replay before does not enter."""
    B, N, Nkv, H, C, bs = 4, 8, 2, 128, 4096, 64
    first = make((dtype, B, 1, N, Nkv, H, C, bs, (4000, 3000, 3500, 4096), None, -1, 0, 0, 1, 1), seed=62)
    op = GroupQueryAttention(N, Nkv)
    run_gpu(first, op, total=C)
    t = {k: dev(first[k]) for k in ("q", "k", "v")}
    seq, cache = dev(first["totals"] - 1), to_gpu_cache(first["cache"], bs)
    w, pw = dev(first["past_w"]), torch.full((B, Nkv, C), 7.5, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = op.block_forward(t["q"], t["k"], t["v"], seq, C, cache, past_weights=w, present_weights=pw)
    for rep, totals in enumerate([(4000, 3000, 3500, 4096), (33, 100, 64, 200), (4, 1, 2000, 1), (40, 33, 300, 64)]):
        d = make((dtype, B, 1, N, Nkv, H, C, bs, totals, None, -1, 0, 0, 1, 1), seed=63 + rep)
        for k, x in t.items():
            x.copy_(dev(d[k]))
        seq.copy_(dev(d["totals"] - 1))
        for x, y in zip(cache.tensors(), d["cache"]):
            x.copy_(dev(y))
        w.copy_(dev(d["past_w"]))
        pw.fill_(7.5)
        graph.replay()
        torch.cuda.synchronize()
        check(d, (out.cpu().numpy(), from_gpu_cache(cache), pw.cpu().numpy(), op))


def test_no_live_slot():
    d = make(("f16", 4, 1, 8, 2, 128, 2048, 64, (0, 0, 0, 0), (0, 0, 0, 0), -1, 0, 0, 1, 1), seed=66)
    got = run_gpu(d, poisoned(d), total=d["C"])
    check(d, got)
    assert not got[0].any() and (got[2] == 7.5).all()
