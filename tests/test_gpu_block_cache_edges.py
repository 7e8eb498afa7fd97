"""Block-scaled cache on the GPU: scales, group sizes and sizes at the edges of its kernels' index arithmetic."""

import numpy as np
import pytest
import torch

from oracle import block_cache as ob
from grouped_query_attention_gb300 import BlockCache, GroupQueryAttention, capi
from test_gpu_block_cache import (CASES, check, dev, from_gpu_cache, make, output_tolerance, regime, run_gpu,
                                  score_error, smallest_step)

pytestmark = pytest.mark.gpu


def check_with(d, got, **attrs):
    """check() for an operator with its own scale or smooth softmax."""
    out, cache, w, op = got
    rcache = [x.copy() for x in d["cache"]]
    rw = None if d["past_w"] is None else np.full(d["past_w"].shape, 7.5)
    ref, mag, reach = ob.step(d["q"], d["k"], d["v"], d["totals"] - 1, d["news"], rcache, d["bs"], d["N"], d["Nkv"],
                              softcap=d["softcap"], window=d["window"], sink=d["sink"],
                              past_weights=d["past_w"], weights=rw, **attrs)
    reach = np.abs(reach)
    assert op.block_status() == 0
    tol = output_tolerance(ref, mag, reach, d["dtype"], d["H"]) + smallest_step(d, rcache)
    assert (np.abs(out.astype(np.float64) - ref) <= tol).all()
    if w is not None:
        rel = 2 * score_error(reach.max(axis=(1, 2)), d["H"])[:, None, None] + 2.0 ** -19
        assert (np.abs(w - rw) <= rel * np.abs(rw) + 2.0 ** -23 * np.abs(rw) + 2.0 ** -30).all()


@pytest.mark.parametrize("scale", [-0.07, 0.3])
@pytest.mark.parametrize("name", ["one_token", "softcap_sink", "long_split", "h80_f32", "prompt_f32_h128", "prefill_past",
                                  "prefill_softcap_small", "prefill_two_tiles_f32", "prefill_window"])
def test_scale_of_either_sign(name, scale):
    d = make(CASES[name], seed=50)
    op = GroupQueryAttention(d["N"], d["Nkv"], softcap=float(d["softcap"]), local_window_size=d["window"], scale=scale)
    got = run_gpu(d, op)
    if name.startswith("prefill"):   # the prefill takes row maxima before the scale
        assert (regime(op) == capi.GQA_REGIME_PREFILL) == (scale > 0)
    check_with(d, got, scale=scale)


@pytest.mark.parametrize("name", ["one_token_f32", "softcap_sink", "long_split", "prompt_h128", "prefill_past",
                                  "prefill_two_tiles_f32", "prefill_softcap_small"])
def test_smooth_softmax(name):
    d = make(CASES[name], seed=54)
    op = GroupQueryAttention(d["N"], d["Nkv"], softcap=float(d["softcap"]), local_window_size=d["window"], smooth_softmax=1)
    check_with(d, run_gpu(d, op), smooth=True)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("H", [16, 64, 128, 256])
def test_cache_of_one_row(dtype, H):
    for total in (1, 0):
        d = make((dtype, 1, 1, 2, 1, H, 1, 16, (total,), (total,), -1, 0, 0, 1, 1), seed=55)
        check(d, run_gpu(d))


@pytest.mark.parametrize("softcap", [0.0, 4.0])
@pytest.mark.parametrize("N,Nkv,S,total,window", [(8, 8, 130, 257, -1), (8, 4, 70, 300, 65), (64, 1, 9, 400, -1),
                                                  (128, 1, 5, 333, -1), (128, 1, 7, 200, 90)])
def test_prompt_weights_of_group_sizes(N, Nkv, S, total, window, softcap):
    """Weights on the tensor cores: groups of 1 to 128 heads against tiles of 64 rows."""
    d = make(("f16", 4, S, N, Nkv, 128, 448, 64, (total, total - 3, S, total), (S, S - 2, S, 0), window, softcap, 1, 1, 1),
             seed=51)
    got = run_gpu(d)
    assert regime(got[3]) == capi.GQA_REGIME_PREFILL
    check(d, got)


@pytest.mark.parametrize("softcap", [0.0, 4.0])
@pytest.mark.parametrize("dtype,N,Nkv,H,S,total,window",
                         [("f16", 14, 2, 128, 90, 300, -1), ("f32", 6, 2, 128, 150, 150, -1), ("f16", 5, 1, 64, 130, 257, 70),
                          ("f32", 12, 1, 96, 60, 129, -1), ("f16", 8, 4, 16, 200, 200, -1), ("f32", 3, 3, 32, 150, 290, 33),
                          ("f16", 48, 1, 80, 20, 150, -1), ("f32", 100, 1, 48, 6, 200, -1), ("f16", 65, 1, 112, 7, 140, -1),
                          ("f16", 9, 3, 64, 129, 400, -1)])
def test_prefill_of_odd_heads_and_groups(dtype, N, Nkv, H, S, total, window, softcap):
    """Head sizes below 128 and groups that leave rows of a query tile empty, padded and empty sequences among them."""
    d = make((dtype, 4, S, N, Nkv, H, 448, 32, (total, total - 3, S - 1, 0), (S, S - 3, S - 1, 0), window, softcap, 1, 1, 1),
             seed=56)
    got = run_gpu(d)
    assert regime(got[3]) == capi.GQA_REGIME_PREFILL
    check(d, got)


ONE_TILE = {   # at most 128 query rows a KV head
    "f16": ("f16", 4, 30, 8, 2, 128, 448, 32, (300, 447, 30, 5), (30, 17, 30, 0), -1, 0, 1, 1, 1),
    "f16_softcap": ("f16", 4, 30, 8, 2, 96, 448, 64, (300, 447, 30, 5), (30, 17, 30, 0), 100, 6.0, 0, 1, 1),
    "f16_long": ("f16", 8, 32, 32, 8, 128, 1600, 64, (1500, 1100, 1600, 32, 33, 900, 1599, 700), None, -1, 0, 0, 1, 0),
    "f32": ("f32", 16, 18, 14, 2, 64, 448, 16, (300, 447, 18, 5) * 4, (18, 17, 18, 0) * 4, -1, 0, 1, 1, 1),
    "f32_softcap_long": ("f32", 16, 16, 16, 4, 128, 800, 64, (700,) * 16, None, -1, 6.0, 0, 0, 0),
}


@pytest.mark.parametrize("name", list(ONE_TILE))
def test_prefill_of_one_query_tile(name):
    d = make(ONE_TILE[name], seed=58)
    got = run_gpu(d)
    assert regime(got[3]) == capi.GQA_REGIME_PREFILL
    check(d, got)


@pytest.mark.parametrize("name,tile", [("f16", 0), ("f16_softcap", 1), ("f32", 1)])
def test_withheld_copies_of_one_query_tile_time_out(name, tile):
    d = make(ONE_TILE[name], seed=59)
    op = GroupQueryAttention(d["N"], d["Nkv"], softcap=float(d["softcap"]), local_window_size=d["window"])
    capi.gqa_set_wait_limit(op.handle, 200000, tile)
    run_gpu(d, op)
    assert op.block_status() == capi.GQA_DEVICE_TIMEOUT
    capi.gqa_set_wait_limit(op.handle, 0, -1)
    check(d, run_gpu(d, op))


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("dtype,N,Nkv,H", [("f16", 14, 2, 128), ("f32", 6, 2, 96), ("f16", 24, 8, 64)])
def test_prefill_padding_and_free_rows_are_not_read(dtype, N, Nkv, H, bad):
    """Padding rows of query, key and value, and scales of blocks behind the sequences, may hold anything."""
    d = make((dtype, 3, 140, N, Nkv, H, 448, 32, (300, 139, 41), (140, 100, 41), -1, 0, 1, 1, 1), seed=57)
    for b, (t, n) in enumerate(zip(d["totals"], d["news"])):
        for x in (d["q"], d["k"], d["v"]):
            x[b, n:] = bad
        for x in d["cache"][2:]:
            x[b, :, -(-int(t) // 32):] = bad
        d["past_w"][b, :, t - n:] = bad
    got = run_gpu(d)
    assert regime(got[3]) == capi.GQA_REGIME_PREFILL
    out, cache, w, op = got
    ref = [x.copy() for x in d["cache"]]
    for a, x, b in zip(cache, ref, range(4)):
        if b >= 2:   # compare what the oracle compares: NaN equals NaN there
            np.nan_to_num(a, copy=False), np.nan_to_num(x, copy=False)
    d["cache"] = ref
    check(d, (out, cache, w, op))


@pytest.mark.parametrize("dtype,S", [("f16", 1), ("f32", 2), ("f16", 100), ("f32", 60)])
def test_cache_offsets_beyond_32_bits(dtype, S):
    """A cache of 4.6 GB of codes each: the last sequence's rows lie behind 2^32."""
    B, N, Nkv, H, C, bs, small = 2, 32, 8, 128, 2_200_000, 64, 384
    d = make((dtype, B, S, N, Nkv, H, small, bs, (S + 5, 383), None, -1, 0, 0, 1, 1), seed=52)
    big = BlockCache.empty(B, Nkv, C, H, bs)
    for t, x in zip(big.tensors(), d["cache"]):
        t[:, :, :x.shape[2]] = dev(x)
    w = torch.full((B, Nkv, C), 7.5, device="cuda")
    w[:, :, :small] = dev(d["past_w"])
    op = GroupQueryAttention(N, Nkv)
    out = op.block_forward(dev(d["q"]), dev(d["k"]), dev(d["v"]), dev(d["totals"] - 1), 383, big, past_weights=w,
                           present_weights=w)
    torch.cuda.synchronize()
    cut = [t[:, :, :x.shape[2]].contiguous().cpu().numpy() for t, x in zip(big.tensors(), d["cache"])]
    pw = w[:, :, :small].cpu().numpy()
    for b, t in enumerate(d["totals"]):
        assert np.array_equal(pw[b, :, t:], d["past_w"][b, :, t:])
        pw[b, :, t:] = 7.5
    check(d, (out.cpu().numpy(), cut, pw, op))
    assert not big.key_codes[:, :, small:].any() and not big.value_codes[:, :, small:].any()
    assert (w[:, :, small:] == 7.5).all()

    # ... and eviction from there
    into, to_w = BlockCache.empty(B, Nkv, 128, H, bs), torch.full((B, Nkv, 128), 7.5, device="cuda")
    kept, seq = op.block_evict(big, w, dev(d["totals"] - 1), 383, 100, into, to_w, recent=20, first=4)
    ref = [np.zeros((B, Nkv, 128, H), np.int8) for _ in range(2)] + [np.zeros((B, Nkv, 2), np.float32) for _ in range(2)]
    rw = np.full((B, Nkv, 128), 7.5)
    rk, rl = ob.evict(cut, w[:, :, :small].cpu().numpy(), d["totals"] - 1, 100, 20, 4, bs, ref, rw)
    assert np.array_equal(kept.cpu().numpy(), rk) and np.array_equal(seq.cpu().numpy(), rl)
    for a, b in zip(from_gpu_cache(into), ref):
        assert np.array_equal(a, b)
    assert np.array_equal(to_w.cpu().numpy(), rw.astype(np.float32))


def test_captured_prompt_eviction_and_step():
    """A prompt with weights, an eviction and a decode step in one graph, replayed with new data."""
    B, S, N, Nkv, H, C, bs, keep = 2, 200, 16, 4, 128, 256, 64, 96
    rng = np.random.default_rng(53)
    op = GroupQueryAttention(N, Nkv)

    def data():
        return [rng.standard_normal((B, n, m * H)).astype(np.float16) for n in (S, 1) for m in (N, Nkv, Nkv)]

    bufs = [dev(x) for x in data()]
    seq = torch.full((B,), S - 1, dtype=torch.int32, device="cuda")
    cache, small = BlockCache.empty(B, Nkv, C, H, bs), BlockCache.empty(B, Nkv, 128, H, bs)
    w = torch.zeros((B, Nkv, C), device="cuda")

    def run():
        a = op.block_forward(*bufs[:3], seq, S, cache, present_weights=w)
        kept, left = op.block_evict(cache, w, seq, S, keep, small, recent=16, first=2)
        b = op.block_forward(*bufs[3:], left + 1, keep + 1, small)
        return a, kept, left, b

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for _ in range(3):
        for t, x in zip(bufs, data()):
            t.copy_(dev(x))
        for t in (*cache.tensors(), *small.tensors(), w):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*outs, *cache.tensors(), *small.tensors(), w)]
        for t in (*cache.tensors(), *small.tensors(), w):
            t.zero_()
        again = run()
        torch.cuda.synchronize()
        for x, y in zip(got, (*again, *cache.tensors(), *small.tensors(), w)):
            assert torch.equal(x, y)
    assert op.block_status() == 0


def test_arguments_past_32_bits_are_refused():
    """An integer whose low 32 bits alone would be a valid one."""
    d = make(CASES["one_token"], seed=60)
    op = GroupQueryAttention(d["N"], d["Nkv"])
    run_gpu(d, op)
    from test_gpu_block_cache import to_gpu_cache
    cache, into, big = to_gpu_cache(d["cache"], 64), BlockCache.empty(3, 2, 200, 128), 1 << 32
    q, w, seq = dev(d["q"]), dev(d["past_w"]), dev(d["totals"] - 1)
    calls = [lambda: op.block_forward(q, None, None, seq, big + 200, cache),
             lambda: op.block_forward(q, None, None, seq, 200, BlockCache(*cache.tensors(), big + 64)),
             lambda: op.block_evict(cache, w, seq, big + 200, 20, into),
             lambda: op.block_evict(cache, w, seq, 200, big + 20, into),
             lambda: op.block_evict(cache, w, seq, 200, 20, into, recent=big + 1),
             lambda: op.block_evict(cache, w, seq, 200, 20, into, first=big + 1)]
    for call in calls:
        with pytest.raises(ValueError):
            call()
    check(d, run_gpu(d, op))


@pytest.mark.parametrize("C", [64, 20000, 140000])
def test_eviction_made_here_holds_no_rows_of_a_skipped_sequence(C):
    """kept and the lengths that the call allocates are -1 there (the allocator's memory is filled beforehand)."""
    op, keep = GroupQueryAttention(2, 2), C // 3
    cache, into = BlockCache.empty(3, 2, C, 16, 16), BlockCache.empty(3, 2, keep, 16, 16)
    w = torch.rand((3, 2, C), device="cuda")
    seq = torch.tensor([C, C - 5, -2], dtype=torch.int32, device="cuda")
    for given in range(4):
        junk = [torch.full((3, 2, keep), 12345, dtype=torch.int32, device="cuda") for _ in range(4)] + \
               [torch.full((3,), 12345, dtype=torch.int32, device="cuda") for _ in range(4)]
        own = (junk[0] if given & 1 else None, junk[4] if given & 2 else None)
        del junk
        kept, lens = op.block_evict(cache, w, seq, C, keep, into, recent=3, kept=own[0], into_seqlens_k=own[1])
        assert op.block_status() == capi.GQA_DEVICE_BAD_SEQLEN
        for b in (0, 2):
            assert (kept[b] == (12345 if given & 1 else -1)).all()
            assert int(lens[b]) == (12345 if given & 2 else -1)
        assert int(lens[1]) == keep - 1 and bool((kept[1, :, 1:] > kept[1, :, :-1]).all())
        assert bool((kept[1, :, -3:] == torch.arange(C - 7, C - 4, device="cuda")).all())
