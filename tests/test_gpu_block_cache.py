"""GPU tests of the multi-axis rotary, attention over the block-scaled int8 cache and the eviction from it, against
the fp64 definitions of oracle/block_cache.py.

Tolerances, derived from the roundings (u = 2^-24, the half step of fp32):
  codes, block scales, kept rows, lengths: equal.
  output: its own rounding, half a step of its type; each probability enters the product with V rounded to fp16
    (2^-11 relative; two fp16 parts, 2^-22, for fp32); a score is a sum of H products in fp32 (at most (H + 16) 2 u
    of max|q| sum|k| scale with its factors; fp32 queries enter as two fp16 parts, within 2 u of max|q|), and an
    error d of the scores changes a probability by 2 d at most; exp2 and the fp32 sums 2^-20. All of these weigh
    sum_j p_j |v_j|. The smallest step of fp16 is 2^-24: a factor p_j s_j 2^(6 - w) (s_j the V scale, 2^w at most
    twice the largest) below 2^-14 is off by up to 2^-25 whatever its size, which is 2^-30 of the largest scale times
    |code| <= 127 for every key.
  attention weights: the same without V.
"""

import numpy as np
import pytest
import torch

from grouped_query_attention_gb300 import BlockCache, GroupQueryAttention, GqaError, capi
from oracle import block_cache as ob

pytestmark = pytest.mark.gpu

NP = {"f16": np.float16, "f32": np.float32}


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def random_cache(rng, B, Nkv, C, H, bs):
    nb = -(-C // bs)
    return [rng.integers(-127, 128, (B, Nkv, C, H)).astype(np.int8) for _ in range(2)] + \
           [(rng.uniform(0.01, 0.03, (B, Nkv, nb)) * np.where(rng.random((B, Nkv, nb)) < 0.1, 8, 1)).astype(np.float32)
            for _ in range(2)]


def to_gpu_cache(cache, bs):
    return BlockCache(*(dev(x) for x in cache), bs)


def from_gpu_cache(c):
    return [t.cpu().numpy() for t in c.tensors()]


def score_error(reach, H):
    return (H + 20) * 2.0 ** -23 * reach


def smallest_step(d, cache):
    """What probabilities below fp16's normal range may add up to, (B, 1, 1)."""
    bs, out = d["bs"], np.zeros((d["B"], 1, 1))
    for b, t in enumerate(d["totals"]):
        if t > 0:
            out[b] = t * 127 * cache[3][b, :, :-(-int(t) // bs)].max() * 2.0 ** -30
    return out


def output_tolerance(out, mag, reach, dtype, H):
    B, S = out.shape[:2]
    d = np.repeat(score_error(reach, H), H, axis=-1).reshape(out.shape)
    p = 2.0 ** -11 if dtype == "f16" else 2.0 ** -22
    half = 2.0 ** -11 if dtype == "f16" else 2.0 ** -24
    return half * np.abs(out) + (p * (1 + half) + 2 * d + 2.0 ** -20) * mag + 2.0 ** -25


CASES = {
    # name: dtype, B, S, N, Nkv, H, C, bs, totals, news (None: S), window, softcap, sink, weights, key given
    "one_token": ("f16", 3, 1, 8, 2, 128, 200, 64, (1, 64, 197), None, -1, 0, 0, 1, 1),
    "one_token_f32": ("f32", 3, 1, 8, 2, 128, 200, 64, (1, 65, 200), None, -1, 0, 0, 1, 1),
    "one_token_first_of_block": ("f16", 2, 1, 4, 4, 64, 130, 64, (65, 129), None, -1, 0, 0, 0, 1),
    "h16": ("f16", 2, 2, 3, 3, 16, 50, 16, (2, 50), None, -1, 0, 0, 1, 1),
    "h16_f32": ("f32", 2, 2, 3, 3, 16, 50, 16, (2, 50), None, -1, 0, 0, 1, 1),
    "h48_g3": ("f16", 2, 1, 6, 2, 48, 70, 32, (33, 70), None, -1, 0, 0, 0, 1),
    "h80_f32": ("f32", 2, 3, 10, 2, 80, 90, 16, (40, 90), (3, 2), -1, 0, 1, 1, 1),
    "h96_ragged": ("f16", 4, 5, 6, 2, 96, 300, 32, (300, 5, 77, 0), (5, 5, 1, 0), -1, 0, 0, 1, 1),
    "h192": ("f16", 2, 4, 4, 2, 192, 100, 64, (100, 37), None, -1, 0, 0, 1, 1),
    "h256_f32": ("f32", 2, 1, 4, 1, 256, 140, 128, (140, 3), None, -1, 0, 0, 1, 1),
    "h256_chunk": ("f16", 1, 20, 4, 2, 256, 64, 16, (64,), None, -1, 0, 0, 1, 1),
    "g12": ("f16", 2, 1, 12, 1, 64, 100, 16, (100, 17), None, -1, 0, 1, 1, 1),
    "g16_f32": ("f32", 1, 1, 16, 1, 64, 100, 16, (100,), None, -1, 0, 0, 1, 1),
    "window": ("f16", 3, 2, 8, 2, 64, 400, 32, (400, 150, 9), None, 100, 0, 0, 1, 1),
    "window_0_f32": ("f32", 2, 3, 4, 2, 64, 100, 16, (100, 33), None, 0, 0, 0, 1, 1),
    "softcap_sink": ("f16", 2, 1, 8, 2, 128, 300, 64, (300, 130), None, -1, 5.0, 1, 1, 1),
    "softcap_f32": ("f32", 2, 7, 8, 4, 64, 100, 16, (100, 50), None, 40, 5.0, 1, 1, 1),
    "long_split": ("f16", 2, 1, 4, 2, 128, 9000, 64, (9000, 5001), None, -1, 0, 0, 1, 1),
    "long_split_f32": ("f32", 1, 1, 2, 1, 64, 20000, 256, (19999,), None, -1, 0, 0, 1, 1),
    "attend_only": ("f16", 2, 3, 8, 2, 64, 100, 32, (99, 3), None, -1, 0, 0, 1, 0),
    "prompt": ("f16", 2, 70, 4, 2, 64, 128, 64, (70, 41), (70, 41), -1, 0, 0, 1, 1),
    "prompt_f32_h128": ("f32", 2, 70, 4, 2, 128, 128, 64, (70, 41), (70, 41), -1, 0, 0, 1, 1),
    "prompt_h128": ("f16", 2, 150, 8, 2, 128, 256, 64, (150, 99), (150, 99), -1, 0, 0, 1, 1),
    "chunk_h128_window": ("f16", 2, 40, 8, 2, 128, 600, 16, (600, 300), None, 130, 0, 1, 1, 1),
    "prefill_softcap_g16": ("f16", 1, 60, 64, 4, 128, 300, 32, (300,), None, -1, 4.0, 0, 1, 1),
    "chunk_h128_f32": ("f32", 2, 33, 8, 2, 128, 300, 32, (300, 40), (33, 7), -1, 0, 1, 1, 1),
    "prefill_two_tiles": ("f16", 1, 300, 4, 1, 128, 512, 64, (300,), None, -1, 0, 0, 1, 1),
    "prefill_two_tiles_f32": ("f32", 1, 200, 16, 4, 128, 512, 128, (200,), None, -1, 0, 1, 1, 1),
    "prefill_past": ("f16", 3, 90, 8, 2, 128, 700, 16, (700, 333, 90), (90, 17, 90), -1, 0, 1, 1, 1),
    "prefill_window": ("f16", 2, 200, 4, 2, 128, 700, 32, (641, 222), None, 77, 0, 0, 1, 1),
    "prefill_window_f32": ("f32", 2, 100, 16, 4, 128, 700, 256, (641, 222), (100, 50), 200, 0, 0, 1, 1),
    "prefill_softcap_small": ("f16", 1, 200, 16, 4, 128, 512, 64, (400,), None, -1, 50.0, 1, 1, 1),
    "prefill_softcap_large": ("f32", 1, 100, 16, 4, 128, 512, 64, (301,), None, 150, 1.5, 1, 1, 1),
    "prefill_flush_f32": ("f32", 1, 50, 64, 8, 128, 1200, 64, (1100,), None, -1, 0, 0, 1, 1),
    "prefill_flush_softcap_f32": ("f32", 1, 50, 64, 8, 128, 1200, 64, (1100,), None, -1, 20.0, 0, 1, 1),
    "flush_h80_f32": ("f32", 2, 9, 4, 2, 80, 1500, 64, (1500, 700), None, -1, 0, 0, 1, 1),
    "prefill_g1": ("f16", 1, 200, 2, 2, 128, 256, 16, (199,), (190,), -1, 0, 0, 1, 1),
    "prefill_g32": ("f16", 1, 20, 32, 1, 128, 256, 64, (150,), None, -1, 0, 0, 1, 1),
    "prefill_g128": ("f32", 1, 3, 128, 1, 128, 64, 16, (40,), None, -1, 0, 0, 1, 1),
    "prefill_attend_only": ("f16", 2, 60, 8, 2, 128, 200, 32, (199, 60), None, -1, 0, 0, 0, 0),
    "chunk_g3": ("f16", 2, 30, 6, 2, 128, 200, 64, (200, 30), None, -1, 0, 0, 1, 1),
    "chunk_g7_f32": ("f32", 1, 20, 7, 1, 96, 200, 16, (123,), None, 64, 0, 0, 1, 1),
    "empty_slots": ("f16", 4, 2, 4, 2, 64, 64, 16, (0, 10, 0, 64), (0, 0, 0, 2), -1, 0, 0, 1, 1),
}


def make(case, seed=0):
    dtype, B, S, N, Nkv, H, C, bs, totals, news, window, softcap, sink, weights, has_kv = case
    rng = np.random.default_rng(seed)
    t = NP[dtype]
    d = dict(dtype=dtype, B=B, S=S, N=N, Nkv=Nkv, H=H, C=C, bs=bs, window=window, softcap=softcap,
             totals=np.array(totals, np.int32), news=None if news is None else np.array(news, np.int32))
    d["cache"] = random_cache(rng, B, Nkv, C, H, bs)
    d["q"] = (2 * rng.standard_normal((B, S, N * H))).astype(t)
    d["k"] = rng.standard_normal((B, S, Nkv * H)).astype(t) if has_kv else None
    d["v"] = rng.standard_normal((B, S, Nkv * H)).astype(t) if has_kv else None
    d["sink"] = rng.standard_normal(N).astype(t) if sink else None
    d["past_w"] = rng.random((B, Nkv, C)).astype(np.float32) if weights else None
    return d


def run_oracle(d):
    cache = [x.copy() for x in d["cache"]]
    w = None
    if d["past_w"] is not None:
        w = np.full(d["past_w"].shape, 7.5)   # what the present buffer holds beforehand
    out, mag, reach = ob.step(d["q"], d["k"], d["v"], d["totals"] - 1, d["news"], cache, d["bs"], d["N"], d["Nkv"],
                              softcap=d["softcap"], window=d["window"], sink=d["sink"], past_weights=d["past_w"],
                              weights=w)
    return out, mag, reach, cache, w


def run_gpu(d, op=None, total=None):
    op = op or GroupQueryAttention(d["N"], d["Nkv"], softcap=float(d["softcap"]), local_window_size=d["window"])
    cache = to_gpu_cache(d["cache"], d["bs"])
    pw = None if d["past_w"] is None else torch.full(d["past_w"].shape, 7.5, device="cuda")
    out = op.block_forward(dev(d["q"]), dev(d["k"]), dev(d["v"]), dev(d["totals"] - 1),
                           max(1, int(d["totals"].max())) if total is None else total, cache, new_lens=dev(d["news"]),
                           head_sink=dev(d["sink"]), past_weights=dev(d["past_w"]), present_weights=pw)
    torch.cuda.synchronize()
    return out.cpu().numpy(), from_gpu_cache(cache), None if pw is None else pw.cpu().numpy(), op


def check(d, got):
    out, cache, w, op = got
    ref, mag, reach, rcache, rw = run_oracle(d)
    assert op.block_status() == 0
    for name, a, b in zip(("key codes", "value codes", "key scales", "value scales"), cache, rcache):
        assert np.array_equal(a, b), f"{name}: {np.sum(a != b)} differ"
    err = np.abs(out.astype(np.float64) - ref)
    tol = output_tolerance(ref, mag, reach, d["dtype"], d["H"]) + smallest_step(d, rcache)
    assert (err <= tol).all(), f"output off by {err.max()} (worst {np.max(err / tol)} of its tolerance)"
    if w is not None:
        # sum over a sequence's probabilities; each within 2 d + 2^-20 of itself
        r = reach.max(axis=(1, 2)) if reach.size else np.zeros(d["B"])
        rel = 2 * score_error(r, d["H"])[:, None, None] + 2.0 ** -19
        tol = rel * np.abs(rw) + 2.0 ** -23 * np.abs(rw) + 2.0 ** -30
        err = np.abs(w - rw)
        assert (err <= tol).all(), f"weights off by {err.max()} (worst {np.max(err / tol)} of its tolerance)"


def regime(op):
    return capi.gqa_block_describe_plan(op.handle, *op._block_calls["forward"].structs).regime


@pytest.mark.parametrize("name", list(CASES))
def test_step(name):
    d = make(CASES[name])
    got = run_gpu(d)
    if name.startswith("prefill"):
        assert regime(got[3]) == capi.GQA_REGIME_PREFILL
    check(d, got)


def test_capacity_beyond_the_lengths():
    d = make(CASES["h96_ragged"], seed=4)
    check(d, run_gpu(d, total=d["C"]))


def test_a_gross_error_breaks_the_tolerance():
    d = make(CASES["one_token"])
    out, cache, w, op = run_gpu(d)
    d["cache"][3][:] *= np.float32(1.01)      # planted in the oracle's inputs
    with pytest.raises(AssertionError):
        check(d, (out, cache, w, op))


def test_garbage_behind_the_rows_does_not_enter():
    """Codes and scales behind the live rows, padding rows and past weights of new rows are not read as data."""
    d = make(CASES["h96_ragged"], seed=5)
    bs = d["bs"]
    for b, t in enumerate(d["totals"]):
        first_free = -(-int(t) // bs)
        for s in d["cache"][2:]:
            s[b, :, first_free:] = np.nan
        for x in (d["q"], d["k"], d["v"]):
            x[b, d["news"][b]:] = np.nan
        d["past_w"][b, :, t - d["news"][b]:] = np.nan
    check_nan = run_gpu(d)
    assert not np.isnan(check_nan[0]).any()
    ref = dict(d)
    ref["past_w"] = np.where(np.isnan(d["past_w"]), 0, d["past_w"])
    out, cache, w, op = check_nan
    cache = [np.where(np.isnan(c), 0, c) if c.dtype == np.float32 else c for c in cache]
    ref["cache"] = [np.where(np.isnan(c), 0, c) if c.dtype == np.float32 else c for c in d["cache"]]
    check(ref, (out, cache, w, op))


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_append_of_odd_values(dtype):
    """Zero blocks, infinities and NaN, subnormals, ties, a growing and a staying scale, block by block."""
    rng = np.random.default_rng(6)
    B, Nkv, H, C, bs = 1, 2, 64, 128, 16
    t = NP[dtype]
    S = 112
    k = rng.standard_normal((B, S, Nkv * H)).astype(t)
    k[0, 0:16] = 0
    k[0, 16:32] *= t(1e-7)
    k[0, 33, 5], k[0, 34, 6], k[0, 35, 7] = np.inf, -np.inf, np.nan
    k[0, 48:64] = np.round(k[0, 48:64] * 20) / 2       # many ties once the largest is 127
    k[0, 48, ::H] = 127
    k[0, 64:80] = np.nan
    v = (k[::-1] * t(0.5)).copy()
    op = GroupQueryAttention(2, Nkv)
    cache, ref = to_gpu_cache([np.zeros((B, Nkv, C, H), np.int8)] * 2 + [np.zeros((B, Nkv, 8), np.float32)] * 2, bs), \
        [np.zeros((B, Nkv, C, H), np.int8) for _ in range(2)] + [np.zeros((B, Nkv, 8), np.float32) for _ in range(2)]
    done = 0
    for n in (7, 1, 30, 50, 24):
        rows = slice(done, done + n)
        done += n
        op.block_forward(torch.zeros((B, n, 2 * H), dtype=torch.float16 if dtype == "f16" else torch.float32,
                                     device="cuda"), dev(k[:, rows]), dev(v[:, rows]),
                         torch.tensor([done - 1], dtype=torch.int32, device="cuda"), C, cache)
        for g in range(Nkv):
            for x, c, s in ((k, ref[0], ref[2]), (v, ref[1], ref[3])):
                ob.append(c[0, g], s[0, g], x[0, rows].reshape(n, Nkv, H)[:, g], done - n, bs)
        for name, a, b in zip(("kc", "vc", "ks", "vs"), from_gpu_cache(cache), ref):
            assert np.array_equal(a, b), (name, done, np.argwhere(a != b)[:4])
    assert op.block_status() == 0


def test_wide_range_of_value_scales():
    """Blocks whose scales differ by 2^12 keep the small ones' precision where the large ones have no weight."""
    for dtype in ("f16", "f32"):
        d = make((dtype, 1, 1, 2, 1, 64, 512, 16, (512,), None, -1, 0, 0, 0, 0), seed=7)
        d["cache"][3][:] = 0.01
        d["cache"][3][0, 0, 3] = 0.01 * 4096
        d["cache"][3][0, 0, 20] = 0.0
        d["cache"][3][0, 0, 25] = 1e-30
        d["cache"][0][0, 0, 48:64] = -127 * np.sign(d["q"][0, 0, :64].astype(np.float32)).astype(np.int8)  # no weight
        d["q"][0, 0, 64:] = d["q"][0, 0, :64]
        check(d, run_gpu(d))


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_wide_range_of_value_scales_prefill(dtype):
    d = make((dtype, 1, 60, 64, 4, 128, 512, 16, (512,), None, -1, 0, 0, 1, 0), seed=7)
    d["cache"][3][:] = 0.01
    d["cache"][3][0, 0, 3] = 0.01 * 64
    d["cache"][3][0, 0, 20] = 0.0
    d["cache"][3][0, 0, 25] = 1e-30
    d["cache"][2][0, 0, 21] = 0.0
    d["cache"][1][0, 0, 320:336] = 0
    got = run_gpu(d)
    assert regime(got[3]) == capi.GQA_REGIME_PREFILL
    check(d, got)


@pytest.mark.parametrize("name,tile", [("one_token", 0), ("long_split", 1), ("prefill_past", 0), ("prefill_past", 1),
                                       ("prefill_two_tiles_f32", 1)])
def test_withheld_copies_time_out(name, tile):
    """A pipeline wait that runs out ends the call with a status bit; the operator works afterwards."""
    d = make(CASES[name])
    op = GroupQueryAttention(d["N"], d["Nkv"], softcap=float(d["softcap"]), local_window_size=d["window"])
    capi.gqa_set_wait_limit(op.handle, 200000, tile)
    run_gpu(d, op)
    assert op.block_status() == capi.GQA_DEVICE_TIMEOUT
    capi.gqa_set_wait_limit(op.handle, 0, -1)
    check(d, run_gpu(d, op))


@pytest.mark.parametrize("bad", [(200, 1), (-2, 1), (5, 6), (5, -1), (3, 4)])
def test_bad_lengths_skip_the_sequence(bad):
    d = make(("f16", 2, 5, 4, 2, 64, 100, 16, (50, 60), (3, 5), -1, 0, 0, 1, 1), seed=8)
    good = make(("f16", 2, 5, 4, 2, 64, 100, 16, (50, 60), (3, 5), -1, 0, 0, 1, 1), seed=8)
    d["totals"], d["news"] = np.array([bad[0], 60], np.int32), np.array([bad[1], 5], np.int32)
    op = GroupQueryAttention(4, 2)
    cache = to_gpu_cache(d["cache"], 16)
    out = torch.full((2, 5, 256), 3.0, dtype=torch.float16, device="cuda")
    pw = torch.full((2, 2, 100), 7.5, device="cuda")
    op.block_forward(dev(d["q"]), dev(d["k"]), dev(d["v"]), dev(d["totals"] - 1), 100, cache, new_lens=dev(d["news"]),
                     past_weights=dev(d["past_w"]), present_weights=pw, output=out)
    assert op.block_status() == capi.GQA_DEVICE_BAD_SEQLEN and op.block_status() == 0
    got = from_gpu_cache(cache)
    ref, mag, reach, rcache, rw = run_oracle(good)
    for a, b, c in zip(got, rcache, d["cache"]):
        assert np.array_equal(a[1], b[1]) and np.array_equal(a[0], c[0])
    out, pw = out.cpu().numpy(), pw.cpu().numpy()
    assert (out[0] == 3).all() and (pw[0] == 7.5).all()
    tol = output_tolerance(ref, mag, reach, "f16", 64) + smallest_step(good, rcache)
    assert (np.abs(out[1] - ref[1]) <= tol[1]).all()


# ------------------------------------------------------------------ rotary

ROTARY = {
    # name: dtype, B, S, N, Nkv (0: no key), H, sections, interleaved, norm, fp32 tables
    "three_axes": ("f16", 2, 5, 8, 2, 128, (16, 24, 24), 0, 0, 0),
    "three_axes_norm": ("f16", 2, 5, 8, 2, 128, (16, 24, 24), 0, 1, 0),
    "odd_sections": ("f16", 3, 7, 3, 1, 64, (5, 20, 7), 0, 0, 1),
    "interleaved": ("f32", 2, 9, 4, 2, 96, (16, 16, 16), 1, 1, 0),
    "partial": ("f32", 1, 33, 5, 5, 80, (3, 13), 0, 1, 0),
    "partial_interleaved": ("f16", 1, 3, 5, 5, 80, (8, 5, 3), 1, 0, 1),
    "one_axis_h16": ("f32", 2, 3, 2, 1, 16, (8,), 0, 0, 0),
    "eight_axes_h256": ("f16", 1, 4, 2, 2, 256, (16,) * 8, 1, 1, 0),
    "query_only": ("f16", 2, 1, 7, 0, 128, (64,), 0, 1, 0),
    "many_heads": ("f16", 1, 2, 65, 13, 32, (4, 12), 0, 0, 0),
    "many_tokens": ("f16", 2, 3000, 4, 2, 64, (8, 12, 12), 0, 1, 0),
}


def rotary_inputs(case, seed=0):
    dtype, B, S, N, Nkv, H, sec, inter, norm, f32tab = case
    rng = np.random.default_rng(seed)
    t = NP[dtype]
    R, pairs = 97, sum(sec)
    ang = np.arange(R)[:, None] * 1e4 ** (-np.arange(pairs) / pairs)
    tt = np.float32 if f32tab else t
    return dict(q=rng.standard_normal((B, S, N * H)).astype(t),
                k=rng.standard_normal((B, S, Nkv * H)).astype(t) if Nkv else None,
                pos=rng.integers(0, R, (len(sec), B, S)).astype(np.int32), cos=np.cos(ang).astype(tt),
                sin=np.sin(ang).astype(tt), qw=(1 + 0.1 * rng.standard_normal(H)).astype(t) if norm else None,
                kw=(1 + 0.1 * rng.standard_normal(H)).astype(t) if norm and Nkv else None)


@pytest.mark.parametrize("name", list(ROTARY))
@pytest.mark.parametrize("in_place", [False, True])
def test_rotary(name, in_place):
    dtype, B, S, N, Nkv, H, sec, inter, norm, _ = case = ROTARY[name]
    i = rotary_inputs(case)
    op = GroupQueryAttention(N, Nkv or 1)
    q, k = dev(i["q"]), dev(i["k"])
    oq, ok = op.rotary_axes(q, k, dev(i["pos"]), dev(i["cos"]), dev(i["sin"]), sec, bool(inter), dev(i["qw"]),
                            dev(i["kw"]), out_query=q if in_place else None, out_key=k if in_place else None)
    assert op.block_status() == 0
    half = 2.0 ** -11 if dtype == "f16" else 2.0 ** -24
    for x, y, n, w in ((i["q"], oq, N, i["qw"]), (i["k"], ok, Nkv, i["kw"])):
        if x is None:
            assert y is None
            continue
        ref = ob.rotary_axes(x, n, i["pos"], i["cos"], i["sin"], sec, bool(inter), w)
        # an fp32 rotation: two rounded products and a sum (3 u of |x| + |partner|); the norm's sum of H squares,
        # root and products: (H / 8 + 8) u; then one rounding to the type
        y0 = np.abs(ob.rotary_axes(x, n, 0 * i["pos"], np.ones_like(i["cos"]), 0 * i["sin"], sec, bool(inter), w))
        y0 = y0.reshape(B, S, n, H)
        pairs = sum(sec)
        both = y0.copy()
        both[..., :pairs] += y0[..., pairs:2 * pairs]
        both[..., pairs:2 * pairs] += y0[..., :pairs]
        tol = half * np.abs(ref) + 2.0 ** -24 * (4 + (H / 8 + 8) * norm) * both.reshape(ref.shape) + 2.0 ** -25
        err = np.abs(y.cpu().numpy().astype(np.float64) - ref)
        assert (err <= tol).all(), (err / tol).max()


def test_rotary_of_one_axis_is_the_stored_rows_rotary():
    """At head size 128 and positions past + i the rows equal those gqa_forward stores, byte for byte."""
    B, S, N, Nkv, H, C = 2, 9, 4, 2, 128, 16
    i = rotary_inputs(("f16", B, S, N, Nkv, H, (64,), 0, 1, 0), seed=3)
    i["pos"] = np.broadcast_to(np.arange(S, dtype=np.int32), (1, B, S))
    op = GroupQueryAttention(N, Nkv)
    _, k = op.rotary_axes(dev(i["q"]), dev(i["k"]), dev(i["pos"]), dev(i["cos"]), dev(i["sin"]), (64,),
                          q_norm_weight=dev(i["qw"]), k_norm_weight=dev(i["kw"]))
    full = GroupQueryAttention(N, Nkv, do_rotary=1)
    pk, pv = (torch.zeros((B, Nkv, C, H), dtype=torch.float16, device="cuda") for _ in range(2))
    full(dev(i["q"]), dev(i["k"]), dev(i["k"]), torch.full((B,), S - 1, dtype=torch.int32, device="cuda"), S, pk, pv,
         cos_cache=dev(i["cos"]), sin_cache=dev(i["sin"]), q_norm_weight=dev(i["qw"]), k_norm_weight=dev(i["kw"]))
    assert torch.equal(pk[:, :, :S], k.view(B, S, Nkv, H).transpose(1, 2))


def test_rotary_position_out_of_range_leaves_the_token():
    i = rotary_inputs(ROTARY["three_axes"])
    i["pos"][1, 0, 2] = 97
    i["pos"][2, 1, 4] = -1
    op = GroupQueryAttention(8, 2)
    q, k = dev(i["q"]), dev(i["k"])
    op.rotary_axes(q, k, dev(i["pos"]), dev(i["cos"]), dev(i["sin"]), (16, 24, 24), out_query=q, out_key=k)
    assert op.block_status() == capi.GQA_DEVICE_BAD_ROTARY
    q, k = q.cpu().numpy(), k.cpu().numpy()
    for b, s in ((0, 2), (1, 4)):
        assert np.array_equal(q[b, s], i["q"][b, s]) and np.array_equal(k[b, s], i["k"][b, s])
    assert not np.array_equal(q[0, 1], i["q"][0, 1])


# ------------------------------------------------------------------ eviction

EVICT = {
    # B, Nkv, H, C, bs, C of into, totals, keep, recent, first
    "plain": (2, 2, 64, 300, 32, 128, (300, 170), 100, 20, 4),
    "short_and_empty": (4, 2, 64, 200, 16, 64, (0, 1, 64, 200), 64, 10, 2),
    "no_forced": (1, 3, 128, 500, 64, 256, (499,), 77, 0, 0),
    "all_forced": (1, 2, 48, 100, 16, 48, (100,), 40, 30, 10),
    "keep_one": (2, 1, 16, 100, 16, 16, (100, 2), 1, 0, 0),
    "keep_more_than_there_is": (2, 2, 64, 100, 64, 100, (100, 50), 5000, 20, 4),
    "long": (1, 2, 128, 70000, 128, 4096, (69999,), 3000, 100, 8),
    "two_ctas": (1, 1, 16, 40000, 64, 2048, (33001,), 2000, 1, 0),
    "several_rounds": (1, 1, 16, 300000, 256, 8192, (299999,), 8000, 100, 3),
    "block_256": (2, 2, 256, 600, 256, 512, (600, 513), 300, 1, 0),
}


@pytest.mark.parametrize("ties", [0, 1, 2])
@pytest.mark.parametrize("name", list(EVICT))
def test_evict(name, ties):
    B, Nkv, H, C, bs, Cto, totals, keep, recent, first = EVICT[name]
    rng = np.random.default_rng(11)
    cache = random_cache(rng, B, Nkv, C, H, bs)
    w = rng.random((B, Nkv, C)).astype(np.float32) ** 8
    if ties == 1:
        w = np.round(w * 3) / 3 * np.where(rng.random(w.shape) < 0.5, 1, -1).astype(np.float32)   # ties, -0, negatives
    if ties == 2:
        w[:] = 0
        w[..., ::7] = np.nan
        w[..., 3::11] = np.inf
        w[..., 4::13] = -np.inf
    w = w.astype(np.float32)
    into = random_cache(rng, B, Nkv, Cto, H, bs)
    iw = rng.random((B, Nkv, Cto)).astype(np.float32)
    seq = np.array(totals, np.int32) - 1
    op = GroupQueryAttention(Nkv, Nkv)
    g_into, g_iw = to_gpu_cache(into, bs), dev(iw)
    kept, lens = op.block_evict(to_gpu_cache(cache, bs), dev(w), dev(seq), max(1, max(totals)), keep, g_into, g_iw,
                                recent=recent, first=first)
    assert op.block_status() == 0
    rk, rl = ob.evict(cache, w, seq, keep, recent, first, bs, into, iw)
    assert np.array_equal(kept.cpu().numpy(), rk) and np.array_equal(lens.cpu().numpy(), rl)
    assert np.array_equal(g_iw.cpu().numpy(), iw, equal_nan=True)
    for n, a, b in zip(("kc", "vc", "ks", "vs"), from_gpu_cache(g_into), into):
        assert np.array_equal(a, b), (n, np.sum(a != b))


def test_evict_bad_length():
    rng = np.random.default_rng(1)
    cache, into = random_cache(rng, 2, 1, 64, 64, 16), random_cache(rng, 2, 1, 32, 64, 16)
    op = GroupQueryAttention(1, 1)
    g = to_gpu_cache(into, 16)
    kept = torch.full((2, 1, 20), 9, dtype=torch.int32, device="cuda")
    lens = torch.full((2,), 9, dtype=torch.int32, device="cuda")
    op.block_evict(to_gpu_cache(cache, 16), torch.zeros((2, 1, 64), device="cuda"),
                   torch.tensor([64, 40], dtype=torch.int32, device="cuda"), 64, 20, g, kept=kept, into_seqlens_k=lens)
    assert op.block_status() == capi.GQA_DEVICE_BAD_SEQLEN
    assert (kept[0] == 9).all() and lens.tolist() == [9, 19]
    assert np.array_equal(from_gpu_cache(g)[0][0], into[0][0])


# ------------------------------------------------------------------ together, and how calls may be made

def test_generation_with_eviction():
    """Rotate, step, evict, step: the loop of a serving program, against the oracle run the same way."""
    rng = np.random.default_rng(21)
    B, N, Nkv, H, bs, C = 2, 8, 2, 128, 16, 96
    sec, R = (16, 24, 24), 200
    ang = np.arange(R)[:, None] * 1e4 ** (-np.arange(64) / 64)
    cos, sin = np.cos(ang).astype(np.float16), np.sin(ang).astype(np.float16)
    op = GroupQueryAttention(N, Nkv)
    caches = [BlockCache.empty(B, Nkv, C, H, bs) for _ in range(2)]
    ws = [torch.zeros((B, Nkv, C), device="cuda") for _ in range(2)]
    ref = [[np.zeros((B, Nkv, C, H), np.int8) for _ in range(2)] + [np.zeros((B, Nkv, C // bs), np.float32) for _ in range(2)]
           for _ in range(2)]
    rws = [np.zeros((B, Nkv, C)) for _ in range(2)]
    lens = np.zeros(B, np.int64)
    seen = np.zeros(B, np.int64)
    cur = 0
    for n in (60, 1, 3, 20, 1, 1, 40, 2):
        if lens.max() + n > C:
            keep, recent, first = 40, 8, 2
            kept, seq = op.block_evict(caches[cur], ws[cur], dev((lens - 1).astype(np.int32)), C, keep, caches[1 - cur],
                                       ws[1 - cur], recent=recent, first=first)
            # weights differ from the oracle's by roundings: take the GPU's for its selection
            w = ws[cur].cpu().numpy()
            rk, rl = ob.evict(ref[cur], w, lens - 1, keep, recent, first, bs, ref[1 - cur], rws[1 - cur])
            assert np.array_equal(kept.cpu().numpy(), rk)
            cur, lens = 1 - cur, rl.astype(np.int64) + 1
            assert np.array_equal(seq.cpu().numpy(), lens - 1)
        q, k, v = (rng.standard_normal((B, n, m * H)).astype(np.float16) for m in (N, Nkv, Nkv))
        pos = np.stack([seen[:, None] + np.arange(n), seen[:, None] + np.arange(n) // 2, np.broadcast_to(np.arange(n), (B, n))])
        pos = pos.astype(np.int32)
        gq, gk = op.rotary_axes(dev(q), dev(k), dev(pos), dev(cos), dev(sin), sec)
        seen, lens = seen + n, lens + n
        before = ws[cur].cpu().numpy()
        out = op.block_forward(gq, gk, dev(v), dev((lens - 1).astype(np.int32)), int(lens.max()), caches[cur],
                               past_weights=ws[cur], present_weights=ws[cur])      # in place
        d = dict(dtype="f16", B=B, N=N, Nkv=Nkv, H=H, bs=bs, window=-1, softcap=0.0, sink=None, totals=lens, news=None,
                 q=gq.cpu().numpy(), k=gk.cpu().numpy(), v=v, cache=ref[cur], past_w=before)
        rout, mag, reach, rcache, _ = run_oracle(d)
        ref[cur] = rcache
        tol = output_tolerance(rout, mag, reach, "f16", H) + smallest_step(d, rcache)
        assert (np.abs(out.cpu().numpy() - rout) <= tol).all()
        for a, b in zip(from_gpu_cache(caches[cur]), ref[cur]):
            assert np.array_equal(a, b)
        w = ws[cur].cpu().numpy()
        for b in range(B):   # every query's probabilities add up to one
            grown = w[b, :, :lens[b]].sum() - before[b, :, :lens[b] - n].sum()
            assert abs(grown - n * N) < 1e-3 * n * N
    assert op.block_status() == 0


def test_guard_regions():
    """Nothing outside the outputs, the cache, the weights and the workspace's bytes is written."""
    for name in ("h96_ragged", "prompt_h128", "prefill_past", "chunk_h128_f32", "window"):
        d = make(CASES[name], seed=9)
        op = GroupQueryAttention(d["N"], d["Nkv"], softcap=float(d["softcap"]), local_window_size=d["window"])
        bufs = []

        def guarded(x):
            x = np.ascontiguousarray(x)
            buf = torch.full((x.nbytes + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
            buf[4096:4096 + x.nbytes].copy_(torch.from_numpy(x.view(np.uint8).reshape(-1)))
            bufs.append((buf, x.nbytes))
            return buf[4096:4096 + x.nbytes].view(torch.from_numpy(x.reshape(-1)[:0].copy()).dtype).view(x.shape)

        cache = BlockCache(*(guarded(x) for x in d["cache"]), d["bs"])
        pw, out = guarded(d["past_w"]), guarded(np.zeros_like(d["q"]))
        q, k, v, seq, news = dev(d["q"]), dev(d["k"]), dev(d["v"]), dev(d["totals"] - 1), dev(d["news"])
        total = int(d["totals"].max())
        op.block_forward(q, k, v, seq, total, cache, new_lens=news, head_sink=dev(d["sink"]), past_weights=pw,
                         present_weights=pw, output=out)
        # the same call on a workspace of exactly the size asked for
        rec = op._block_calls["forward"]
        ws = guarded(np.full(rec.nbytes, 0xFF, np.uint8))
        capi.gqa_block_forward(op.handle, *rec.structs, ws.data_ptr(), rec.nbytes, op._status_word(q.device),
                               torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        for buf, n in bufs:
            assert (buf[:4096] == 0xA5).all() and (buf[4096 + n:] == 0xA5).all()


def test_repeated_calls_give_the_same_bytes():
    for name in ("long_split", "prompt_h128", "softcap_f32"):
        d = make(CASES[name], seed=10)
        a, b = run_gpu(d), run_gpu(d)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[2], b[2])


def test_captured_graphs_and_streams():
    """Two graphs captured from one operator, replayed on two streams at once beside eager calls, new data each time."""
    d1, d2 = make(CASES["long_split"], seed=12), make(CASES["softcap_sink"], seed=13)
    op = GroupQueryAttention(4, 2)
    op2 = GroupQueryAttention(8, 2, softcap=5.0)
    run_gpu(d1, op), run_gpu(d2, op2)
    state = []
    for d, o in ((d1, op), (d2, op2), (d1, op)):
        s = dict(q=dev(d["q"]), k=dev(d["k"]), v=dev(d["v"]), seq=dev(d["totals"] - 1), cache=to_gpu_cache(d["cache"], d["bs"]),
                 pw=torch.full(d["past_w"].shape, 7.5, device="cuda"), w=dev(d["past_w"]), sink=dev(d["sink"]), d=d, op=o)
        s["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(s["graph"]):
            s["out"] = o.block_forward(s["q"], s["k"], s["v"], s["seq"], int(d["totals"].max()), s["cache"],
                                       head_sink=s["sink"], past_weights=s["w"], present_weights=s["pw"])
        state.append(s)
    streams = [torch.cuda.Stream() for _ in state]
    torch.cuda.synchronize()
    for rep in range(3):
        for s, st in zip(state, streams):
            with torch.cuda.stream(st):
                s["q"].copy_(dev(make(CASES["long_split" if s["d"] is d1 else "softcap_sink"], seed=30 + rep)["q"]))
                s["graph"].replay()
        eager = run_gpu(d1, op)
        torch.cuda.synchronize()
        check(d1, eager)
        for s in state:
            d = dict(s["d"])
            d["q"] = s["q"].cpu().numpy()
            check(d, (s["out"].cpu().numpy(), from_gpu_cache(s["cache"]), s["pw"].cpu().numpy(), s["op"]))


def test_two_threads_share_an_operator():
    import threading
    ds = [make(CASES["long_split"], seed=40 + i) for i in range(2)]
    op = GroupQueryAttention(4, 2)
    run_gpu(ds[0], op)
    got = [None, None]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                got[i] = run_gpu(ds[i], op)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    for d, g in zip(ds, got):
        check(d, g)


def test_one_operator_serves_changing_shapes():
    op = GroupQueryAttention(8, 2)
    for name in ("one_token", "one_token_f32", "prompt_h128", "attend_only", "chunk_h128_f32", "one_token"):
        d = make(CASES[name], seed=14)
        check(d, run_gpu(d, op))


def test_python_checks():
    op = GroupQueryAttention(8, 2)
    d = make(CASES["one_token"])
    q = dev(d["q"])
    with pytest.raises(ValueError):
        op.block_forward(q, dev(d["k"]).cpu(), dev(d["v"]), dev(d["totals"] - 1), 200, to_gpu_cache(d["cache"], 64))
    with pytest.raises(ValueError):
        op.block_forward(torch.cat((q, q), -1)[..., :q.shape[-1]], None, None, dev(d["totals"] - 1), 200, to_gpu_cache(d["cache"], 64))
    with pytest.raises(GqaError):
        op.block_forward(q, None, None, dev(d["totals"] - 1), 500, to_gpu_cache(d["cache"], 64))
    with pytest.raises(GqaError):
        op.block_forward(q, None, None, dev(d["totals"]).long().int(), 200, to_gpu_cache(d["cache"], 16))
