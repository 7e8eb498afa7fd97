"""Multi-axis rotary, block-scaled cache and eviction without a GPU: the oracle against closed forms, brute force and
invariants, and the host-side checks of the entry points (every refused call returns before any CUDA call; device
pointers are fake aligned addresses)."""

import math
import os
from fractions import Fraction

import numpy as np
import pytest
import torch

from grouped_query_attention_gb300 import GroupQueryAttention, capi
from oracle import block_cache as ob

INVALID, UNSUPPORTED, WORKSPACE = capi.GQA_ERR_INVALID_ARGUMENT, capi.GQA_ERR_UNSUPPORTED, capi.GQA_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(capi.LIB_PATH):
        from grouped_query_attention_gb300 import build
        build.build()
    return capi.load_library()


# ------------------------------------------------------------------ oracle

def test_axis_of_pair():
    assert ob.axis_of_pair([2, 1, 3], False) == [0, 0, 1, 2, 2, 2]
    assert ob.axis_of_pair([4, 2, 2], True) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert ob.axis_of_pair([8], True) == [0] * 8
    assert ob.axis_of_pair([0, 4], False) == [1] * 4


def test_rotary_axes_is_a_rotation_by_each_axis():
    rng = np.random.default_rng(0)
    B, S, heads, H = 2, 3, 2, 32
    x = rng.standard_normal((B, S, heads * H))
    pos = rng.integers(0, 20, (2, B, S))
    ang = np.arange(20)[:, None] * 0.1 ** np.arange(8)
    y = ob.rotary_axes(x, heads, pos, np.cos(ang), np.sin(ang), [3, 5]).reshape(B, S, heads, H)
    x = x.reshape(B, S, heads, H)
    z = (x[..., :8] + 1j * x[..., 8:16]) * np.exp(1j * np.concatenate(
        [ang[pos[0]][..., :3], ang[pos[1]][..., 3:]], -1))[:, :, None]
    assert np.allclose(y[..., :8], z.real, atol=1e-12) and np.allclose(y[..., 8:16], z.imag, atol=1e-12)
    assert np.array_equal(y[..., 16:], x[..., 16:])


def test_nearest_code_is_the_exact_quotients():
    rng = np.random.default_rng(1)
    s = np.float32(0.0237)
    x = np.concatenate([rng.standard_normal(400).astype(np.float32),
                        ((rng.integers(-127, 127, 200) + 0.5) * np.float64(s)).astype(np.float32)])   # beside borders
    want = [max(-127, min(127, round(Fraction(float(v)) / Fraction(float(s))))) for v in x]
    assert ob.nearest_code(x, s).tolist() == want
    assert ob.nearest_code(np.array([np.inf, -np.inf, np.nan]), s).tolist() == [127, -127, 0]
    assert ob.nearest_code(np.array([1.5, 2.5, -0.5]), np.float32(1)).tolist() == [2, 2, 0]


def test_append_grows_a_block_and_recodes_it():
    codes, scales = np.zeros((8, 16), np.int8), np.full(2, 9.0, np.float32)
    ob.append(codes, scales, np.full((2, 16), 1.0), 0, 4)
    s0 = scales[0]
    assert s0 == np.float32(np.float32(1) * np.float32(1 / np.float32(127))) and (codes[:2] == 127).all()
    ob.append(codes, scales, np.full((1, 16), 0.5), 2, 4)       # smaller: the scale stays
    assert scales[0] == s0 and (codes[:2] == 127).all() and scales[1] == 9.0
    ob.append(codes, scales, np.full((3, 16), 2.0), 3, 4)       # larger, and over the block's end
    assert (codes[:2] == 64).all() and (codes[3:6] == 127).all() and scales[1] == scales[0]


def test_step_matches_library_attention():
    rng = np.random.default_rng(2)
    B, S, N, Nkv, H, C, bs = 2, 3, 4, 2, 16, 20, 16
    cache = [rng.integers(-127, 128, (B, Nkv, C, H)).astype(np.int8) for _ in range(2)] + \
            [rng.uniform(0.01, 0.03, (B, Nkv, 2)).astype(np.float32) for _ in range(2)]
    q, k, v = (rng.standard_normal((B, S, n * H)).astype(np.float32) for n in (N, Nkv, Nkv))
    seq = np.array([10, 18])
    w = np.zeros((B, Nkv, C))
    out, _, _ = ob.step(q, k, v, seq, None, cache, bs, N, Nkv, weights=w)
    for b in range(B):
        t = seq[b] + 1
        kk = torch.tensor(np.stack([ob.values(cache[0][b, g], cache[2][b, g], t, bs) for g in range(Nkv)]))
        vv = torch.tensor(np.stack([ob.values(cache[1][b, g], cache[3][b, g], t, bs) for g in range(Nkv)]))
        qq = torch.tensor(q[b], dtype=torch.float64).view(S, N, H).transpose(0, 1)
        mask = torch.arange(t)[None] <= torch.arange(t - S, t)[:, None]
        ref = torch.nn.functional.scaled_dot_product_attention(
            qq, kk.repeat_interleave(2, 0), vv.repeat_interleave(2, 0), attn_mask=mask)
        assert np.allclose(out[b], ref.transpose(0, 1).reshape(S, -1).numpy(), atol=1e-12)
        assert np.allclose(w[b, :, :t].sum(-1), S * N // Nkv) and not w[b, :, t:].any()
    # appended rows are within half a step of what was stored
    for b in range(B):
        got = np.stack([ob.values(cache[0][b, g], cache[2][b, g], seq[b] + 1, bs)[-S:] for g in range(Nkv)], 1)
        assert np.abs(got - k[b].reshape(S, Nkv, H)).max() <= 0.5 * cache[2][b].max() + 1e-6


def test_kept_rows():
    w = np.array([5, 1, 3, 3, 0, 3, 9, 2], np.float32)
    assert ob.kept_rows(w, 8, 5, 1, 1).tolist() == [0, 2, 3, 6, 7]     # the tie goes to the lower rows
    assert ob.kept_rows(w, 4, 5, 1, 1).tolist() == [0, 1, 2, 3]
    assert ob.kept_rows(np.array([np.nan, 1, -1, np.nan, 0]), 5, 3, 0, 0).tolist() == [1, 2, 4]
    assert ob.kept_rows(w, 8, 3, 2, 1).tolist() == [0, 6, 7]


# ------------------------------------------------------------------ host checks

class Call:
    """Descriptors with fake addresses, 16 MiB apart, of the three entry points."""

    def __init__(self, dtype=capi.GQA_F16, B=2, S=3, N=8, Nkv=2, H=64, C=100, bs=32, **attrs):
        self.next = 1 << 32
        self.attrs = dict(num_heads=N, kv_num_heads=Nkv, **attrs)
        t, f, i = dtype, capi.GQA_F32, capi.GQA_I32
        nb = -(-C // bs)
        self.cache = self.make_cache(B, Nkv, C, H, bs, nb)
        self.inp, self.out = capi.GqaBlockInputs(), capi.GqaBlockOutputs()
        self.inp.query = self.t(t, (B, S, N * H))
        self.inp.key = self.t(t, (B, S, Nkv * H))
        self.inp.value = self.t(t, (B, S, Nkv * H))
        self.inp.seqlens_k = self.t(i, (B,))
        self.inp.total_sequence_length = C
        self.out.output = self.t(t, (B, S, N * H))
        self.rin, self.rout = capi.GqaRotaryInputs(), capi.GqaRotaryOutputs()
        self.rin.query, self.rin.key = self.t(t, (B, S, N * H)), self.t(t, (B, S, Nkv * H))
        self.rin.positions = self.t(i, (3, B, S))
        self.rin.cos_cache, self.rin.sin_cache = self.t(t, (50, 32)), self.t(t, (50, 32))
        self.rin.num_axes = 3
        self.rin.sections[0], self.rin.sections[1], self.rin.sections[2] = 8, 12, 12
        self.rout.query, self.rout.key = self.t(t, (B, S, N * H)), self.t(t, (B, S, Nkv * H))
        self.ev = capi.GqaEvictArgs()
        self.ev.source, self.ev.into = self.cache, self.make_cache(B, Nkv, 64, H, bs, 2)
        self.ev.weights = self.t(f, (B, Nkv, C))
        self.ev.seqlens_k, self.ev.into_seqlens_k = self.t(i, (B,)), self.t(i, (B,))
        self.ev.kept = self.t(i, (B, Nkv, 40))
        self.ev.total_sequence_length, self.ev.keep, self.ev.recent, self.ev.first = C, 40, 10, 2

    def t(self, dtype, shape):
        self.next += 1 << 36
        return capi.describe(self.next, dtype, shape)

    def make_cache(self, B, Nkv, C, H, bs, nb):
        c = capi.GqaBlockCache()
        c.key_codes, c.value_codes = self.t(capi.GQA_I8, (B, Nkv, C, H)), self.t(capi.GQA_I8, (B, Nkv, C, H))
        c.key_scales, c.value_scales = self.t(capi.GQA_F32, (B, Nkv, nb)), self.t(capi.GQA_F32, (B, Nkv, nb))
        c.block_size = bs
        return c

    def _run(self, fn):
        h = capi.gqa_create(capi.make_attrs(**self.attrs))
        try:
            return fn(h)
        finally:
            capi.gqa_destroy(h)

    def size(self):
        return self._run(lambda h: capi.gqa_block_workspace_size(h, self.cache, self.inp, self.out))

    def forward(self, ws=0, nbytes=0, status=0):
        return self._run(lambda h: capi.gqa_block_forward(h, self.cache, self.inp, self.out, ws, nbytes, status, 0))

    def rotary(self, status=0):
        return self._run(lambda h: capi.gqa_rotary_axes(h, self.rin, self.rout, status, 0))

    def evict(self, status=0):
        return self._run(lambda h: capi.gqa_block_evict(h, self.ev, status, 0))


def refused(fn, status):
    with pytest.raises(capi.GqaError) as e:
        fn()
    assert e.value.status == status, str(e.value)


def test_workspace_size_grows_with_weights():
    c = Call()
    plain = c.size()
    c.out.present_weights = c.t(capi.GQA_F32, (2, 2, 100))
    assert 0 < plain < c.size()
    c.inp.key = c.inp.value = capi.GqaTensor()     # attend only
    assert c.size() > 0


def test_plan_by_shape():
    """One token: the split over the keys. A prompt: the tensor-core prefill. A few rows on long ranges: the split."""
    def plan(**kw):
        c = Call(**kw)
        return c._run(lambda h: capi.gqa_block_describe_plan(h, c.cache, c.inp, c.out))

    one = plan(S=1, H=128, C=4096)
    assert one.regime == capi.GQA_REGIME_DECODE and one.launches == 3 and one.split_len == 32 and one.max_splits > 0
    prompt = plan(S=1024, H=128, C=1024, B=4)
    assert prompt.regime == capi.GQA_REGIME_PREFILL and prompt.launches == 2
    assert plan(S=16, H=128, C=32768, B=1).regime == capi.GQA_REGIME_DECODE
    assert plan(S=1024, H=96, C=1024, B=4).regime == capi.GQA_REGIME_PREFILL
    assert plan(S=1024, H=128, N=6, C=1024, B=4).regime == capi.GQA_REGIME_PREFILL    # a group of 3
    assert plan(S=1024, H=192, C=1024, B=4).regime == capi.GQA_REGIME_DECODE
    assert plan(S=60000, H=64, C=8_500_000, B=1).regime == capi.GQA_REGIME_DECODE     # past the prefill's grid


@pytest.mark.parametrize("attrs", [dict(causal=0), dict(do_rotary=1), dict(k_quant_type=1, v_quant_type=1),
                                   dict(local_window_size=4, sliding_window_cache=1)])
def test_forward_refuses_attributes(attrs):
    refused(Call(**attrs).size, UNSUPPORTED)


def _set(path, value):
    def change(c):
        obj = c
        *head, last = path.split(".")
        for p in head:
            obj = getattr(obj, p)
        setattr(obj, last, value(c) if callable(value) else value)
    return change


@pytest.mark.parametrize("change,status", [
    (_set("inp.query", capi.GqaTensor()), INVALID),
    (_set("inp.query", lambda c: c.t(capi.GQA_BF16, (2, 3, 512))), UNSUPPORTED),
    (_set("inp.query", lambda c: c.t(capi.GQA_I8, (2, 3, 512))), INVALID),
    (_set("inp.query", lambda c: c.t(capi.GQA_F16, (2, 3, 510))), INVALID),
    (_set("inp.query", lambda c: c.t(capi.GQA_F16, (2, 3, 8 * 24))), UNSUPPORTED),
    (_set("inp.query", lambda c: c.t(capi.GQA_F16, (2, 0, 512))), INVALID),
    (_set("inp.value", capi.GqaTensor()), INVALID),
    (_set("inp.key", lambda c: c.t(capi.GQA_F32, (2, 3, 128))), INVALID),
    (_set("inp.key", lambda c: c.t(capi.GQA_F16, (2, 2, 128))), INVALID),
    (_set("inp.seqlens_k", lambda c: c.t(capi.GQA_F32, (2,))), INVALID),
    (_set("inp.seqlens_k", lambda c: c.t(capi.GQA_I32, (3,))), INVALID),
    (_set("inp.new_lens", lambda c: c.t(capi.GQA_I32, (1,))), INVALID),
    (_set("inp.head_sink", lambda c: c.t(capi.GQA_F16, (2,))), INVALID),
    (_set("inp.past_weights", lambda c: c.t(capi.GQA_F32, (2, 2, 100))), INVALID),      # without present_weights
    (_set("out.present_weights", lambda c: c.t(capi.GQA_F32, (2, 2, 99))), INVALID),
    (_set("out.output", lambda c: c.t(capi.GQA_F32, (2, 3, 512))), INVALID),
    (_set("out.output", lambda c: c.inp.query), INVALID),                               # overlap
    (_set("out.output.data", lambda c: c.out.output.data + 8), INVALID),                # alignment
    (_set("cache.block_size", 24), INVALID),
    (_set("cache.block_size", 64), INVALID),                                            # scales are for 32
    (_set("cache.key_codes", lambda c: c.t(capi.GQA_U8, (2, 2, 100, 64))), INVALID),
    (_set("cache.value_codes", lambda c: c.t(capi.GQA_I8, (2, 2, 99, 64))), INVALID),
    (_set("cache.value_codes", lambda c: c.cache.key_codes), INVALID),                  # overlap
    (_set("cache.key_scales", lambda c: c.t(capi.GQA_F16, (2, 2, 4))), INVALID),
    (_set("inp.total_sequence_length", 101), INVALID),
    (_set("inp.total_sequence_length", 0), INVALID),
    (_set("cache.key_codes", lambda c: c.t(capi.GQA_I8, (2, 2, (1 << 30) + 1, 64))), INVALID),
])
def test_forward_refuses(change, status):
    c = Call()
    change(c)
    refused(c.size, status)
    refused(lambda: c.forward(1 << 20, 1 << 40), status)


def test_forward_refuses_workspace():
    c = Call()
    n = c.size()
    refused(lambda: c.forward(0, n), WORKSPACE)
    refused(lambda: c.forward((1 << 20) + 16, n), WORKSPACE)
    refused(lambda: c.forward(1 << 20, n - 1), WORKSPACE)
    refused(lambda: c.forward(1 << 20, n, status=(1 << 21) + 2), INVALID)


@pytest.mark.parametrize("change,status", [
    (_set("rin.query", capi.GqaTensor()), INVALID),
    (_set("rin.query", lambda c: c.t(capi.GQA_BF16, (2, 3, 512))), UNSUPPORTED),
    (_set("rin.key", lambda c: c.t(capi.GQA_F16, (2, 3, 64))), INVALID),
    (_set("rin.key", capi.GqaTensor()), INVALID),                                       # an output without its input
    (_set("rout.key", capi.GqaTensor()), INVALID),
    (_set("rout.query", lambda c: c.rin.key), INVALID),
    (_set("rout.key", lambda c: c.rout.query), INVALID),
    (_set("rin.num_axes", 0), INVALID),
    (_set("rin.num_axes", 9), INVALID),
    (_set("rin.positions", lambda c: c.t(capi.GQA_I32, (2, 2, 3))), INVALID),           # one axis short
    (_set("rin.interleaved", 2), INVALID),
    (_set("rin.positions", lambda c: c.t(capi.GQA_F32, (3, 2, 3))), INVALID),
    (_set("rin.cos_cache", lambda c: c.t(capi.GQA_F16, (50, 31))), INVALID),
    (_set("rin.sin_cache", lambda c: c.t(capi.GQA_F32, (50, 32))), INVALID),
    (_set("rin.q_norm_weight", lambda c: c.t(capi.GQA_F16, (64,))), INVALID),           # k_norm_weight missing
])
def test_rotary_refuses(change, status):
    c = Call()
    change(c)
    refused(c.rotary, status)


@pytest.mark.parametrize("N", [(1 << 24) + 1, 1 << 26])
def test_rotary_refuses_tokens_past_32_bits(N):
    refused(Call(B=1, S=1, N=N, Nkv=1).rotary, UNSUPPORTED)


@pytest.mark.parametrize("sections,interleaved,status", [((8, 12, 13), 0, INVALID), ((0, 0, 0), 0, INVALID),
                                                         ((40, -4, -4), 0, INVALID), ((4, 4, 4), 0, UNSUPPORTED),
                                                         ((8, 8, 16), 1, INVALID)])
def test_rotary_refuses_sections(sections, interleaved, status):
    c = Call()
    for i, n in enumerate(sections):
        c.rin.sections[i] = n
    c.rin.interleaved = interleaved
    refused(c.rotary, status)


@pytest.mark.parametrize("change,status", [
    (_set("ev.keep", 0), INVALID),
    (_set("ev.keep", 41), INVALID),                                                     # kept is for 40
    (_set("ev.recent", 39), INVALID),
    (_set("ev.first", -1), INVALID),
    (_set("ev.recent", -1), INVALID),
    (_set("ev.total_sequence_length", 0), INVALID),
    (_set("ev.total_sequence_length", 101), INVALID),
    (_set("ev.into.block_size", 16), INVALID),
    (_set("ev.into", lambda c: c.make_cache(2, 2, 32, 64, 32, 1)), INVALID),            # too small for keep
    (_set("ev.into", lambda c: c.make_cache(2, 1, 64, 64, 32, 2)), INVALID),
    (_set("ev.into", lambda c: c.ev.source), INVALID),                                  # in place
    (_set("ev.weights", lambda c: c.t(capi.GQA_F16, (2, 2, 100))), INVALID),
    (_set("ev.into_weights", lambda c: c.ev.weights), INVALID),
    (_set("ev.into_seqlens_k", lambda c: c.ev.seqlens_k), INVALID),
    (_set("ev.kept", capi.GqaTensor()), INVALID),
    (_set("ev.fill_skipped", 4), INVALID),
    (_set("ev.fill_skipped", -1), INVALID),
])
def test_evict_refuses(change, status):
    c = Call()
    change(c)
    refused(c.evict, status)


def test_null_arguments():
    lib = capi.load_library()
    c = Call()
    assert lib.gqa_rotary_axes(None, c.rin, c.rout, None, None) == INVALID
    assert lib.gqa_block_forward(None, c.cache, c.inp, c.out, None, 0, None, None) == INVALID
    assert lib.gqa_block_evict(None, c.ev, None, None) == INVALID
    h = capi.gqa_create(capi.make_attrs(8, 2))
    assert lib.gqa_rotary_axes(h, None, c.rout, None, None) == INVALID
    assert lib.gqa_block_workspace_size(h, c.cache, c.inp, c.out, None) == INVALID
    assert lib.gqa_block_evict(h, None, None, None) == INVALID
    capi.gqa_destroy(h)


def test_python_refuses_tensors_off_the_gpu_or_strided():
    op = GroupQueryAttention(2, 1)
    x = torch.zeros(1, 1, 128)
    with pytest.raises(ValueError):
        op.rotary_axes(x, None, torch.zeros(1, 1, 1, dtype=torch.int32), torch.zeros(4, 32), torch.zeros(4, 32), [32])
    with pytest.raises(ValueError):
        from grouped_query_attention_gb300.block_cache import tensor_desc
        tensor_desc(torch.zeros(4, 4).t())


def test_scale_attribute_default_is_the_frameworks():
    assert math.isclose(1 / math.sqrt(64), 0.125)
    rng = np.random.default_rng(3)
    cache = [rng.integers(-127, 128, (1, 1, 16, 16)).astype(np.int8) for _ in range(2)] + [np.ones((1, 1, 1), np.float32) * 0.02] * 2
    q = rng.standard_normal((1, 1, 16)).astype(np.float32)
    a, _, _ = ob.step(q, None, None, np.array([9]), None, cache, 16, 1, 1)
    b, _, _ = ob.step(q, None, None, np.array([9]), None, cache, 16, 1, 1, scale=0.25)
    assert np.array_equal(a, b)


def test_python_integers_past_32_bits_are_refused():
    from grouped_query_attention_gb300.block_cache import _int32
    assert [_int32(v, "x") for v in (-2 ** 31, 0, torch.tensor(5), np.int64(2 ** 31 - 1))] == [-2 ** 31, 0, 5, 2 ** 31 - 1]
    for v in (2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="total_sequence_length"):
            _int32(v, "total_sequence_length")


@pytest.mark.parametrize("B,Nkv,S,T", [(1, 8, 4096, 300), (1, 1, 4096, 1000), (8, 8, 4096, 1000), (64, 2, 1024, 100)])
def test_plan_of_padded_prompts(B, Nkv, S, T):
    """Positions behind total_sequence_length are padding: the plan is that of a prompt of T tokens."""
    plans = []
    for s in (S, T):
        c = Call(B=B, S=s, N=4 * Nkv, Nkv=Nkv, H=128, C=4096, bs=64)
        c.inp.total_sequence_length = T
        plans.append(c._run(lambda h: capi.gqa_block_describe_plan(h, c.cache, c.inp, c.out)).regime)
    assert plans == [capi.GQA_REGIME_PREFILL] * 2
