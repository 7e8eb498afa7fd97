"""Drafted-token operators without a GPU: the oracle against library attention, a chain against plain causal steps,
the verification against the distribution it has to keep, and the host-side checks of the entry points (every refused
call returns before any CUDA call; device pointers are fake aligned addresses)."""

import ctypes
import os

import numpy as np
import pytest
import torch

from grouped_query_attention_gb300 import GroupQueryAttention, capi
from oracle import tree as ot

INVALID, UNSUPPORTED, WORKSPACE = capi.GQA_ERR_INVALID_ARGUMENT, capi.GQA_ERR_UNSUPPORTED, capi.GQA_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(capi.LIB_PATH):
        from grouped_query_attention_gb300 import build
        build.build()
    return capi.load_library()


# ------------------------------------------------------------------ oracle

def _case(rng, B=2, S=5, N=4, Nkv=2, H=16, C=30):
    q, k, v = (rng.standard_normal((B, S, n * H)).astype(np.float32) for n in (N, Nkv, Nkv))
    pk, pv = (rng.standard_normal((B, Nkv, C, H)).astype(np.float32) for _ in range(2))
    return q, k, v, pk, pv


@pytest.mark.parametrize("window", [-1, 3])
def test_forward_matches_library_attention(window):
    rng = np.random.default_rng(0)
    q, k, v, pk, pv = _case(rng)
    parents = np.array([[-1, 0, 0, 1, 3], [-1, 0, 1, 1, -1]])
    seq, lens = np.array([14, 9]), np.array([5, 5])
    old = pk.copy()
    out, _, _ = ot.forward(q, k, v, parents, seq, None, pk, pv, 4, 2, window=window)
    for b in range(2):
        t = seq[b] + 1
        past = t - lens[b]
        assert np.array_equal(pk[b, :, :past], old[b, :, :past]) and np.array_equal(pk[b, :, t:], old[b, :, t:])
        assert np.array_equal(pk[b, :, past:t], k[b].reshape(5, 2, 16).transpose(1, 0, 2))
        mask = torch.zeros(5, t, dtype=torch.bool)
        depth = []
        for i in range(5):
            a = parents[b, i]
            depth.append(0 if a < 0 else depth[a] + 1)
            if a >= 0:
                mask[i, past:] = mask[a, past:]
            mask[i, past + i] = True
            mask[i, :past] = True
        for i in range(5):
            if window >= 0:
                for j in range(t):
                    at = j - past if j < past else depth[j - past]
                    mask[i, j] &= bool(at >= depth[i] - window)
        qq = torch.tensor(q[b], dtype=torch.float64).view(5, 4, 16).transpose(0, 1)
        kk, vv = (torch.tensor(x[b, :, :t], dtype=torch.float64).repeat_interleave(2, 0) for x in (pk, pv))
        ref = torch.nn.functional.scaled_dot_product_attention(qq, kk, vv, attn_mask=mask)
        assert np.allclose(out[b], ref.transpose(0, 1).reshape(5, -1).numpy(), atol=1e-12)


def test_a_chain_is_causal_attention():
    """Nodes in a row see what single causal steps see; rows before the sequence's end do not change."""
    from oracle import gqa_forward
    rng = np.random.default_rng(1)
    q, k, v, pk, pv = _case(rng, S=4)
    parents = np.array([[-1, 0, 1, 2]])
    seq = np.array([12, 29])
    k2, v2 = pk.copy(), pv.copy()
    out, _, _ = ot.forward(q, k, v, parents, seq, None, k2, v2, 4, 2)
    for b in range(2):
        inp = dict(query=q[b:b + 1], key=k[b:b + 1], value=v[b:b + 1], past_key=pk[b:b + 1], past_value=pv[b:b + 1],
                   seqlens_k=seq[b:b + 1].astype(np.int32), total_sequence_length=np.array([seq[b] + 1], np.int32))
        ref = gqa_forward(inp, dict(num_heads=4, kv_num_heads=2), pk[b:b + 1].copy(), pv[b:b + 1].copy(), True)
        assert np.allclose(out[b:b + 1], ref["output_f64"], atol=1e-12)
        assert np.array_equal(k2[b:b + 1], ref["present_key"])


def test_bad_parents_are_roots():
    par = np.array([[0, 0, 2, -2, 7]])
    assert [ot.ancestors(par, 0, i) for i in range(5)] == [[0], [1, 0], [2], [3], [4]]


def _emitted(path, lens, token, tokens):
    """The token behind the root in every sequence: the first accepted draft, or the drawn one."""
    return [int(tokens[b, path[b, 1]]) if lens[b] > 1 else int(token[b]) for b in range(len(lens))]


@pytest.mark.parametrize("drafts", [True, False])
def test_verification_keeps_the_targets_distribution(drafts):
    """20000 sequences of a root with three children: the token behind the root is distributed as the target's row.
    (99.99 % of a binomial share of 20000 lie within 3.9 standard deviations, 0.0138 at most.)"""
    rng = np.random.default_rng(2)
    n, V = 20000, 5
    p = np.array([0.45, 0.3, 0.15, 0.1, 0.0])
    q = np.array([0.1, 0.5, 0.1, 0.1, 0.2])
    parents = np.array([[-1, 0, 0, 0]])
    tokens = rng.choice(V, (n, 4), p=q) if drafts else np.tile([0, 1, 0, 3], (n, 1))
    rows = np.broadcast_to(p, (n, 4, V))
    path, lens, token = ot.verify(tokens, parents, rows, rng.random((n, 4)), rng.random(n),
                                  np.broadcast_to(q, (n, 4, V)) if drafts else None)
    share = np.bincount(_emitted(path, lens, token, tokens), minlength=V) / n
    assert np.abs(share - p).max() < 0.0138
    assert 0.3 < (lens > 1).mean() < 0.95 and path.max() <= 3


def test_verification_by_hand():
    p = np.zeros((1, 4, 4))
    p[0, 0] = [0.5, 0.25, 0.25, 0.0]
    p[0, 2] = [0.0, 0.0, 0.0, 1.0]
    q = np.full((1, 4, 4), 0.25)
    tok, par = np.array([[9, 3, 0, 1]]), np.array([[-1, 0, 0, 0]])
    # node 1 (token 3) has p = 0; then r = [1/4, 0, 0, 0], Z = 1/4: node 2 (token 0) passes every number below 1
    path, lens, token = ot.verify(tok, par, p, np.full((1, 4), 0.999), np.array([0.3]), q)
    assert path.tolist() == [[0, 2, -1, -1]] and lens.tolist() == [2] and token.tolist() == [3]
    # certain drafts: node 1 fails, node 2 fails at u >= 1/2, node 3 (token 1) is tested on [0, 1/4, 1/4, 0], Z = 1/2
    path, lens, token = ot.verify(tok, par, p, np.array([[0, 0, 0.5, 0.5]]), np.array([0.0]), None)
    assert path.tolist() == [[0, -1, -1, -1]] and token.tolist() == [2]
    path, lens, token = ot.verify(tok, par, p, np.array([[0, 0, 0.5, 0.49]]), np.array([0.0]), None, np.array([3]))
    assert path.tolist() == [[0, -1, -1, -1]] and token.tolist() == [1]     # node 3 is padding; [0, 1/4, 1/4, 0] is left
    # nothing left (q covers p): the target's own row
    path, lens, token = ot.verify(np.array([[9, 3]]), np.array([[-1, 0]]), p[:, [0, 0]], np.zeros((1, 2)), np.array([0.6]),
                                  np.full((1, 2, 4), 0.5))
    assert path.tolist() == [[0, -1]] and token.tolist() == [1]
    assert ot.verify(tok, par, p, p[0, :1] * 0, np.zeros(1), None, np.array([0]))[2].tolist() == [-1]
    assert ot.verify(tok, par, p * np.nan, p[0, :1] * 0, np.zeros(1), None)[2].tolist() == [-1]


def test_accept_moves_rows():
    c = [np.arange(2 * 1 * 10 * 2, dtype=np.float32).reshape(2, 1, 10, 2) for _ in range(2)]
    path = np.array([[0, 2, 3, -1], [0, 2, 2, -1]])
    out = ot.accept(c, path, np.array([3, 3]), np.array([6, 7]))
    assert out.tolist() == [5, -1]
    assert c[0][0, 0, :, 0].tolist() == [0, 2, 4, 6, 10, 12, 12, 14, 16, 18]
    assert c[1][1, 0, :, 0].tolist() == list(range(20, 40, 2))


# ------------------------------------------------------------------ host checks

class Call:
    """Descriptors with fake addresses, 64 GiB apart, of the three entry points."""

    def __init__(self, dtype=capi.GQA_F16, B=2, S=6, N=8, Nkv=2, H=64, C=100, V=1000, layers=2, **attrs):
        self.next = 1 << 32
        self.attrs = dict(num_heads=N, kv_num_heads=Nkv, **attrs)
        t, f, i = dtype, capi.GQA_F32, capi.GQA_I32
        self.inp, self.out = capi.GqaTreeInputs(), capi.GqaTreeOutputs()
        self.inp.query = self.t(t, (B, S, N * H))
        self.inp.key, self.inp.value = self.t(t, (B, S, Nkv * H)), self.t(t, (B, S, Nkv * H))
        self.inp.parents, self.inp.seqlens_k = self.t(i, (B, S)), self.t(i, (B,))
        self.inp.total_sequence_length = C
        self.out.output = self.t(t, (B, S, N * H))
        self.out.present_key, self.out.present_value = self.t(t, (B, Nkv, C, H)), self.t(t, (B, Nkv, C, H))
        v = self.ver = capi.GqaVerifyArgs()
        v.tokens, v.parents = self.t(i, (B, S)), self.t(i, (1, S))
        v.target_probs, v.draft_probs = self.t(f, (B, S, V)), self.t(f, (B, S, V))
        v.accept_uniforms, v.sample_uniforms = self.t(f, (B, S)), self.t(f, (B,))
        v.path, v.path_lens, v.next_token = self.t(i, (B, S)), self.t(i, (B,)), self.t(i, (B,))
        a = self.acc = capi.GqaAcceptArgs()
        a.cache = self.t(t, (B, Nkv, C, H))
        self.keys, self.values = ((ctypes.c_void_p * layers)(*(self.t(t, (1,)).data for _ in range(layers))) for _ in range(2))
        a.present_keys, a.present_values, a.num_layers = self.keys, self.values, layers
        a.path, a.path_lens, a.seqlens_k, a.into_seqlens_k = self.t(i, (B, S)), self.t(i, (B,)), self.t(i, (B,)), self.t(i, (B,))

    def t(self, dtype, shape):
        self.next += 1 << 36
        return capi.describe(self.next, dtype, shape)

    def _run(self, fn):
        h = capi.gqa_create(capi.make_attrs(**self.attrs))
        try:
            return fn(h)
        finally:
            capi.gqa_destroy(h)

    def size(self):
        return self._run(lambda h: capi.gqa_tree_workspace_size(h, self.inp, self.out))

    def forward(self, ws=0, nbytes=0, status=0):
        return self._run(lambda h: capi.gqa_tree_forward(h, self.inp, self.out, ws, nbytes, status, 0))

    def verify(self, status=0):
        return self._run(lambda h: capi.gqa_tree_verify(h, self.ver, status, 0))

    def accept(self, status=0):
        return self._run(lambda h: capi.gqa_tree_accept(h, self.acc, status, 0))


def refused(fn, status):
    with pytest.raises(capi.GqaError) as e:
        fn()
    assert e.value.status == status, str(e.value)


def _set(path, value):
    def change(c):
        obj = c
        *head, last = path.split(".")
        for p in head:
            obj = getattr(obj, p)
        setattr(obj, last, value(c) if callable(value) else value)
    return change


def test_plan():
    c = Call()
    plan = c._run(lambda h: capi.gqa_tree_describe_plan(h, c.inp, c.out))
    assert plan.launches == 2 and plan.workspace_bytes == c.size() > 0 and plan.max_splits > 0 and plan.split_len > 0


@pytest.mark.parametrize("kw", [dict(B=64, S=512, N=64, Nkv=8, H=128, C=8192), dict(B=1, S=1, N=1, Nkv=1, H=16, C=1),
                                dict(B=1, S=26, N=16, Nkv=2, H=64, C=2_000_000),
                                dict(dtype=capi.GQA_F32, B=8, S=512, N=128, Nkv=1, H=256, C=4096)])
def test_workspace_stays_small(kw):
    assert 0 < Call(**kw).size() <= 128 << 20


@pytest.mark.parametrize("attrs", [dict(causal=0), dict(do_rotary=1), dict(k_quant_type=1, v_quant_type=1),
                                   dict(local_window_size=4, sliding_window_cache=1)])
def test_forward_refuses_attributes(attrs):
    refused(Call(**attrs).size, UNSUPPORTED)


@pytest.mark.parametrize("change,status", [
    (_set("inp.query", capi.GqaTensor()), INVALID),
    (_set("inp.query", lambda c: c.t(capi.GQA_BF16, (2, 6, 512))), UNSUPPORTED),
    (_set("inp.query", lambda c: c.t(capi.GQA_I8, (2, 6, 512))), INVALID),
    (_set("inp.query", lambda c: c.t(capi.GQA_F16, (2, 6, 510))), INVALID),
    (_set("inp.query", lambda c: c.t(capi.GQA_F16, (2, 6, 8 * 24))), UNSUPPORTED),
    (_set("inp.query", lambda c: c.t(capi.GQA_F16, (2, 0, 512))), INVALID),
    (_set("inp.query", lambda c: c.t(capi.GQA_F16, (2, 513, 512))), UNSUPPORTED),       # too many nodes
    (_set("inp.key", capi.GqaTensor()), INVALID),
    (_set("inp.value", capi.GqaTensor()), INVALID),
    (_set("inp.key", lambda c: c.t(capi.GQA_F32, (2, 6, 128))), INVALID),
    (_set("inp.key", lambda c: c.t(capi.GQA_F16, (2, 5, 128))), INVALID),
    (_set("inp.parents", capi.GqaTensor()), INVALID),
    (_set("inp.parents", lambda c: c.t(capi.GQA_I32, (3, 6))), INVALID),
    (_set("inp.parents", lambda c: c.t(capi.GQA_I32, (2, 5))), INVALID),
    (_set("inp.parents", lambda c: c.t(capi.GQA_I32, (6,))), INVALID),
    (_set("inp.parents", lambda c: c.t(capi.GQA_F32, (2, 6))), INVALID),
    (_set("inp.seqlens_k", lambda c: c.t(capi.GQA_F32, (2,))), INVALID),
    (_set("inp.seqlens_k", lambda c: c.t(capi.GQA_I32, (3,))), INVALID),
    (_set("inp.new_lens", lambda c: c.t(capi.GQA_I32, (1,))), INVALID),
    (_set("inp.head_sink", lambda c: c.t(capi.GQA_F16, (2,))), INVALID),
    (_set("out.output", lambda c: c.t(capi.GQA_F32, (2, 6, 512))), INVALID),
    (_set("out.output", lambda c: c.inp.query), INVALID),                               # overlap
    (_set("out.output.data", lambda c: c.out.output.data + 8), INVALID),                # alignment
    (_set("out.present_key", lambda c: c.t(capi.GQA_F32, (2, 2, 100, 64))), INVALID),   # another dtype
    (_set("out.present_key", lambda c: c.t(capi.GQA_I8, (2, 2, 100, 64))), INVALID),
    (_set("out.present_key", lambda c: c.t(capi.GQA_F16, (2, 8, 100, 64))), INVALID),
    (_set("out.present_value", lambda c: c.t(capi.GQA_F16, (2, 2, 99, 64))), INVALID),
    (_set("out.present_value", lambda c: c.out.present_key), INVALID),                  # overlap
    (_set("out.present_value", capi.GqaTensor()), INVALID),
    (_set("inp.total_sequence_length", 101), INVALID),
    (_set("inp.total_sequence_length", 0), INVALID),
])
def test_forward_refuses(change, status):
    c = Call()
    change(c)
    refused(c.size, status)
    refused(lambda: c.forward(1 << 20, 1 << 40), status)


def test_forward_refuses_large_caches():
    refused(Call(C=(1 << 30) + 1).size, UNSUPPORTED)
    refused(Call(B=65536, Nkv=1, N=1, S=1).size, UNSUPPORTED)


def test_forward_refuses_workspace():
    c = Call()
    n = c.size()
    refused(lambda: c.forward(0, n), WORKSPACE)
    refused(lambda: c.forward((1 << 20) + 16, n), WORKSPACE)
    refused(lambda: c.forward(1 << 20, n - 1), WORKSPACE)
    refused(lambda: c.forward(1 << 20, n, status=(1 << 21) + 2), INVALID)


@pytest.mark.parametrize("change,status", [
    (_set("ver.target_probs", capi.GqaTensor()), INVALID),
    (_set("ver.target_probs", lambda c: c.t(capi.GQA_BF16, (2, 6, 1000))), UNSUPPORTED),
    (_set("ver.target_probs", lambda c: c.t(capi.GQA_I32, (2, 6, 1000))), INVALID),
    (_set("ver.target_probs", lambda c: c.t(capi.GQA_F32, (2, 6, 0))), INVALID),
    (_set("ver.target_probs", lambda c: c.t(capi.GQA_F32, (2, 513, 10))), UNSUPPORTED),
    (_set("ver.draft_probs", lambda c: c.t(capi.GQA_F16, (2, 6, 1000))), INVALID),      # another dtype
    (_set("ver.draft_probs", lambda c: c.t(capi.GQA_F32, (2, 6, 999))), INVALID),
    (_set("ver.tokens", lambda c: c.t(capi.GQA_I32, (2, 5))), INVALID),
    (_set("ver.tokens", capi.GqaTensor()), INVALID),
    (_set("ver.parents", lambda c: c.t(capi.GQA_I32, (6,))), INVALID),
    (_set("ver.accept_uniforms", lambda c: c.t(capi.GQA_F16, (2, 6))), INVALID),
    (_set("ver.accept_uniforms", lambda c: c.t(capi.GQA_F32, (2, 1))), INVALID),
    (_set("ver.sample_uniforms", lambda c: c.t(capi.GQA_F32, (2, 6))), INVALID),
    (_set("ver.new_lens", lambda c: c.t(capi.GQA_I32, (3,))), INVALID),
    (_set("ver.path", lambda c: c.ver.tokens), INVALID),                                # overlap
    (_set("ver.path", lambda c: c.t(capi.GQA_I32, (2, 7))), INVALID),
    (_set("ver.path_lens", capi.GqaTensor()), INVALID),
    (_set("ver.next_token", lambda c: c.ver.path_lens), INVALID),
    (_set("ver.target_probs.data", lambda c: c.ver.target_probs.data + 4), INVALID),
])
def test_verify_refuses(change, status):
    c = Call()
    change(c)
    refused(c.verify, status)
    refused(lambda: Call().verify(status=2), INVALID)


@pytest.mark.parametrize("change,status", [
    (_set("acc.num_layers", 0), INVALID),
    (_set("acc.num_layers", 129), INVALID),
    (_set("acc.path", lambda c: c.t(capi.GQA_I32, (3, 6))), INVALID),
    (_set("acc.path", lambda c: c.t(capi.GQA_I32, (2, 513))), UNSUPPORTED),
    (_set("acc.path", lambda c: c.t(capi.GQA_I32, (2, 0))), INVALID),
    (_set("acc.path_lens", lambda c: c.t(capi.GQA_I32, (2, 6))), INVALID),
    (_set("acc.seqlens_k", capi.GqaTensor()), INVALID),
    (_set("acc.new_lens", lambda c: c.t(capi.GQA_F32, (2,))), INVALID),
    (_set("acc.into_seqlens_k", lambda c: c.acc.seqlens_k), INVALID),                   # overlap
    (lambda c: c.keys.__setitem__(1, c.keys[0]), INVALID),                              # one cache twice
    (lambda c: c.values.__setitem__(0, c.keys[1]), INVALID),
    (lambda c: c.values.__setitem__(0, c.keys[1] + 2 * 2 * 100 * 64 * 2 - 16), INVALID),   # another's last bytes
    (lambda c: setattr(c.acc.path, "data", c.keys[1] + 64), INVALID),
    (lambda c: setattr(c.acc.into_seqlens_k, "data", c.values[1]), INVALID),
    (lambda c: c.keys.__setitem__(1, c.keys[1] + 8), INVALID),                          # alignment
    (lambda c: c.values.__setitem__(1, None), INVALID),
    (_set("acc.cache", lambda c: c.t(capi.GQA_I8, (2, 2, 100, 64))), INVALID),
    (_set("acc.cache", lambda c: c.t(capi.GQA_BF16, (2, 2, 100, 64))), UNSUPPORTED),
    (_set("acc.cache", lambda c: c.t(capi.GQA_F16, (2, 4, 100, 64))), INVALID),
    (_set("acc.cache", lambda c: c.t(capi.GQA_F16, (2, 2, 100, 24))), UNSUPPORTED),
    (_set("acc.cache", lambda c: c.t(capi.GQA_F16, (2, 2, 6400))), INVALID),
])
def test_accept_refuses(change, status):
    c = Call()
    change(c)
    refused(c.accept, status)
    refused(lambda: Call().accept(status=2), INVALID)


def test_null_arguments():
    lib = capi.load_library()
    c = Call()
    assert lib.gqa_tree_forward(None, c.inp, c.out, None, 0, None, None) == INVALID
    assert lib.gqa_tree_verify(None, c.ver, None, None) == INVALID
    assert lib.gqa_tree_accept(None, c.acc, None, None) == INVALID
    h = capi.gqa_create(capi.make_attrs(8, 2))
    assert lib.gqa_tree_workspace_size(h, c.inp, c.out, None) == INVALID
    assert lib.gqa_tree_describe_plan(h, c.inp, None, capi.GqaPlanInfo()) == INVALID
    assert lib.gqa_tree_verify(h, None, None, None) == INVALID
    c.acc.present_keys = None
    assert lib.gqa_tree_accept(h, c.acc, None, None) == INVALID
    capi.gqa_destroy(h)


def test_python_refuses_tensors_off_the_gpu_and_odd_lists():
    op = GroupQueryAttention(2, 1)
    x, i = torch.zeros(1, 1, 128), torch.zeros(1, 1, dtype=torch.int32)
    cache = torch.zeros(1, 1, 4, 64)
    with pytest.raises(ValueError):
        op.tree_forward(x, x[..., :64].contiguous(), x[..., :64].contiguous(), i, i[0], 1, cache, cache.clone())
    with pytest.raises(ValueError):
        op.tree_verify(i, i, torch.zeros(1, 1, 8), torch.zeros(1, 1), torch.zeros(1))
    with pytest.raises(ValueError):
        op.tree_accept([(cache, cache)], i, i[0], i[0])
    for caches in ([], [(cache,)], [(cache, cache)] * 129, [(cache, cache, cache), (cache,)], [(cache, cache[..., :32].contiguous())],
                   [(cache, cache.half())]):
        with pytest.raises(ValueError, match="caches"):
            op.tree_accept(caches, i, i[0], i[0])
    with pytest.raises(ValueError, match="contiguous"):
        op.tree_accept([(cache, cache.transpose(2, 3))], i, i[0], i[0])
