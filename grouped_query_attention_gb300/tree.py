"""Attention for drafted tokens, their verification and the move of the accepted cache rows for torch tensors.

Argument marshalling only: the entry points are ``gqa_tree_forward``, ``gqa_tree_verify`` and ``gqa_tree_accept`` of
include/gqa.h, which also states shapes, types and semantics.
"""

from __future__ import annotations

import ctypes
from itertools import chain
from operator import attrgetter

import torch

from . import capi
from .block_cache import _current_device, _int32, _raw_stream, tensor_desc

_shape, _dtype = attrgetter("shape"), attrgetter("dtype")


class TreeOps:
    """The drafted-token methods of ``GroupQueryAttention``; streams, workspaces and the status word as in
    ``BlockCacheOps``."""

    def tree_forward(self, query, key, value, parents, seqlens_k, total_sequence_length, present_key, present_value,
                     new_lens=None, head_sink=None, output=None):
        """Store the nodes' key / value behind the cached rows of present_key / present_value (in place) and attend
        from every node to the cached rows, its ancestors and itself. Returns ``output``. parents: (B, S), or (1, S)
        for one tree of all sequences; -1 for the root. total_sequence_length is an upper bound of the lengths.
        Nothing of a sequence of a bad length is written (block_status tells), also not in an output made here."""
        index = query.get_device()
        if index >= 0 and index != _current_device():
            with torch.cuda.device(index):
                return self.tree_forward(query, key, value, parents, seqlens_k, total_sequence_length, present_key,
                                         present_value, new_lens, head_sink, output)
        if output is None:
            output = torch.empty_like(query, memory_format=torch.contiguous_format)

        def build():
            inp, out = capi.GqaTreeInputs(), capi.GqaTreeOutputs()
            return (inp, out), [inp.query, inp.key, inp.value, inp.parents, inp.seqlens_k, inp.new_lens, inp.head_sink,
                                out.output, out.present_key, out.present_value]

        with self._block_lock:
            rec = self._bind("tree_forward", (query, key, value, parents, seqlens_k, new_lens, head_sink, output,
                                              present_key, present_value), None, build)
            inp = rec.structs[0]
            if rec.nbytes is None or inp.total_sequence_length != total_sequence_length:
                rec.nbytes = None
                inp.total_sequence_length = _int32(total_sequence_length, "total_sequence_length")
                rec.nbytes = capi.gqa_tree_workspace_size(self.handle, *rec.structs)
            stream = _raw_stream(index)
            status = self._block_status_ptr.get(index) or self._status_word(query.device)
            ws = self._scratch(rec.nbytes, index, stream)
            capi.gqa_tree_forward(self.handle, *rec.refs, ws.data_ptr(), ws.numel(), status, stream)
        return output

    def tree_verify(self, tokens, parents, target_probs, accept_uniforms, sample_uniforms, draft_probs=None,
                    new_lens=None, path=None, path_lens=None, next_token=None):
        """Test the drafted tokens against the target's probabilities with the given random numbers. Returns (path,
        path_lens, next_token): the accepted nodes from the root on (-1 behind the last), their number, and the token
        drawn behind the last one. Without draft_probs every draft counts as certain (a most likely token)."""
        index = tokens.get_device()
        if index >= 0 and index != _current_device():
            with torch.cuda.device(index):
                return self.tree_verify(tokens, parents, target_probs, accept_uniforms, sample_uniforms, draft_probs,
                                        new_lens, path, path_lens, next_token)
        if path is None:
            path = torch.empty_like(tokens, memory_format=torch.contiguous_format)
        if path_lens is None:
            path_lens = tokens.new_empty(tokens.shape[0])
        if next_token is None:
            next_token = tokens.new_empty(tokens.shape[0])

        def build():
            a = capi.GqaVerifyArgs()
            return (a,), [a.tokens, a.parents, a.target_probs, a.draft_probs, a.accept_uniforms, a.sample_uniforms,
                          a.new_lens, a.path, a.path_lens, a.next_token]

        with self._block_lock:
            rec = self._bind("tree_verify", (tokens, parents, target_probs, draft_probs, accept_uniforms,
                                             sample_uniforms, new_lens, path, path_lens, next_token), None, build)
            status = self._block_status_ptr.get(index) or self._status_word(tokens.device)
            capi.gqa_tree_verify(self.handle, *rec.refs, status, _raw_stream(index))
        return path, path_lens, next_token

    def tree_accept(self, caches, path, path_lens, seqlens_k, new_lens=None, into_seqlens_k=None):
        """Move the rows of the accepted nodes together in ``caches``, the (present_key, present_value) of every
        layer, in place. path, path_lens: see ``tree_verify``; seqlens_k, new_lens: as they were for
        ``tree_forward``. Returns the new seqlens_k (-1 for a sequence of a bad length or path, see block_status)."""
        index = path.get_device()
        if index >= 0 and index != _current_device():
            with torch.cuda.device(index):
                return self.tree_accept(caches, path, path_lens, seqlens_k, new_lens, into_seqlens_k)
        tensors = list(chain.from_iterable(caches))
        layers = len(tensors) // 2
        if not 1 <= layers <= capi.GQA_MAX_TREE_LAYERS or set(map(len, caches)) != {2}:
            raise ValueError(f"caches: 1 to {capi.GQA_MAX_TREE_LAYERS} pairs (present_key, present_value)")
        # Two tensors a layer: a check is one pass over all of them.
        first, count = tensors[0], len(tensors)
        if not all(map(torch.Tensor.is_contiguous, tensors)):
            raise ValueError("tensors passed to the GQA library must be contiguous")
        if (list(map(_shape, tensors)).count(first.shape) != count or list(map(_dtype, tensors)).count(first.dtype) != count
                or list(map(torch.Tensor.get_device, tensors)).count(index) != count):
            raise ValueError("caches must be of one shape and dtype, on the other tensors' CUDA device")
        if into_seqlens_k is None:
            into_seqlens_k = torch.empty_like(seqlens_k, memory_format=torch.contiguous_format)

        def build():
            a = capi.GqaAcceptArgs()
            addresses = [(ctypes.c_void_p * layers)() for _ in range(2)]
            a.cache = tensor_desc(first)
            a.present_keys, a.present_values, a.num_layers = *addresses, layers
            return (a, *addresses), [a.path, a.path_lens, a.seqlens_k, a.new_lens, a.into_seqlens_k]

        with self._block_lock:
            rec = self._bind("tree_accept", (path, path_lens, seqlens_k, new_lens, into_seqlens_k),
                             (layers, first.shape, first.dtype), build)
            addresses = list(map(torch.Tensor.data_ptr, tensors))
            rec.structs[1][:], rec.structs[2][:] = addresses[::2], addresses[1::2]
            status = self._block_status_ptr.get(index) or self._status_word(path.device)
            capi.gqa_tree_accept(self.handle, rec.refs[0], status, _raw_stream(index))
        return into_seqlens_k
