"""The multi-axis rotary, the block-scaled int8 cache and its eviction for torch tensors.

Argument marshalling only: the entry points are ``gqa_rotary_axes``, ``gqa_block_forward`` and
``gqa_block_evict`` of include/gqa.h, which also states shapes, types and semantics.
"""

from __future__ import annotations

import ctypes
import threading

import torch

from . import capi

# The current stream's handle without a Stream object (2 us less per call), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
# Likewise the current device and whether a graph is being captured (asked once a CUDA tensor is in hand).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or torch.cuda.is_current_stream_capturing

_DTYPE_CODE = {torch.float32: capi.GQA_F32, torch.float16: capi.GQA_F16, torch.int8: capi.GQA_I8,
               torch.uint8: capi.GQA_U8, torch.int32: capi.GQA_I32, torch.bfloat16: capi.GQA_BF16}


def tensor_desc(t: torch.Tensor | None) -> capi.GqaTensor:
    """C descriptor of a contiguous CUDA tensor (or an absent input for None)."""
    if t is None:
        return capi.GqaTensor()
    if not t.is_contiguous():
        raise ValueError("tensors passed to the GQA library must be contiguous")
    if t.dtype not in _DTYPE_CODE:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return capi.describe(t.data_ptr(), _DTYPE_CODE[t.dtype], tuple(t.shape))


def _int32(value, name: str) -> int:
    """`value` as the C int it becomes (a ctypes field would keep its low 32 bits without a word)."""
    v = int(value)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name} {v} does not fit 32 bits")
    return v


class BlockCache:
    """An int8 K/V cache with one scale per block of tokens and KV head (``gqa_block_cache``).

    key/value_codes: int8 (B, N_kv, C, H); key/value_scales: float32 (B, N_kv, ceil(C / block_size)). Row r of a
    head is ``code * scale[r // block_size]``. The tensors are the caller's; every step updates them in place.
    """

    __slots__ = ("key_codes", "value_codes", "key_scales", "value_scales", "block_size")

    def __init__(self, key_codes, value_codes, key_scales, value_scales, block_size: int):
        self.key_codes, self.value_codes = key_codes, value_codes
        self.key_scales, self.value_scales = key_scales, value_scales
        self.block_size = int(block_size)

    @classmethod
    def empty(cls, batch: int, kv_num_heads: int, capacity: int, head_size: int, block_size: int = 64,
              device="cuda") -> "BlockCache":
        """A cache of zero rows (codes and scales 0)."""
        codes = [torch.zeros((batch, kv_num_heads, capacity, head_size), dtype=torch.int8, device=device)
                 for _ in range(2)]
        blocks = -(-capacity // block_size)
        scales = [torch.zeros((batch, kv_num_heads, blocks), device=device) for _ in range(2)]
        return cls(*codes, *scales, block_size)

    def tensors(self):
        return self.key_codes, self.value_codes, self.key_scales, self.value_scales


class _Bound:
    """C structs of one kind of call, kept while the tensors' shapes and dtypes stay; pointers are set per call."""

    __slots__ = ("extra", "sigs", "fields", "structs", "refs", "nbytes")


class BlockCacheOps:
    """The block-cache methods of ``GroupQueryAttention``. Calls run on torch's current stream of the tensors'
    device; one call at a time per operator is marshalled (other threads wait)."""

    def _init_block_ops(self) -> None:
        self._block_lock = threading.Lock()
        self._block_calls: dict[str, _Bound] = {}
        self._block_ws: dict[tuple[int, int], torch.Tensor] = {}
        self._block_status: dict[int, torch.Tensor] = {}
        self._block_status_ptr: dict[int, int] = {}

    # ---- marshalling

    def _bind(self, kind: str, tensors, extra, build) -> _Bound:
        """The structs of a call of this kind with the tensors' pointers set. ``build()`` makes new structs:
        (structs, [descriptor of each tensor])."""
        index = tensors[0].get_device()   # negative: not a CUDA tensor
        rec = self._block_calls.get(kind)
        if rec is not None and index >= 0 and rec.extra == extra:
            for t, sig, f in zip(tensors, rec.sigs, rec.fields):
                if t is None:
                    if sig is not None:
                        break
                elif (sig is None or t.shape != sig[0] or t.dtype is not sig[1] or t.get_device() != index
                      or not t.is_contiguous()):
                    break
                else:
                    f.data = t.data_ptr()
            else:
                return rec
        dev = tensors[0].device
        for t in tensors:
            if t is None:
                continue
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"expected a torch.Tensor, got {type(t).__name__}")
            if t.device != dev or t.device.type != "cuda":
                raise ValueError("tensors passed to the GQA library must be on one CUDA device")
        rec = _Bound()
        rec.extra = extra
        rec.sigs = [None if t is None else (t.shape, t.dtype) for t in tensors]
        descs = [tensor_desc(t) for t in tensors]
        rec.structs, rec.fields = build()
        for d, f in zip(descs, rec.fields):
            ctypes.memmove(ctypes.byref(f), ctypes.byref(d), ctypes.sizeof(d))
        rec.refs = tuple(ctypes.byref(x) for x in rec.structs)
        rec.nbytes = None
        self._block_calls[kind] = rec
        return rec

    def _status_word(self, dev: torch.device) -> int:
        s = self._block_status.get(dev.index)
        if s is None:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("run one call on this device before capturing (it makes the status word)")
            s = torch.zeros(64, dtype=torch.int32, device=dev)
            torch.cuda.current_stream(dev).synchronize()   # other streams may use it from now on
            self._block_status[dev.index] = s
            self._block_status_ptr[dev.index] = s.data_ptr()
        return s.data_ptr()

    def _scratch(self, nbytes: int, index: int, stream: int) -> torch.Tensor | None:
        """Workspace of a call: one per (device, stream); a captured call gets its own from the graph's pool."""
        captured = _capturing()
        ws = None if captured else self._block_ws.get((index, stream))
        if ws is None or ws.numel() < nbytes:
            ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=torch.device("cuda", index))
            if not captured:
                self._block_ws[(index, stream)] = ws
        return ws

    def block_status(self, device=None) -> int:
        """Synchronise the current stream, then return and clear the GQA_DEVICE_* bits that ``rotary_axes``,
        ``block_forward`` and ``block_evict`` calls of this operator set on `device` since the last reading."""
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        index = torch.cuda.current_device() if dev.index is None else dev.index
        s = self._block_status.get(index)
        if s is None:
            return 0
        with torch.cuda.device(index):
            return capi.gqa_read_device_status(self.handle, s.data_ptr(), torch.cuda.current_stream().cuda_stream)

    # ---- operators

    def rotary_axes(self, query, key, positions, cos_cache, sin_cache, sections, interleaved=False,
                    q_norm_weight=None, k_norm_weight=None, out_query=None, out_key=None):
        """Rotate query (and key, or None) at positions (axes, B, S) on several axes; returns (query, key).

        sections: pairs of each axis. out_query / out_key may be the inputs (in place). A token of a bad position
        is not written (block_status tells), also not in tensors made here."""
        index = query.get_device()
        if index >= 0 and index != _current_device():
            with torch.cuda.device(index):
                return self.rotary_axes(query, key, positions, cos_cache, sin_cache, sections, interleaved,
                                        q_norm_weight, k_norm_weight, out_query, out_key)
        if out_query is None:
            out_query = torch.empty_like(query, memory_format=torch.contiguous_format)
        if out_key is None and key is not None:
            out_key = torch.empty_like(key, memory_format=torch.contiguous_format)
        extra = (tuple(sections), bool(interleaved))

        def build():
            sec = extra[0]
            if not 1 <= len(sec) <= capi.GQA_MAX_ROTARY_AXES:
                raise ValueError(f"sections: 1 to {capi.GQA_MAX_ROTARY_AXES} axes")
            inp, out = capi.GqaRotaryInputs(), capi.GqaRotaryOutputs()
            for i, n in enumerate(sec):
                inp.sections[i] = _int32(n, "a section")
            inp.num_axes, inp.interleaved = len(sec), int(extra[1])
            return (inp, out), [inp.query, inp.key, inp.positions, inp.cos_cache, inp.sin_cache, inp.q_norm_weight,
                                inp.k_norm_weight, out.query, out.key]

        with self._block_lock:
            rec = self._bind("rotary", (query, key, positions, cos_cache, sin_cache, q_norm_weight, k_norm_weight,
                                        out_query, out_key), extra, build)
            status = self._block_status_ptr.get(index) or self._status_word(query.device)
            capi.gqa_rotary_axes(self.handle, *rec.refs, status, _raw_stream(index))
        return out_query, out_key

    def block_forward(self, query, key, value, seqlens_k, total_sequence_length, cache: BlockCache, new_lens=None,
                      head_sink=None, past_weights=None, present_weights=None, output=None):
        """One step over a block-scaled cache: store key / value (None: already stored), attend, and with
        present_weights add up the attention weight of every cache row. Returns ``output``. total_sequence_length is
        an upper bound of the lengths. Nothing of a sequence of a bad length is written (block_status tells), also
        not in an output made here."""
        index = query.get_device()
        if index >= 0 and index != _current_device():
            with torch.cuda.device(index):
                return self.block_forward(query, key, value, seqlens_k, total_sequence_length, cache, new_lens,
                                          head_sink, past_weights, present_weights, output)
        if output is None:
            output = torch.empty_like(query, memory_format=torch.contiguous_format)
        extra = cache.block_size

        def build():
            inp, out, c = capi.GqaBlockInputs(), capi.GqaBlockOutputs(), capi.GqaBlockCache()
            c.block_size = _int32(extra, "block_size")
            return (c, inp, out), [inp.query, inp.key, inp.value, inp.seqlens_k, inp.new_lens, inp.head_sink,
                                   inp.past_weights, out.present_weights, out.output, c.key_codes, c.value_codes,
                                   c.key_scales, c.value_scales]

        with self._block_lock:
            rec = self._bind("forward", (query, key, value, seqlens_k, new_lens, head_sink, past_weights,
                                         present_weights, output, *cache.tensors()), extra, build)
            inp = rec.structs[1]
            if rec.nbytes is None or inp.total_sequence_length != total_sequence_length:
                rec.nbytes = None
                inp.total_sequence_length = _int32(total_sequence_length, "total_sequence_length")
                rec.nbytes = capi.gqa_block_workspace_size(self.handle, *rec.structs)
            stream = _raw_stream(index)
            status = self._block_status_ptr.get(index) or self._status_word(query.device)
            ws = self._scratch(rec.nbytes, index, stream)
            capi.gqa_block_forward(self.handle, *rec.refs, ws.data_ptr(), ws.numel(), status, stream)
        return output

    def block_evict(self, cache: BlockCache, weights, seqlens_k, total_sequence_length, keep: int, into: BlockCache,
                    into_weights=None, recent: int = 0, first: int = 0, kept=None, into_seqlens_k=None):
        """Copy the rows of `cache` that stay (first, recent, and the largest weights between) to `into`.
        Returns (kept, into_seqlens_k): the source row of every kept row (-1 behind the last) and the lengths.
        For a sequence of a bad length (see block_status) both are -1 where they are made here, and left as they
        were where they are given."""
        index = weights.get_device()
        if index >= 0 and index != _current_device():
            with torch.cuda.device(index):
                return self.block_evict(cache, weights, seqlens_k, total_sequence_length, keep, into, into_weights,
                                        recent, first, kept, into_seqlens_k)
        extra = (_int32(keep, "keep"), int(recent), int(first), cache.block_size, into.block_size,
                 (capi.GQA_FILL_KEPT if kept is None else 0) | (capi.GQA_FILL_SEQLENS if into_seqlens_k is None else 0))
        if kept is None:
            kept = torch.empty((*weights.shape[:2], max(0, extra[0])), dtype=torch.int32, device=weights.device)
        if into_seqlens_k is None:
            into_seqlens_k = torch.empty_like(seqlens_k, memory_format=torch.contiguous_format)

        def build():
            a = capi.GqaEvictArgs()
            names = ("keep", "recent", "first", "block_size", "block_size of into", "fill_skipped")
            a.keep, a.recent, a.first, a.source.block_size, a.into.block_size, a.fill_skipped = map(_int32, extra, names)
            return (a,), [a.weights, a.seqlens_k, a.into_weights, a.kept, a.into_seqlens_k, a.source.key_codes,
                          a.source.value_codes, a.source.key_scales, a.source.value_scales, a.into.key_codes,
                          a.into.value_codes, a.into.key_scales, a.into.value_scales]

        with self._block_lock:
            rec = self._bind("evict", (weights, seqlens_k, into_weights, kept, into_seqlens_k, *cache.tensors(),
                                       *into.tensors()), extra, build)
            rec.structs[0].total_sequence_length = _int32(total_sequence_length, "total_sequence_length")
            status = self._block_status_ptr.get(index) or self._status_word(weights.device)
            capi.gqa_block_evict(self.handle, *rec.refs, status, _raw_stream(index))
        return kept, into_seqlens_k
