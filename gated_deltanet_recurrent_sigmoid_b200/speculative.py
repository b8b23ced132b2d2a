"""Thin ctypes binding of ``libgdn_spec.so`` (C ABI in include/gdn_spec.h): the
operators of a speculative decode step around the state update.

One step of a batch, all on the GPU (``binding.decode_update`` and the model's
other layers lie between them):

    step_maps(lengths, context, slots, ...)      cu_seqlens, state_indices, rows
    decode_update(..., intermediate_states=...)  the state after every fed token
    token_probs(logits, probs, ...)              the target's probabilities
    verify_drafts(probs, drafts, ...)            tokens emitted, counts kept
    commit_states(intermediate_states, ...)      the kept state into the pool

Argument marshalling only, as in ``binding``: every step runs in the library's
kernels, each call launches one, on ``stream`` or else on the stream that is
current when the call is made, on the tensors' device.  A non-zero status
raises ``binding.GdnError``; tensors that are not on one CUDA device raise
ValueError.  The ``Prepared*`` classes keep the descriptors of a call that is
made again and again on the same buffers, which must stay alive; several
threads may use one object, each on its own current stream.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import binding as _binding
from . import build as _build
from .binding import ERR_CUDA, ERR_SHAPE, OK, GdnError, GdnExtra, GdnTensor, LAUNCH_PDL, status_string

CHECK_ONLY = 1 << 16

DEV_BAD_SEQ = 1 << 3
DEV_BAD_TEMPERATURE = 1 << 4
DEV_BAD_TOKEN = 1 << 5
DEV_BAD_PROBS = 1 << 6
DEV_BAD_COUNT = 1 << 7
DEV_BAD_LENGTH = 1 << 8
DEV_BAD_BLOCKS = 1 << 9
DEV_NO_ROOM = 1 << 10

MAX_VOCAB = 393216

_P = ctypes.POINTER(GdnTensor)
_MAPS_TENSORS = ("lengths", "context", "slots", "cu_seqlens", "state_indices", "row_seq", "positions", "block_tables",
                 "blocks_held", "free_blocks", "free_head", "blocks_held_out", "free_head_out", "slot_map")


class GdnStepMapsCall(ctypes.Structure):
    _fields_ = ([(n, _P) for n in _MAPS_TENSORS] +
                [("block_size", ctypes.c_int32), ("flags", ctypes.c_uint32), ("extra", ctypes.POINTER(GdnExtra))])


_LIB = None
_STREAMS_KEPT = 64       # streams that a prepared call remembers its arguments for


def library_path() -> str:
    return _build.SPEC_LIB_PATH


def load() -> ctypes.CDLL:
    """Load the in-tree library; raise if it has not been built."""
    global _LIB
    if _LIB is None:
        path = _build.SPEC_LIB_PATH
        if not os.path.exists(path):
            raise GdnError(ERR_CUDA, f"{path} is missing: build it with "
                                     "`python -m gated_deltanet_recurrent_sigmoid_b200.build`")
        lib = ctypes.CDLL(path)
        E = ctypes.POINTER(GdnExtra)
        lib.gdn_token_probs.argtypes = [_P] * 4 + [ctypes.c_uint32, E]
        lib.gdn_verify_drafts.argtypes = [_P] * 8 + [ctypes.c_uint32, E]
        lib.gdn_commit_states.argtypes = [_P] * 5 + [ctypes.c_uint32, E]
        lib.gdn_step_maps.argtypes = [ctypes.POINTER(GdnStepMapsCall)]
        lib.gdn_spec_version.argtypes = []
        for name in ("gdn_token_probs", "gdn_verify_drafts", "gdn_commit_states", "gdn_step_maps", "gdn_spec_version"):
            getattr(lib, name).restype = ctypes.c_int
        # the same functions without argument types: prepared calls pass pointers made once
        lib.untyped = ctypes.CDLL(path)
        _LIB = lib
    return _LIB


def _describe(t: Optional[torch.Tensor]) -> Optional[GdnTensor]:
    d = _binding.describe(t)
    if d is not None and t.dtype == torch.int64:
        d.dtype = 4
    return d


class _Prepared:
    """One call of the library on fixed tensors.  The host checks run once
    here (a bad argument raises at once) and again in every call."""

    def __init__(self, tensors, device_status: Optional[torch.Tensor], stream: Optional[torch.cuda.Stream]):
        self._keep = (tensors, device_status, stream)
        given = [t for t in (*tensors, device_status) if t is not None]
        self._descs = [_describe(t) for t in tensors]
        self._extra = GdnExtra()
        if device_status is not None:
            if device_status.dtype != torch.int32 or device_status.numel() < 1:
                raise GdnError(ERR_SHAPE, "device_status must be an int32 tensor")
            self._extra.device_status = device_status.data_ptr()
        if stream is not None:
            self._extra.stream = stream.cuda_stream
        self._follow = stream is None
        self._check(self._bind(CHECK_ONLY))
        devices = {t.device for t in given}
        if len(devices) != 1 or next(iter(devices)).type != "cuda":
            raise ValueError(f"the tensors of a call must be on one CUDA device, not {sorted(map(str, devices))}")
        self._device = next(iter(devices)).index
        if stream is not None and stream.device_index != self._device:
            raise ValueError("the stream is not one of the tensors' device")

    def _bind(self, more_flags: int = 0, extra: Optional[GdnExtra] = None):
        """(function, arguments) with ``more_flags`` beside the call's own, and
        ``extra`` in the place of the object's."""
        raise NotImplementedError

    @staticmethod
    def _check(call) -> None:
        fn, args = call
        status = fn(*args)
        if status != OK:
            raise GdnError(status, status_string(status))

    def _ready(self) -> None:
        fn, _ = self._bind()
        self._fn = getattr(load().untyped, fn.__name__)
        self._by_stream = {}
        self._args = None if self._follow else self._for_stream(self._extra.stream)

    def _for_stream(self, stream: int):
        """The arguments on ``stream`` (pointers, and what they point at).  They
        are never written again: the library runs without the interpreter's
        lock, so another thread may be inside a call with its own."""
        extra = GdnExtra.from_buffer_copy(self._extra)
        extra.stream = stream
        _, args = self._bind(extra=extra)
        return tuple(ctypes.c_void_p(ctypes.addressof(a._obj)) if hasattr(a, "_obj") else a for a in args), args

    def __call__(self) -> None:
        device, bound = self._device, self._args
        if bound is None:
            stream = torch._C._cuda_getCurrentRawStream(device)
            bound = self._by_stream.get(stream)
            if bound is None:
                if len(self._by_stream) >= _STREAMS_KEPT:
                    self._by_stream = {}
                bound = self._by_stream[stream] = self._for_stream(stream)
        if torch._C._cuda_getDevice() == device:
            status = self._fn(*bound[0])
        else:
            with torch.cuda.device(device):
                status = self._fn(*bound[0])
        if status != OK:
            raise GdnError(status, status_string(status))

    def _refs(self):
        return [None if d is None else ctypes.byref(d) for d in self._descs]

    def _once(self) -> None:
        """Call now, for tensors that the caller may free right after it."""
        self()
        tensors, status, stream = self._keep
        if stream is not None and stream.cuda_stream != torch._C._cuda_getCurrentRawStream(self._device):
            for t in (*tensors, status):
                if t is not None:
                    t.record_stream(stream)


class PreparedTokenProbs(_Prepared):
    """``token_probs`` with its descriptors built once."""

    def __init__(self, logits, probs, temperature=None, row_seq=None, flags: int = 0, device_status=None, stream=None):
        self._flags = int(flags)
        super().__init__((logits, temperature, row_seq, probs), device_status, stream)
        self._ready()

    def _bind(self, more_flags: int = 0, extra: Optional[GdnExtra] = None):
        return load().gdn_token_probs, (*self._refs(), ctypes.c_uint32(self._flags | more_flags),
                                        ctypes.byref(extra or self._extra))


class PreparedVerifyDrafts(_Prepared):
    """``verify_drafts`` with its descriptors built once."""

    def __init__(self, target_probs, draft_tokens, draft_probs, uniforms, out_tokens, num_tokens, cu_seqlens=None,
                 state_indices=None, flags: int = 0, device_status=None, stream=None):
        self._flags = int(flags)
        super().__init__((target_probs, draft_tokens, draft_probs, uniforms, cu_seqlens, state_indices, out_tokens,
                          num_tokens), device_status, stream)
        self._ready()

    def _bind(self, more_flags: int = 0, extra: Optional[GdnExtra] = None):
        return load().gdn_verify_drafts, (*self._refs(), ctypes.c_uint32(self._flags | more_flags),
                                          ctypes.byref(extra or self._extra))


class PreparedCommitStates(_Prepared):
    """``commit_states`` with its descriptors built once."""

    def __init__(self, intermediate_states, num_tokens, state_pool, state_indices, cu_seqlens=None, flags: int = 0,
                 device_status=None, stream=None):
        self._flags = int(flags)
        super().__init__((intermediate_states, num_tokens, state_pool, state_indices, cu_seqlens), device_status,
                         stream)
        self._ready()

    def _bind(self, more_flags: int = 0, extra: Optional[GdnExtra] = None):
        return load().gdn_commit_states, (*self._refs(), ctypes.c_uint32(self._flags | more_flags),
                                          ctypes.byref(extra or self._extra))


class PreparedStepMaps(_Prepared):
    """``step_maps`` with its descriptors built once."""

    def __init__(self, lengths, context, slots, cu_seqlens, state_indices, row_seq, positions, block_tables=None,
                 blocks_held=None, free_blocks=None, free_head=None, blocks_held_out=None, free_head_out=None,
                 slot_map=None, block_size: int = 0, flags: int = 0, device_status=None, stream=None):
        self._flags, self._block_size = int(flags), int(block_size)
        super().__init__((lengths, context, slots, cu_seqlens, state_indices, row_seq, positions, block_tables,
                          blocks_held, free_blocks, free_head, blocks_held_out, free_head_out, slot_map),
                         device_status, stream)
        self._ready()

    def _bind(self, more_flags: int = 0, extra: Optional[GdnExtra] = None):
        call = GdnStepMapsCall()
        for name, d in zip(_MAPS_TENSORS, self._descs):
            if d is not None:
                setattr(call, name, ctypes.pointer(d))
        call.block_size = self._block_size
        call.flags = self._flags | more_flags
        call.extra = ctypes.pointer(extra or self._extra)
        return load().gdn_step_maps, (ctypes.byref(call),)


def token_probs(logits: torch.Tensor, probs: torch.Tensor, temperature: Optional[torch.Tensor] = None,
                row_seq: Optional[torch.Tensor] = None, flags: int = 0, device_status: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``probs[r] = softmax(logits[r] / temperature[row_seq[r]])`` (bf16 or
    fp32 in and out, [R, vocab]).  Without ``row_seq`` the temperatures are per
    row, without ``temperature`` they are 1; 0 gives 1 at the row's first
    largest logit.  Rows with ``row_seq`` = -1 are left as they were.  Returns
    ``probs``."""
    PreparedTokenProbs(logits, probs, temperature, row_seq, flags, device_status, stream)._once()
    return probs


def verify_drafts(target_probs: torch.Tensor, draft_tokens: torch.Tensor, draft_probs: Optional[torch.Tensor],
                  uniforms: torch.Tensor, out_tokens: torch.Tensor, num_tokens: torch.Tensor,
                  cu_seqlens: Optional[torch.Tensor] = None, state_indices: Optional[torch.Tensor] = None,
                  flags: int = 0, device_status: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> tuple:
    """Judge ``draft_tokens`` [N, D] against the packed rows of
    ``target_probs`` with the random numbers ``uniforms`` [N, D + 1], and draw
    each sequence's next token with the last of them.  ``draft_probs``
    [N, D, vocab], or None for drafts that were certain.  Writes and returns
    ``out_tokens`` [N, D + 1] (accepted drafts, the drawn token, then -1) and
    ``num_tokens`` [N], the number of either."""
    PreparedVerifyDrafts(target_probs, draft_tokens, draft_probs, uniforms, out_tokens, num_tokens, cu_seqlens,
                         state_indices, flags, device_status, stream)._once()
    return out_tokens, num_tokens


def commit_states(intermediate_states: torch.Tensor, num_tokens: torch.Tensor, state_pool: torch.Tensor,
                  state_indices: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None, flags: int = 0,
                  device_status: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Copy the state after each sequence's ``num_tokens``-th fed token from
    ``intermediate_states`` into its slot of ``state_pool``.  Returns
    ``state_pool``."""
    PreparedCommitStates(intermediate_states, num_tokens, state_pool, state_indices, cu_seqlens, flags, device_status,
                         stream)._once()
    return state_pool


def step_maps(lengths: torch.Tensor, context: torch.Tensor, slots: torch.Tensor, cu_seqlens: torch.Tensor,
              state_indices: torch.Tensor, row_seq: torch.Tensor, positions: torch.Tensor,
              block_tables: Optional[torch.Tensor] = None, blocks_held: Optional[torch.Tensor] = None,
              free_blocks: Optional[torch.Tensor] = None, free_head: Optional[torch.Tensor] = None,
              blocks_held_out: Optional[torch.Tensor] = None, free_head_out: Optional[torch.Tensor] = None,
              slot_map: Optional[torch.Tensor] = None, block_size: int = 0, flags: int = 0,
              device_status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Fill a step's index arrays from its requests' ``lengths``, ``context``
    and ``slots`` ([N] int32): ``cu_seqlens`` and ``state_indices`` for
    ``decode_update``, ``row_seq`` and ``positions`` per packed row, and with a
    cache in blocks of ``block_size`` tokens the blocks that the step lacks
    (``block_tables``, ``blocks_held_out``, ``free_head_out``) and each row's
    place in it (``slot_map``, int64)."""
    PreparedStepMaps(lengths, context, slots, cu_seqlens, state_indices, row_seq, positions, block_tables, blocks_held,
                     free_blocks, free_head, blocks_held_out, free_head_out, slot_map, block_size, flags,
                     device_status, stream)._once()
