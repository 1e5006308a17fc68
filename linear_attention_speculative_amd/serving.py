"""Python binding of the operators around the verify in a serving step:
prefill of prompts, single-token decode, the step's index tables, and sampling
with draft acceptance.

Argument marshalling only, as in `ops`; every computation runs in the HIP
library.  Beyond the library's own checks these functions check what the C
ABI cannot see: that every tensor lives on one GPU (the launch is made with
that device current, on its current stream unless one is given) and that
index arrays are int32, contiguous and long enough.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _abi
from .ops import (_DT, _pack_format, _ptr, _raise, _tensor_values)


def _launch(entry, args, kwargs, stream) -> None:
    """Calls `entry` with the tensors' GPU current, on that GPU's current
    stream or the one given."""
    on = {t.get_device() for t in kwargs.values()
          if isinstance(t, torch.Tensor)}
    if len(on) > 1:
        raise ValueError(f"tensors on different devices (indexes {on}, -1 "
                         "being the host)")
    index = on.pop() if on else -1
    if index < 0:
        raise ValueError("the tensors must be on a GPU")
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    elif isinstance(stream, torch.cuda.Stream):
        if stream.device.index != index:
            raise ValueError(f"a stream of {stream.device} for tensors on "
                             f"GPU {index}")
        handle = stream.cuda_stream
    else:
        handle = int(stream)
    if torch.cuda.current_device() == index:
        rc = entry(ctypes.byref(args), handle)
    else:
        with torch.cuda.device(index):
            rc = entry(ctypes.byref(args), handle)
    if rc != _abi.KDA_OK:
        _raise(rc)


def _ints(t, name: str, size: int) -> int:
    """Pointer of an int32 index array of at least `size` entries (0 for
    None)."""
    if t is None:
        return 0
    if t.dim() != 1 or t.numel() < size:
        raise ValueError(f"{name} needs {size} entries (got "
                         f"{list(t.shape)})")
    return _ptr(t) or 0


_PREFILL_PACK = struct.Struct("<" + _pack_format(_abi.KdaPrefillArgs))
_DECODE_PACK = struct.Struct("<" + _pack_format(_abi.KdaDecodeArgs))


def prefill_workspace_size(tokens: int, batch: int, num_heads: int,
                           head_dim: int, act_dtype: torch.dtype,
                           out_dtype: torch.dtype = None) -> int:
    """Bytes of workspace for a prefill of up to `tokens` rows and `batch`
    requests (outputs in `out_dtype`, default the activations' dtype)."""
    n = _abi.load().kda_prefill_workspace_size(
        tokens, batch, num_heads, head_dim, _DT.get(act_dtype, -1),
        _DT.get(out_dtype or act_dtype, -1))
    if n <= 0:
        raise ValueError("no prefill has these sizes and dtypes")
    return n


def prefill_args(*, mixed_qkv, raw_gate, raw_beta, A_log, dt_bias,
                 lower_bound, state, out, query_start_loc, state_indices,
                 workspace, conv_state=None, conv_weight=None,
                 spec_query_len=1, conv_dim_first=True,
                 initial_state_indices=None, num_accepted_tokens=None,
                 null_block_id=0) -> _abi.KdaPrefillArgs:
    """kda_prefill_args for these tensors."""
    B = state_indices.shape[0]
    if not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    vals = (*_tensor_values(mixed_qkv), *_tensor_values(raw_gate),
            *_tensor_values(raw_beta), *_tensor_values(A_log),
            *_tensor_values(dt_bias), *_tensor_values(state),
            *_tensor_values(out), *_tensor_values(conv_state),
            *_tensor_values(conv_weight),
            _ints(query_start_loc, "query_start_loc", B + 1),
            _ints(state_indices, "state_indices", B),
            _ints(initial_state_indices, "initial_state_indices", B),
            _ints(num_accepted_tokens, "num_accepted_tokens", B),
            workspace.data_ptr(),
            workspace.numel() * workspace.element_size(),
            B, spec_query_len, null_block_id, 1 if conv_dim_first else 0,
            0 if lower_bound is None else 1,
            0.0 if lower_bound is None else float(lower_bound))
    return _abi.KdaPrefillArgs.from_buffer_copy(_PREFILL_PACK.pack(*vals))


def check_prefill(**kwargs) -> int:
    """Host-only validation (no launch); returns the kda_status code."""
    return _abi.load().kda_check_prefill(ctypes.byref(prefill_args(**kwargs)))


def conv_prefill(*, stream=None, **kwargs) -> None:
    """One KDA layer over whole prompts, with the short convolution fused:
    request b's tokens are rows query_start_loc[b] .. query_start_loc[b + 1]
    of the activations, it starts from slot `initial_state_indices[b]` (zeros
    where null or not given) and leaves its checkpoint and conv history in
    slot `state_indices[b]`, ready for the verify or the decode with accepted
    count 1.  Arguments follow kda_prefill_args in
    include/kda_recoverssm.h; `lower_bound` is None (softplus gate) or at
    most 0; `workspace` is scratch memory of `prefill_workspace_size`
    bytes."""
    _launch(_abi.load().kda_conv_prefill, prefill_args(**kwargs),
            kwargs, stream)


def check_prefill_qkv(**kwargs) -> int:
    """Host-only validation of the unfused prefill (no launch)."""
    _no_conv(kwargs)
    return _abi.load().kda_check_prefill_qkv(
        ctypes.byref(prefill_args(**kwargs)))


def prefill_qkv(*, stream=None, **kwargs) -> None:
    """`conv_prefill` on already convolved q | k | v (no conv state, taps or
    accepted counts)."""
    _no_conv(kwargs)
    _launch(_abi.load().kda_prefill_qkv, prefill_args(**kwargs),
            kwargs, stream)


def decode_args(*, mixed_qkv, raw_gate, raw_beta, A_log, dt_bias,
                lower_bound, state, out, state_indices, conv_state=None,
                conv_weight=None, spec_query_len=1, conv_dim_first=True,
                final_state_indices=None, num_accepted_tokens=None,
                null_block_id=0) -> _abi.KdaDecodeArgs:
    """kda_decode_args for these tensors."""
    B = state_indices.shape[0]
    vals = (*_tensor_values(mixed_qkv), *_tensor_values(raw_gate),
            *_tensor_values(raw_beta), *_tensor_values(A_log),
            *_tensor_values(dt_bias), *_tensor_values(state),
            *_tensor_values(out), *_tensor_values(conv_state),
            *_tensor_values(conv_weight),
            _ints(state_indices, "state_indices", B),
            _ints(final_state_indices, "final_state_indices", B),
            _ints(num_accepted_tokens, "num_accepted_tokens", B),
            B, spec_query_len, null_block_id, 1 if conv_dim_first else 0,
            0 if lower_bound is None else 1,
            0.0 if lower_bound is None else float(lower_bound))
    return _abi.KdaDecodeArgs.from_buffer_copy(_DECODE_PACK.pack(*vals))


def check_decode(**kwargs) -> int:
    """Host-only validation (no launch); returns the kda_status code."""
    return _abi.load().kda_check_decode(ctypes.byref(decode_args(**kwargs)))


def conv_update_decode(*, stream=None, **kwargs) -> None:
    """One token per request of one KDA layer, with the short convolution
    fused: row b of the activations advances request b's checkpoint from
    `state_indices[b]` to `final_state_indices[b]` (default: in place), and
    its conv history with it.  Arguments follow kda_decode_args in
    include/kda_recoverssm.h; `lower_bound=None` selects the softplus gate,
    `num_accepted_tokens=None` reads histories at offset 0."""
    _launch(_abi.load().kda_conv_update_decode, decode_args(**kwargs),
            kwargs, stream)


def _no_conv(kwargs):
    for name in ("conv_state", "conv_weight", "num_accepted_tokens"):
        if kwargs.get(name) is not None:
            raise ValueError(f"{name} is not used on convolved q|k|v")


def check_decode_qkv(**kwargs) -> int:
    """Host-only validation of the unfused decode (no launch)."""
    _no_conv(kwargs)
    return _abi.load().kda_check_decode_qkv(
        ctypes.byref(decode_args(**kwargs)))


def decode_qkv(*, stream=None, **kwargs) -> None:
    """`conv_update_decode` on already convolved q | k | v (no conv state,
    taps or accepted counts)."""
    _no_conv(kwargs)
    _launch(_abi.load().kda_decode_qkv, decode_args(**kwargs),
            kwargs, stream)


_TABLES_PACK = struct.Struct("<" + _pack_format(_abi.KdaTablesArgs))


def tables_args(*, query_lens, num_computed_tokens, num_blocks, block_table,
                free_blocks, block_size, query_start_loc, new_num_blocks,
                state_indices, initial_state_indices, final_state_indices,
                positions, slot_mapping, num_allocated, request_indices=None,
                null_block_id=0) -> _abi.KdaTablesArgs:
    """kda_tables_args for these tensors."""
    B = query_lens.shape[0]
    if block_table.dim() != 2 or block_table.dtype != torch.int32:
        raise ValueError("block_table must be a two-dimensional int32 tensor")
    rows, width = block_table.shape
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    if not slot_mapping.is_contiguous() or slot_mapping.dim() != 1 or \
            slot_mapping.shape != positions.shape:
        raise ValueError("positions and slot_mapping must be contiguous "
                         "vectors of one size")
    if request_indices is None and rows < B:
        raise ValueError("without request_indices the tables need a row per "
                         "request")
    vals = (_ints(query_lens, "query_lens", B),
            _ints(num_computed_tokens, "num_computed_tokens", rows),
            _ints(num_blocks, "num_blocks", rows),
            _ints(request_indices, "request_indices", B),
            _ints(free_blocks, "free_blocks", 0), block_table.data_ptr(),
            *block_table.stride(), B, rows, width, block_size,
            free_blocks.shape[0], positions.shape[0], null_block_id, 0,
            _ints(query_start_loc, "query_start_loc", B + 1),
            _ints(new_num_blocks, "new_num_blocks", rows),
            _ints(state_indices, "state_indices", B),
            _ints(initial_state_indices, "initial_state_indices", B),
            _ints(final_state_indices, "final_state_indices", B),
            _ints(positions, "positions", 0), slot_mapping.data_ptr(),
            _ints(num_allocated, "num_allocated", 1))
    return _abi.KdaTablesArgs.from_buffer_copy(_TABLES_PACK.pack(*vals))


def check_step_tables(**kwargs) -> int:
    """Host-only validation (no launch); returns the kda_status code."""
    return _abi.load().kda_check_step_tables(
        ctypes.byref(tables_args(**kwargs)))


def step_tables(*, stream=None, **kwargs) -> None:
    """The index arrays of one serving step, built on the GPU from request
    lengths (kda_tables_args in include/kda_recoverssm.h): token offsets, new
    blocks from `free_blocks` appended to the rows of `block_table`, the
    state slots that prefill, decode and verify read and write, and each
    token's position and cache slot.  `num_allocated` receives how many
    blocks the step asked for; more than `free_blocks` holds means that some
    requests got null blocks."""
    _launch(_abi.load().kda_step_tables, tables_args(**kwargs),
            kwargs, stream)


_SAMPLE_PACK = struct.Struct("<" + _pack_format(_abi.KdaSampleArgs))


def _floats(t, name: str, size: int) -> int:
    """Pointer of a float32 array of at least `size` entries (0 for None)."""
    if t is None:
        return 0
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    if t.dim() != 1 or t.numel() < size or not t.is_contiguous():
        raise ValueError(f"{name} needs {size} contiguous entries (got "
                         f"{list(t.shape)})")
    return t.data_ptr()


def sample_workspace_size(rows: int, vocab: int) -> int:
    """Bytes of workspace for sampling up to `rows` rows of `vocab` logits."""
    n = _abi.load().kda_sample_workspace_size(rows, vocab)
    if n <= 0:
        raise ValueError("no sampling has these sizes")
    return n


def sample_args(*, logits, uniform, tokens, workspace, temperature=None,
                top_k=None, top_p=None, min_p=None, query_start_loc=None,
                draft_tokens=None, num_accepted=None,
                next_tokens=None) -> _abi.KdaSampleArgs:
    """kda_sample_args for these tensors."""
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocabulary]")
    M = logits.shape[0]
    B = M if query_start_loc is None else query_start_loc.numel() - 1
    if B < 0:
        raise ValueError("query_start_loc needs batch + 1 entries")
    if not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    vals = (*_tensor_values(logits), _floats(uniform, "uniform", M),
            _floats(temperature, "temperature", B),
            _ints(top_k, "top_k", B), _floats(top_p, "top_p", B),
            _floats(min_p, "min_p", B),
            _ints(query_start_loc, "query_start_loc", B + 1),
            _ints(draft_tokens, "draft_tokens", M),
            _ints(tokens, "tokens", M),
            _ints(num_accepted, "num_accepted", B),
            _ints(next_tokens, "next_tokens", B), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), B, 0)
    return _abi.KdaSampleArgs.from_buffer_copy(_SAMPLE_PACK.pack(*vals))


def check_sample(**kwargs) -> int:
    """Host-only validation (no launch); returns the kda_status code."""
    return _abi.load().kda_check_sample(ctypes.byref(sample_args(**kwargs)))


def sample(*, stream=None, **kwargs) -> None:
    """A token for every row of `logits` from the given `uniform` numbers,
    under the temperature, top-k, top-p and min-p of the row's request
    (kda_sample_args in include/kda_recoverssm.h).  With `draft_tokens` (the
    windows' tokens, rows as in the verify) also each request's accepted
    count, as `CommitContext.plan` and `commit_step` take it, and the token
    that follows the accepted ones.  `workspace` is scratch memory of
    `sample_workspace_size` bytes."""
    _launch(_abi.load().kda_sample, sample_args(**kwargs), kwargs, stream)
