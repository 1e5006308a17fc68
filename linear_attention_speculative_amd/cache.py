"""Python binding of the operators on token caches and token histories: the
attention layers over paged latent caches, and the changes of logits in front
of `sample`.

Argument marshalling and the checks that the C ABI cannot make, as in
`serving`; every computation runs in the HIP library.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _abi
from .ops import _DT, _pack_format, _tensor_values
from .serving import _floats, _ints, _launch

_WRITE_PACK = struct.Struct("<" + _pack_format(_abi.KdaLatentWriteArgs))


def latent_write_args(*, latent, cache, slot_mapping, rope_key=None,
                      null_block_id=0) -> _abi.KdaLatentWriteArgs:
    """kda_latent_write_args for these tensors."""
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    if slot_mapping.dim() != 1 or not slot_mapping.is_contiguous() or \
            slot_mapping.shape[0] < latent.shape[0]:
        raise ValueError("slot_mapping needs a contiguous entry per token")
    vals = (*_tensor_values(latent), *_tensor_values(rope_key),
            *_tensor_values(cache), slot_mapping.data_ptr(), null_block_id, 0)
    return _abi.KdaLatentWriteArgs.from_buffer_copy(_WRITE_PACK.pack(*vals))


def check_latent_write(**kwargs) -> int:
    """Host-only validation (no launch); returns the kda_status code."""
    return _abi.load().kda_check_latent_write(
        ctypes.byref(latent_write_args(**kwargs)))


def latent_write(*, stream=None, **kwargs) -> None:
    """Each token's `latent` (and `rope_key`) into its place of a paged cache
    (kda_latent_write_args in include/kda_recoverssm.h); `slot_mapping` as
    `step_tables` gives it, of which the first entry per row of `latent` is
    read, -1 writing nothing."""
    _launch(_abi.load().kda_latent_write, latent_write_args(**kwargs), kwargs,
            stream)


def _table(block_table, request_indices, batch):
    """(pointer, strides, rows, width) of a block table."""
    if block_table.dim() != 2 or block_table.dtype != torch.int32:
        raise ValueError("block_table must be a two-dimensional int32 tensor")
    rows, width = block_table.shape
    if request_indices is None and rows < batch:
        raise ValueError("without request_indices the table needs a row per "
                         "request")
    return block_table.data_ptr(), block_table.stride(), rows, width


def _workspace(t):
    if not t.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def latent_attention_workspace_size(tokens: int, batch: int, num_heads: int,
                                    latent_dim: int, rope_dim: int,
                                    act_dtype: torch.dtype) -> int:
    """Bytes of workspace for a latent attention over `tokens` rows of `batch`
    requests.  Batches of other sizes may need more or less: a workspace for
    several takes the largest."""
    n = _abi.load().kda_latent_attention_workspace_size(
        tokens, batch, num_heads, latent_dim, rope_dim,
        _DT.get(act_dtype, -1))
    if n <= 0:
        raise ValueError("no latent attention has these sizes and dtype")
    return n


_LATENT_PACK = struct.Struct("<" + _pack_format(_abi.KdaLatentArgs))


def latent_args(*, q, cache, out, query_start_loc, num_computed_tokens,
                block_table, softmax_scale, workspace, lse=None,
                request_indices=None, null_block_id=0) -> _abi.KdaLatentArgs:
    """kda_latent_args for these tensors."""
    B = query_start_loc.numel() - 1
    if B < 0:
        raise ValueError("query_start_loc needs batch + 1 entries")
    table, strides, rows, width = _table(block_table, request_indices, B)
    work, size = _workspace(workspace)
    vals = (*_tensor_values(q), *_tensor_values(cache), *_tensor_values(out),
            *_tensor_values(lse),
            _ints(query_start_loc, "query_start_loc", B + 1),
            _ints(num_computed_tokens, "num_computed_tokens", rows),
            _ints(request_indices, "request_indices", B), table, *strides,
            work, size, B, rows, width, null_block_id, float(softmax_scale),
            0)
    return _abi.KdaLatentArgs.from_buffer_copy(_LATENT_PACK.pack(*vals))


def check_latent_attention(**kwargs) -> int:
    """Host-only validation (no launch); returns the kda_status code."""
    return _abi.load().kda_check_latent_attention(
        ctypes.byref(latent_args(**kwargs)))


def latent_attention(*, stream=None, **kwargs) -> None:
    """Attention of single tokens, draft windows or short prompt pieces in
    latent space, over a paged cache that holds their own entries already
    (`latent_write`): each query sees its request's positions up to its own.
    Arguments follow kda_latent_args in include/kda_recoverssm.h; `q` and
    `out` are [tokens, heads, ..], `lse` (optional) receives the log of each
    softmax's sum, `workspace` is scratch memory of
    `latent_attention_workspace_size` bytes."""
    _launch(_abi.load().kda_latent_attention, latent_args(**kwargs), kwargs,
            stream)


_EXPAND_PACK = struct.Struct("<" + _pack_format(_abi.KdaLatentExpandArgs))


def latent_expand_args(*, cache, weight, key, value, key_start_loc,
                       block_table, rope_key=None, request_indices=None,
                       null_block_id=0) -> _abi.KdaLatentExpandArgs:
    """kda_latent_expand_args for these tensors."""
    B = key_start_loc.numel() - 1
    if B < 0:
        raise ValueError("key_start_loc needs batch + 1 entries")
    table, strides, rows, width = _table(block_table, request_indices, B)
    vals = (*_tensor_values(cache), *_tensor_values(weight),
            *_tensor_values(key), *_tensor_values(rope_key),
            *_tensor_values(value),
            _ints(key_start_loc, "key_start_loc", B + 1),
            _ints(request_indices, "request_indices", B), table, *strides, B,
            rows, width, null_block_id)
    return _abi.KdaLatentExpandArgs.from_buffer_copy(_EXPAND_PACK.pack(*vals))


def check_latent_expand(**kwargs) -> int:
    """Host-only validation (no launch); returns the kda_status code."""
    return _abi.load().kda_check_latent_expand(
        ctypes.byref(latent_expand_args(**kwargs)))


def latent_expand(*, stream=None, **kwargs) -> None:
    """Keys and values of every head from the cached latents of whole requests
    (kda_latent_expand_args in include/kda_recoverssm.h): rows
    key_start_loc[b] .. key_start_loc[b + 1] of `key`, `value` and `rope_key`
    (optional: the cached rope keys) are request b's positions from 0 on.
    `weight` is [heads, 2 * head_dim, latent], keys' rows before values'."""
    _launch(_abi.load().kda_latent_expand, latent_expand_args(**kwargs),
            kwargs, stream)


_PROMPT_PACK = struct.Struct("<" + _pack_format(_abi.KdaLatentPrefillArgs))


def latent_prefill_args(*, q, key, value, out, query_start_loc, key_start_loc,
                        softmax_scale, rope_key=None,
                        lse=None) -> _abi.KdaLatentPrefillArgs:
    """kda_latent_prefill_args for these tensors."""
    B = query_start_loc.numel() - 1
    if B < 0:
        raise ValueError("query_start_loc needs batch + 1 entries")
    vals = (*_tensor_values(q), *_tensor_values(key),
            *_tensor_values(rope_key), *_tensor_values(value),
            *_tensor_values(out), *_tensor_values(lse),
            _ints(query_start_loc, "query_start_loc", B + 1),
            _ints(key_start_loc, "key_start_loc", B + 1), B,
            float(softmax_scale))
    return _abi.KdaLatentPrefillArgs.from_buffer_copy(
        _PROMPT_PACK.pack(*vals))


def check_latent_prefill(**kwargs) -> int:
    """Host-only validation (no launch); returns the kda_status code."""
    return _abi.load().kda_check_latent_prefill(
        ctypes.byref(latent_prefill_args(**kwargs)))


def latent_prefill(*, stream=None, **kwargs) -> None:
    """Causal attention of prompts, or pieces of prompts behind computed
    tokens, over expanded keys and values (`latent_expand`): request b's
    queries are its last positions among its keys.  Arguments follow
    kda_latent_prefill_args in include/kda_recoverssm.h; the last values of a
    query go with `rope_key`, which all heads share."""
    _launch(_abi.load().kda_latent_prefill, latent_prefill_args(**kwargs),
            kwargs, stream)


_LOGITS_PACK = struct.Struct("<" + _pack_format(_abi.KdaLogitsArgs))


def _int_rows(t, name):
    """(pointer, row stride, rows, columns) of a two-dimensional int32 tensor
    with contiguous rows."""
    if t is None:
        return 0, 0, 0, 0
    if t.dim() != 2 or t.dtype != torch.int32:
        raise ValueError(f"{name} must be a two-dimensional int32 tensor")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} needs contiguous rows")
    return t.data_ptr(), t.stride(0), t.shape[0], t.shape[1]


def logits_args(*, logits, query_start_loc=None, draft_tokens=None,
                request_indices=None, token_ids=None, prompt_lens=None,
                token_lens=None, repetition_penalty=None,
                frequency_penalty=None, presence_penalty=None,
                bias_start=None, bias_tokens=None, bias_values=None,
                mask=None, mask_rows=None) -> _abi.KdaLogitsArgs:
    """kda_logits_args for these tensors."""
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocabulary]")
    M, V = logits.shape
    B = M if query_start_loc is None else query_start_loc.numel() - 1
    if B < 0:
        raise ValueError("query_start_loc needs batch + 1 entries")
    ids, s_ids, rows, length = _int_rows(token_ids, "token_ids")
    if token_ids is not None:
        if request_indices is None and rows < B:
            raise ValueError("without request_indices token_ids needs a row "
                             "per request")
        if rows and (prompt_lens is None or token_lens is None):
            raise ValueError("token_ids need prompt_lens and token_lens")
    words, s_mask, masks, width = _int_rows(mask, "mask")
    if mask is not None:
        if masks and width < (V + 31) // 32:
            raise ValueError("mask needs a bit for every token")
        if mask_rows is None and masks < M:
            raise ValueError("without mask_rows there is a mask per row")
    n = 0
    if bias_start is not None:
        if bias_tokens is None or bias_values is None:
            raise ValueError("bias_start needs bias_tokens and bias_values")
        n = min(bias_tokens.numel(), bias_values.numel())
    vals = (*_tensor_values(logits),
            _ints(query_start_loc, "query_start_loc", B + 1),
            _ints(draft_tokens, "draft_tokens", M),
            _ints(request_indices, "request_indices", B), ids, s_ids,
            _ints(prompt_lens, "prompt_lens", rows),
            _ints(token_lens, "token_lens", rows),
            _floats(repetition_penalty, "repetition_penalty", B),
            _floats(frequency_penalty, "frequency_penalty", B),
            _floats(presence_penalty, "presence_penalty", B),
            _ints(bias_start, "bias_start", B + 1),
            _ints(bias_tokens, "bias_tokens", n),
            _floats(bias_values, "bias_values", n), words, s_mask,
            _ints(mask_rows, "mask_rows", M), B, rows, length, n, masks, 0)
    return _abi.KdaLogitsArgs.from_buffer_copy(_LOGITS_PACK.pack(*vals))


def check_adjust_logits(**kwargs) -> int:
    """Host-only validation (no launch); returns the kda_status code."""
    return _abi.load().kda_check_adjust_logits(
        ctypes.byref(logits_args(**kwargs)))


def adjust_logits(*, stream=None, **kwargs) -> None:
    """Logits changed in place in front of `sample`: biases, repetition,
    frequency and presence penalties from the token histories (and a window's
    drafts), grammar masks (kda_logits_args in include/kda_recoverssm.h).
    Rows belong to requests as in `sample`; every change is optional."""
    _launch(_abi.load().kda_adjust_logits, logits_args(**kwargs), kwargs,
            stream)
