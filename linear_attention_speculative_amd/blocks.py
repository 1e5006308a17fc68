"""Python binding of the operators on cache blocks: copies over all pools of a
model, forks of requests, references and free blocks, compaction.

Argument marshalling and the checks that the C ABI cannot make, as in
`serving`; every computation runs in the HIP library.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Sequence

import torch

from . import _abi
from .cache import _table, _workspace
from .ops import _pack_format
from .serving import _ints, _launch


def _pairs(t, name="copy_pairs"):
    """(pointer, rows) of an int32 [rows, 2] tensor."""
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if t.dim() != 2 or t.shape[1] != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [pairs, 2] tensor")
    return t.data_ptr(), t.shape[0]


class BlockPools:
    """Every pool of a model whose first dimension is the block: states, conv
    states, caches.  Their addresses go to the GPU once; `copy` then moves
    blocks of all of them in one launch."""

    def __init__(self, pools: Sequence[torch.Tensor], null_block_id: int = 0):
        if not pools:
            raise ValueError("at least one pool is needed")
        self.num_blocks = pools[0].shape[0]
        self.null_block_id = null_block_id
        rows = []
        for i, t in enumerate(pools):
            if t.dim() < 2 or t.shape[0] != self.num_blocks or \
                    t.numel() == 0:
                raise ValueError(f"pool {i} must be [{self.num_blocks}, ..] "
                                 "as the first one")
            if t.device != pools[0].device:
                raise ValueError("the pools must be on one device")
            if not _dense(t[0]):
                raise ValueError(f"a block of pool {i} must be one piece of "
                                 "memory")
            es = t.element_size()
            rows.append((t.data_ptr(), t.stride(0) * es, t[0].numel() * es))
        self.pools = list(pools)               # (their addresses are kept)
        host = [v for col in zip(*rows) for v in col]
        self._host = (ctypes.c_int64 * len(host))(*host)
        self._tables = torch.tensor(host, dtype=torch.int64,
                                    device=pools[0].device)

    def args(self, copy_pairs, num_pairs=None) -> _abi.KdaCopyArgs:
        """kda_copy_args for these pairs."""
        pairs, n = _pairs(copy_pairs)
        return _abi.KdaCopyArgs(
            self._tables.data_ptr(),
            ctypes.cast(self._host, ctypes.POINTER(ctypes.c_int64)), pairs,
            _ints(num_pairs, "num_pairs", 1), self.num_blocks,
            len(self.pools), n, self.null_block_id, 0)

    def check(self, copy_pairs, num_pairs=None) -> int:
        """Host-only validation (no launch); returns the kda_status code."""
        return _abi.load().kda_check_copy_blocks(
            ctypes.byref(self.args(copy_pairs, num_pairs)))

    def copy(self, copy_pairs, num_pairs=None, *, stream=None) -> None:
        """Copies block `copy_pairs[i, 0]` to `copy_pairs[i, 1]` in every pool,
        for the first `num_pairs` (a one-element tensor; default: all) pairs
        (kda_copy_args in include/kda_recoverssm.h)."""
        _launch(_abi.load().kda_copy_blocks, self.args(copy_pairs, num_pairs),
                dict(pairs=copy_pairs, num=num_pairs, tables=self._tables),
                stream)


def _dense(t) -> bool:
    """Whether a tensor's elements fill one piece of memory, in any order of
    its dimensions."""
    dims = sorted((st, n) for st, n in zip(t.stride(), t.shape) if n > 1)
    want = 1
    for st, n in dims:
        if st != want:
            return False
        want *= n
    return True


_FORK_PACK = struct.Struct("<" + _pack_format(_abi.KdaForkArgs))


def fork_args(*, parent_rows, child_rows, num_computed_tokens, num_blocks,
              block_table, free_blocks, block_size, copy_pairs, num_allocated,
              null_block_id=0) -> _abi.KdaForkArgs:
    """kda_fork_args for these tensors."""
    F = parent_rows.shape[0]
    table, strides, rows, width = _table(block_table, parent_rows, 0)
    pairs, n = _pairs(copy_pairs)
    if n < F:
        raise ValueError("copy_pairs needs a pair per fork")
    vals = (_ints(parent_rows, "parent_rows", F),
            _ints(child_rows, "child_rows", F),
            _ints(num_computed_tokens, "num_computed_tokens", rows),
            _ints(num_blocks, "num_blocks", rows), table, *strides,
            _ints(free_blocks, "free_blocks", 0), pairs,
            _ints(num_allocated, "num_allocated", 1), F, rows, width,
            block_size, free_blocks.shape[0], null_block_id)
    return _abi.KdaForkArgs.from_buffer_copy(_FORK_PACK.pack(*vals))


def check_fork_blocks(**kwargs) -> int:
    """Host-only validation (no launch); returns the kda_status code."""
    return _abi.load().kda_check_fork_blocks(ctypes.byref(fork_args(**kwargs)))


def fork_blocks(*, stream=None, **kwargs) -> None:
    """Child rows that continue their parents' tokens: whole blocks shared, the
    running one new (kda_fork_args in include/kda_recoverssm.h).  Updates
    `block_table`, `num_blocks` and `num_computed_tokens` in place;
    `BlockPools.copy(copy_pairs)` then copies the running blocks; of a longer
    `copy_pairs`, `copy_pairs[:forks]` (the rows behind stay as they were)."""
    _launch(_abi.load().kda_fork_blocks, fork_args(**kwargs), kwargs, stream)


def blocks_workspace_size(total_blocks: int) -> int:
    """Bytes of workspace of `free_blocks` and `compact_blocks`."""
    n = _abi.load().kda_blocks_workspace_size(total_blocks)
    if n <= 0:
        raise ValueError("too many blocks")
    return n


_FREE_PACK = struct.Struct("<" + _pack_format(_abi.KdaFreeArgs))


def free_args(*, released_rows, block_table, num_blocks, new_num_blocks,
              ref_counts, free_blocks, num_free, workspace, pinned=None,
              null_block_id=0) -> _abi.KdaFreeArgs:
    """kda_free_args for these tensors."""
    R, N = released_rows.shape[0], ref_counts.shape[0]
    table, strides, rows, width = _table(block_table, released_rows, 0)
    work, size = _workspace(workspace)
    vals = (_ints(released_rows, "released_rows", R), table, *strides,
            _ints(num_blocks, "num_blocks", rows), _ints(pinned, "pinned", N),
            _ints(new_num_blocks, "new_num_blocks", rows),
            _ints(ref_counts, "ref_counts", N),
            _ints(free_blocks, "free_blocks", N),
            _ints(num_free, "num_free", 1), work, size, R, rows, width, N,
            null_block_id, 0)
    return _abi.KdaFreeArgs.from_buffer_copy(_FREE_PACK.pack(*vals))


def check_free_blocks(**kwargs) -> int:
    """Host-only validation (no launch); returns the kda_status code."""
    return _abi.load().kda_check_free_blocks(ctypes.byref(free_args(**kwargs)))


def free_blocks(*, stream=None, **kwargs) -> None:
    """Releases rows, counts the references of every block anew and lists the
    free ones in rising order, as `step_tables` takes them
    (kda_free_args in include/kda_recoverssm.h).  The number of blocks is that
    of `ref_counts`."""
    _launch(_abi.load().kda_free_blocks, free_args(**kwargs), kwargs, stream)


_COMPACT_PACK = struct.Struct("<" + _pack_format(_abi.KdaCompactBlocksArgs))


def compact_blocks_args(*, ref_counts, block_table, num_blocks,
                        new_block_table, new_ref_counts, copy_pairs,
                        num_pairs, workspace,
                        null_block_id=0) -> _abi.KdaCompactBlocksArgs:
    """kda_compact_blocks_args for these tensors."""
    N = ref_counts.shape[0]
    table, strides, rows, width = _table(block_table, ref_counts, 0)
    new, new_strides, new_rows, new_width = _table(new_block_table,
                                                   ref_counts, 0)
    if (rows, width) != (new_rows, new_width):
        raise ValueError("block_table and new_block_table must be of one "
                         "size")
    pairs, n = _pairs(copy_pairs)
    work, size = _workspace(workspace)
    vals = (_ints(ref_counts, "ref_counts", N), table, *strides,
            _ints(num_blocks, "num_blocks", rows), new, *new_strides,
            _ints(new_ref_counts, "new_ref_counts", N), pairs,
            _ints(num_pairs, "num_pairs", 1), work, size, n, rows, width, N,
            null_block_id, 0)
    return _abi.KdaCompactBlocksArgs.from_buffer_copy(
        _COMPACT_PACK.pack(*vals))


def check_compact_blocks(**kwargs) -> int:
    """Host-only validation (no launch); returns the kda_status code."""
    return _abi.load().kda_check_compact_blocks(
        ctypes.byref(compact_blocks_args(**kwargs)))


def compact_blocks(*, stream=None, **kwargs) -> None:
    """Plans the moves that bring every live block to the lowest ids, and
    rewrites block table and reference counts (kda_compact_blocks_args in
    include/kda_recoverssm.h); `BlockPools.copy(copy_pairs, num_pairs)` then
    makes the moves.  Pinned blocks move, too: a holder of ids outside the
    block table applies the pairs to them and to its `pinned` counts:

        src, dst = copy_pairs[:int(num_pairs)].long().t()
        pinned[dst], pinned[src] = pinned[src], 0
    """
    _launch(_abi.load().kda_compact_blocks, compact_blocks_args(**kwargs),
            kwargs, stream)
