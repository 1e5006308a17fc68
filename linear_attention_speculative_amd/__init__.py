"""MI355X-native KDA RecoverSSM speculative verify and commit.

The compute path is the HIP library `libkda_recoverssm.so` (C ABI in
include/kda_recoverssm.h); this package is its thin torch binding.
"""
from ._abi import LIB_PATH, load  # noqa: F401
from .blocks import (  # noqa: F401
    BlockPools,
    blocks_workspace_size,
    check_compact_blocks,
    check_fork_blocks,
    check_free_blocks,
    compact_blocks,
    compact_blocks_args,
    fork_args,
    fork_blocks,
    free_args,
    free_blocks,
)
from .cache import (  # noqa: F401
    adjust_logits,
    check_adjust_logits,
    check_latent_attention,
    check_latent_expand,
    check_latent_prefill,
    check_latent_write,
    latent_args,
    latent_attention,
    latent_attention_workspace_size,
    latent_expand,
    latent_expand_args,
    latent_prefill,
    latent_prefill_args,
    latent_write,
    latent_write_args,
    logits_args,
)
from .ops import (  # noqa: F401
    CommitContext,
    KdaError,
    KdaUnaligned,
    abi_version,
    check_verify,
    check_verify_qkv,
    conv_update_verify,
    conv_update_verify_noalloc,
    describe,
    reset_counter,
    set_launch_events,
    verify_args,
    verify_qkv,
)
from .serving import (  # noqa: F401
    check_decode,
    check_decode_qkv,
    check_prefill,
    check_prefill_qkv,
    check_sample,
    check_step_tables,
    conv_prefill,
    conv_update_decode,
    decode_args,
    decode_qkv,
    prefill_args,
    prefill_qkv,
    prefill_workspace_size,
    sample,
    sample_args,
    sample_workspace_size,
    step_tables,
    tables_args,
)
