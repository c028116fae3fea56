"""Fused LM-head + exact Gumbel-max sampling (FlashSampling) for GB300, and the
operators beside it at the vocabulary ends of a model: token log-probabilities
with their gradient, the embedding lookup with its gradient; and speculative decoding:
an 8-bit head, probabilities, the verification of drafted tokens.

The compute path is the C-ABI library ``libfs.so`` (CUDA, sm_103a); this
package is its Python binding plus the seeded synthetic workloads used by the
tests and the benchmark.
"""
from ._binding import (FS_ERR_CUDA, FS_ERR_DEVICE_TIMEOUT, FS_ERR_INVALID_ARG,  # noqa: F401
                       FS_ERR_UNSUPPORTED, FS_ERR_WORKSPACE, FS_FLAG_OVERLAP_PREVIOUS, FS_MERGE_EXACT,
                       FS_MERGE_GROUP_GUMBEL, FS_OK, FS_SYNC_IDS, FS_SYNC_NONE, FS_SYNC_STREAM,
                       FS_BF16, FS_F32, FS_FP8_BLOCK, FS_LOGPROBS_TOPK_MAX,
                       FS_VERIFY_DRAFTS_MAX,
                       FS_TILE, FS_TOPK_MAX, LIB_PATH, FsError, FsLogprobs, FsLogprobsArgs,
                       FsLogprobsGradArgs, FsMatmulFp8Args, FsProbsArgs, FsQuantized,
                       FsSampleArgs, FsVerified, FsVerifyArgs, fs_embed, fs_embed_grad,
                       fs_embed_grad_workspace_size, fs_group_merge, fs_gumbel_noise, fs_gumbel_transform,
                       fs_last_device_error, fs_logprobs, fs_logprobs_grad,
                       fs_logprobs_grad_workspace_size, fs_logprobs_workspace_size,
                       fs_online_merge, fs_sample_topk, fs_topk_workspace_size,
                       fs_matmul_fp8, fs_num_tiles, fs_probs, fs_quantize, fs_sample, fs_sample_host, fs_status_string,
                       fs_verify, fs_wait_timeout_selftest,
                       fs_workspace_size,
                       load_library)
