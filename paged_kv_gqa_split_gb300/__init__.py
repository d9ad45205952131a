"""GB300 (sm_103a) paged-KV GQA decode: h32 / kv4 / d128 / page size 1, bf16.

``run(q, k_cache, v_cache, kv_indptr, kv_indices, sm_scale=None) -> (out, lse)``
calls the CUDA library through its C ABI (include/gqa_paged_decode.h). The
library is built in-tree by ``paged_kv_gqa_split_gb300.build.build()``; it is
loaded on first use, and every call fails loudly if it is missing.
``sparse_run(q, k_cache, v_cache, logical_indices, block_table, token_to_req)``
is the selected-token variant over a block table of any page size,
``run_fp8`` reads an FP8 (e4m3, per-128 fp32 scale) cache, ``mla_run`` is
the dense MLA decode over one 576-value latent KV head (``mla_workspace_size``:
the bytes of a workspace of the caller's for it), and
``kv_append`` stores new tokens' K/V rows into the page pool.

What a serving step runs around them (``serving``): ``rope_inv_freq`` and
``rope`` (rotary positions), ``rope_kv_append`` (Q and K turned, K and V stored
in a bf16 or FP8 cache), ``kv_append_fp8``, ``kv_read_fp8`` and
``mla_kv_append`` (the caches' write and read), and latent attention's
``mla_absorb_q``, ``mla_expand_out``, ``mla_absorbed_run`` (new tokens) and
``mla_prefill`` (prompts).
"""
from ._lib import (GqaError, kv_append, mla_run, mla_workspace_size, run, run_checked, run_fp8,  # noqa: F401
                   sparse_run)
from .serving import (kv_append_fp8, kv_read_fp8, mla_absorb_q, mla_absorbed_run, mla_expand_out,  # noqa: F401
                      mla_kv_append, mla_prefill, rope, rope_inv_freq, rope_kv_append)

__all__ = ["GqaError", "kv_append", "kv_append_fp8", "kv_read_fp8", "mla_absorb_q", "mla_absorbed_run",
           "mla_expand_out", "mla_kv_append", "mla_prefill", "mla_run", "mla_workspace_size", "rope", "rope_inv_freq",
           "rope_kv_append", "run", "run_checked", "run_fp8", "sparse_run"]
