"""NSA selection-attention forward for GB300 (sm_103a).

Public API (GPU only; the CUDA library must be built):

* :func:`sel_attn_fwd` -- O [B,M,H,D] and LSE [B,H,M] fp32 from fp16 or
  bf16 Q [B,M,H,D], K/V [B,N,G,D] and int32 block_indices [B,M,G,T];
* :func:`sel_attn_bwd` -- dQ, dK, dV from dO and the forward's O and LSE;
* :func:`topk_blocks` -- block_indices from per-block scores (top-k with
  forced initial and local blocks);
* :func:`sel_attn_fwd_shared` -- the same forward in two passes: the blocks
  common to a tile of 16 consecutive queries are gathered once per tile;
* :func:`sel_attn_fwd_host` -- the forward with host buffers in and out;
* :func:`swa_fwd` -- GQA sliding-window (or dense) attention forward on the
  tcgen05 tensor cores;
* :func:`swa_bwd` -- dQ, dK, dV from dO and that forward's O and LSE;
* :func:`qk_norm_rope` and :func:`qk_norm_rope_bwd` -- RMS norm of every
  query and key head and the position rotation in one pass, before any of
  the attention calls, and its gradients (:func:`rope_tables` builds the
  angle tables);
* :class:`KvCache` (:func:`kv_cache` makes an empty one): a paged cache of keys
  and values, 16-bit or 4-bit; :func:`kv_append` -- norm and rotation of new
  tokens, with K and V stored in it; :func:`paged_attn` -- their attention over
  the pages, with a window and first tokens; :func:`kv_read` -- rows of it as K
  and V.

The C ABI is declared in ``include/nsa_sel_attn.h``; ``inputs`` draws the
seeded synthetic workloads.
"""

from ._lib import (KvCache, NsaError, kv_append, kv_cache, kv_read, load, paged_attn,   # noqa: F401
                   qk_norm_rope, qk_norm_rope_bwd, rope_tables,
                   sel_attn_bwd, sel_attn_fwd, sel_attn_fwd_host, sel_attn_fwd_shared,
                   status_string, swa_bwd, swa_fwd, topk_blocks)

__all__ = ["sel_attn_fwd", "sel_attn_fwd_shared", "sel_attn_bwd", "sel_attn_fwd_host",
           "topk_blocks", "swa_fwd", "swa_bwd", "qk_norm_rope", "qk_norm_rope_bwd", "rope_tables",
           "KvCache", "kv_cache", "kv_append", "kv_read", "paged_attn",
           "load", "status_string", "NsaError"]
