"""GB300 speculative-sampling verifier.

The verify step of speculative decoding (Algorithm 1 of Leviathan et al.; see
include/specdec.h for the exact contract) runs in hand-written CUDA kernels in
``libspecdec.so``; this package only marshals torch tensors into the C ABI.

    from speculative_decoding_rejection_decode_gb300 import Verifier
    v = Verifier(device=0)
    out = v(target_logits, draft_probs, draft_ids, cu_num_draft_tokens, T=1.0, seed=0)
    out.tokens, out.num_accepted, out.beta

    from speculative_decoding_rejection_decode_gb300 import KVCache, rotary_table
    cache = KVCache.empty(v, num_pages, page_size, kv_heads, head_dim, torch.float8_e4m3fn)
    q = cache.append(k, v_rows, page_table, lengths, cu_num_nodes, node_parent, q=q, rotary=table)
    o = cache.attend(q, page_table, lengths, cu_num_nodes, node_parent)
    lengths = cache.commit(page_table, lengths, cu_num_nodes, out.num_accepted, out.path)

The library is loaded on first use of anything below (``Verifier``,
``uniform``, the ``specdec_*`` functions); that raises ImportError when
libspecdec.so has not been built.  ``inputs`` (synthetic workloads) needs no
library.
"""
from __future__ import annotations

_LAZY = {"Verifier", "VerifyOutput", "SpecdecError", "uniform", "neg_log_uniform",
         "specdec_create", "specdec_reserve", "specdec_rejection_sample",
         "specdec_rejection_sample_ex", "specdec_rejection_sample_topk_topp",
         "specdec_get_error", "specdec_set_path", "specdec_set_timing_events",
         "specdec_set_adjust_counters", "specdec_last_path", "specdec_uniform",
         "specdec_neg_log_uniform", "specdec_selection_mass", "selection_mass",
         "specdec_status_string", "specdec_destroy",
         "specdec_rejection_sample_noalloc", "specdec_tree_verify", "TreeOutput",
         "specdec_rejection_sample_given", "specdec_logprobs", "specdec_logprobs_grad", "LogprobOutput",
         "specdec_rotate", "rotary_axes", "tree_rows", "SPECDEC_MAX_TOP", "SPECDEC_MAX_AXES",
         "SPECDEC_F32", "SPECDEC_BF16",
         "SPECDEC_PATH_AUTO", "SPECDEC_PATH_FUSED", "SPECDEC_PATH_TWO_PASS", "SPECDEC_PATH_SWEEP",
         "SPECDEC_PATH_STREAM", "SPECDEC_PATH_PAIR", "SPECDEC_PATH_DUAL", "SPECDEC_PATH_GREEDY"}


_LAZY_CACHE = {"KVCache", "rotary_table", "specdec_cache_append", "specdec_cache_read",
               "specdec_tree_attention", "specdec_tree_attention_workspace",
               "specdec_cache_append_positions", "specdec_cross_attention",
               "specdec_cross_attention_workspace", "specdec_cache_commit", "SPECDEC_F16", "SPECDEC_E4M3"}


def __getattr__(name):
    if name in _LAZY_CACHE:
        from . import cache
        return getattr(cache, name)
    if name in _LAZY:
        from . import verifier
        return getattr(verifier, name)
    raise AttributeError(name)
