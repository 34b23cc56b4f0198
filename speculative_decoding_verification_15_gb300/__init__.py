"""GB300-native batched speculative-decoding verify/commit (CUDA kernels for sm_103a).

The compute path is libspecverify.so (C ABI in include/spec_verify.h); this package
only builds it and marshals torch tensors into it.
"""
from . import _build, binding  # noqa: F401
from .api import (cache_attention, cache_attention_reset, kv_append, kv_cache, kv_gather, kv_plan, kv_pool,  # noqa: F401
                  markov_draft, markov_draft_topk, prompt_attention, rotary, rotary_frequencies,
                  schedule_threshold, schedule_verify_len, schedule_verify_len_stale,
                  verify_greedy, verify_greedy_early_exit, verify_greedy_flat, verify_sample,
                  verify_sample_early_exit, verify_sample_flat,
                  verify_sample_host, workspace)
from .binding import (KVCache, PagePool, SpecError, spec_cache_attention,  # noqa: F401
                      spec_cache_attention_workspace_size, spec_kv_append, spec_kv_gather, spec_kv_plan,
                      spec_markov_draft, spec_markov_draft_topk, spec_markov_topk_workspace_size,
                      spec_prompt_attention, spec_prompt_attention_workspace_size, spec_rotary,
                      spec_schedule_threshold, spec_schedule_verify_len,
                      spec_schedule_verify_len_stale, spec_verify_greedy, spec_verify_greedy_early_exit,
                      spec_verify_greedy_flat, spec_verify_sample, spec_verify_sample_early_exit,
                      spec_verify_sample_flat, spec_verify_sample_noalloc,
                      spec_verify_workspace_size)


def build(force: bool = False) -> str:
    return _build.build(force=force)
