// prompt_common.cuh -- what the prompt attention's kernels share (sm_103a): a request's
// queries and keys, and which tiles of keys a row tile visits.
#pragma once

#include "kv_common.cuh"

namespace specv {

struct PromptParams {
    const void *q, *k, *v;
    void *out;
    float *lse;
    const int32_t *cu_q, *cu_k;
    int32_t *status;
    int64_t ld_q, ld_k, ld_v;
    int B, n_q, n_k, max_query, Hq, H, group, D, window, sinks;
    float scale_log2;
    int parts;        // of an item's tiles (tensor cores: at most), joined afterwards if more than one
    float *part_o;    // [parts][n_q * Hq][D]
    float2 *part_ml;  // [parts][n_q * Hq]: reference and sum
};

// How the tensor-core kernel cuts a call, from what the host knows of it.
struct PromptPlan {
    int tokens, subs;  // of a row tile; row tiles an item
    int64_t items;     // at most
    int parts;
    size_t bytes;      // of the parts' results
};
inline PromptPlan prompt_plan(int n_q, int n_k, int B, int group, int H, int D, int window, int sinks) {
    constexpr int kSms = 152, kMostParts = 32, kLeastTiles = 8;  // parts: a lane each in the join
    PromptPlan x = {};
    x.tokens = 128 / group;
    x.parts = 1;
    // pairs of row tiles (heads of up to 128 columns), which keep the tensor cores busier;
    // single ones where there is an SM for each (203 tokens of 32 heads: 11.4 us, in pairs 12.8)
    const int64_t pairs = (((int64_t)n_q + 2 * x.tokens - 1) / (2 * x.tokens) + B) * H;
    x.subs = D > 128 || 2 * pairs <= kSms ? 1 : 2;
    x.items = (((int64_t)n_q + x.subs * x.tokens - 1) / (x.subs * x.tokens) + B) * H;
    // Fewer items than SMs, over many keys: each one's tiles in parts, eight tiles or more on
    // average (a part costs its rows' sums in fp32, written and read).  The kernel, which knows
    // the lengths, cuts each request into as many parts as its length asks for, up to x.parts.
    int64_t keys = (int64_t)n_k / B - n_q / B / 2;
    if (window > 0 && keys > (int64_t)window + sinks) keys = (int64_t)window + sinks;
    const int64_t most = keys / 128 / kLeastTiles;
    if (x.items < kSms && B <= 128 && most > 1) {
        x.parts = (int)(most < kMostParts ? most : kMostParts);
        if (D <= 128) x.subs = 2;
        x.items = (((int64_t)n_q + x.subs * x.tokens - 1) / (x.subs * x.tokens) + B) * H;
        const int64_t want = (6 * kSms + x.items - 1) / x.items;
        if (x.parts > want) x.parts = (int)want;
    }
    if (x.parts > 1) x.bytes = (size_t)x.parts * n_q * group * H * (D + 2) * sizeof(float);
    return x;
}

struct Prompt {
    int row0, n, key0, m;  // first query row, queries, first key row, keys; n = 0 where unusable
    bool ok;
};

__device__ __forceinline__ Prompt load_prompt(const PromptParams &p, int b) {
    Prompt r;
    r.row0 = p.cu_q[b];
    const int row1 = p.cu_q[b + 1];
    r.key0 = p.cu_k[b];
    const int key1 = p.cu_k[b + 1];
    r.ok = r.row0 >= 0 && row1 >= r.row0 && row1 <= p.n_q && r.key0 >= 0 && key1 >= r.key0 && key1 <= p.n_k;
    r.n = row1 - r.row0;
    r.m = key1 - r.key0;
    r.ok = r.ok && r.n <= p.max_query;
    if (!r.ok) r.n = r.m = 0;
    return r;
}

__device__ __forceinline__ void write_prompt_statuses(const PromptParams &p, int first, int step) {
    for (int b = first; b < p.B; b += step) p.status[b] = load_prompt(p, b).ok ? SPEC_STATUS_OK : SPEC_STATUS_BAD_LENGTH;
}

// Key tiles of a row tile: [0, s1) hold first tokens kept visible, [w0, end) the rest.
struct Span {
    int s1, w0, count;
    __device__ __forceinline__ int tile(int i) const { return i < s1 ? i : w0 + (i - s1); }
};
template <int TK>
__device__ __forceinline__ Span span_of(const PromptParams &p, int pos0, int pos1) {
    Span s = {0, 0, 0};
    if (pos1 < 0) return s;
    const int low = p.window > 0 ? max(0, max(0, pos0) - p.window + 1) : 0;  // below it only sinks are seen
    s.w0 = low / TK;
    s.s1 = min((min(p.sinks, low) + TK - 1) / TK, s.w0);
    s.count = s.s1 + pos1 / TK + 1 - s.w0;
    return s;
}
__device__ __forceinline__ bool visible(const PromptParams &p, int pos, int j) {
    return j <= pos && (p.window == 0 || j > pos - p.window || j < p.sinks);
}

// The parts for fp32 arithmetic: row tiles of 64 rows or more, key tiles of 64, which take so
// long there that three make a part (64 queries after 8000 keys, 8 heads of 128: 1770 us whole,
// 89 in parts).
inline int rows_parts(int n_q, int n_k, int B, int group, int H, int window, int sinks) {
    constexpr int kSms = 152, kMostParts = 32, kLeastTiles = 3;
    const int64_t items = ((int64_t)n_q * group / 64 + B) * H;
    int64_t keys = (int64_t)n_k / B - n_q / B / 2;
    if (window > 0 && keys > (int64_t)window + sinks) keys = (int64_t)window + sinks;
    const int64_t most = keys / 64 / kLeastTiles, want = (4 * kSms + items - 1) / items;
    if (items >= 2 * kSms || most < 2 || want < 2) return 1;
    const int64_t parts = want < most ? want : most;
    return (int)(parts < kMostParts ? parts : kMostParts);
}

// prompt_join_kernel (prompt_tc.cu), for outputs in bf16 or fp32.
int launch_prompt_join(const PromptParams &p, bool bf16, cudaStream_t st);

// The tensor-core kernel (prompt_tc.cu); SPEC_EUNSUPPORTED where it cannot serve the call.
int launch_prompt_tc(const PromptParams &p, int dev, int sms, cudaStream_t st);

}  // namespace specv
