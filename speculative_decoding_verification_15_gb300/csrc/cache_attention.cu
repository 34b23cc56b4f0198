// cache_attention.cu -- the verify step's attention over the 8-bit paged cache (sm_103a).
//
// Mathematics.  With log2 scores x_j = scale * log2(e) * (q . k_j) and a reference m,
//   out = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m),
// computed in one pass over the cache: each part of the tokens keeps (m, l, o) with
// l = sum 2^(x_j - m), o = sum 2^(x_j - m) v_j, and two parts join as
//   m = max(m1, m2), l = l1 2^(m1 - m) + l2 2^(m2 - m), o likewise.
//
// Work split.  What has to be read is the cache, once: an item is (request, key head,
// row tile), its rows the queries of the request that share the key head (token-major:
// row = t * group + g), and its length is counted in tiles of kTile tokens.  All tiles
// of all items in order are one line that is cut into equal parts, one for each CTA,
// so long and short requests together, one long request alone and a full batch all
// load every SM alike.  A CTA whose part holds an item whole writes its output; an
// item cut by a boundary leaves (m, l, o) of each part in the workspace, and the part
// that arrives last (a counter; nobody waits) joins them in CTA order.
#include "kv_common.cuh"

namespace specv {
namespace {

constexpr int kTile = 128;      // tokens of a tile: a multiple of every page size
constexpr int kMaxCtas = 320;   // CTAs at most; sizes the workspace
constexpr int kMaxRows = 64;    // rows of a row tile at most
constexpr float kLn2 = 0.6931471805599453f;

struct AttnParams {
    spec_kv_cache c;
    const void *q;
    void *out;
    float *lse;
    const int32_t *cu, *seq_len, *table;
    int32_t *status;
    int64_t ld_q;
    int B, ld_table, n_tokens, max_query, Hq, group, window, sinks;
    float scale_log2;  // scale * log2(e)
    int *tickets;      // [kMaxCtas], zero between calls
    float *partial;    // [2 * kMaxCtas][rows * (D + 2)]
};

// What a request asks for, with its positions and its tiles.
struct Request {
    int n, len, row0;    // queries, cached tokens, first query row; n = 0 where unusable
    int low, sinks;      // tokens below `low` are seen only below `sinks` (<= low)
    int s1, w0, nt, rt;  // tiles [0, s1) and [w0, ...), nt in all; row tiles
    bool ok;
};

__device__ __forceinline__ Request load_request(const AttnParams &p, int b, int rows) {
    Request r;
    r.row0 = p.cu[b];
    const int row1 = p.cu[b + 1];
    r.len = p.seq_len[b];
    r.n = row1 - r.row0;
    r.ok = r.row0 >= 0 && row1 >= r.row0 && row1 <= p.n_tokens && r.n <= p.max_query && r.len >= 0 &&
           r.len <= (int64_t)p.ld_table * p.c.page_size;
    if (!r.ok) r.n = r.len = 0;
    const int first = r.len - r.n;  // position of the first query
    r.low = p.window > 0 ? max(0, first - p.window + 1) : 0;
    r.sinks = min(p.sinks, r.low);
    r.w0 = r.low / kTile;
    r.s1 = min((r.sinks + kTile - 1) / kTile, r.w0);
    r.nt = max(1, r.s1 + (r.len + kTile - 1) / kTile - r.w0);
    r.rt = (int)(((int64_t)r.n * p.group + rows - 1) / rows);
    return r;
}

__device__ __forceinline__ int64_t request_tiles(const AttnParams &p, const Request &r) {
    return (int64_t)p.c.num_heads * r.rt * r.nt;
}

// A CTA's place on the line of tiles: [u, end), starting `off` tiles into request b.
// Only as many CTAs as there are tiles take part, so that no share among them is empty
// and the parts of a cut item are those of consecutive CTAs.
struct Share {
    int64_t total, u, end, off;
    int b, ctas;
};

__device__ __forceinline__ int64_t share_start(int64_t total, int cta, int ctas) { return total * cta / ctas; }
// The CTA whose share holds tile u.
__device__ __forceinline__ int cta_of(int64_t total, int64_t u, int ctas) {
    return (int)(((u + 1) * ctas - 1) / total);
}

// Every thread of the CTA calls it (it synchronises); NT threads.
template <int NT>
__device__ Share find_share(const AttnParams &p, int rows) {
    __shared__ int64_t s_warp[NT / 32];
    __shared__ Share s_share;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + NT - 1) / NT, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b) sum += request_tiles(p, load_request(p, b, rows));
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[warp] = incl;
    if (tid == 0) s_share.b = p.B;
    __syncthreads();
    int64_t before = incl - sum, total = 0;
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    const int ctas = (int)min((int64_t)gridDim.x, total), cta = blockIdx.x;
    const int64_t u = cta < ctas ? share_start(total, cta, ctas) : 0;
    const int64_t end = cta < ctas ? share_start(total, cta + 1, ctas) : 0;
    if (u < end && u >= before && u < before + sum) {  // one thread: its requests hold tile u
        int b = b0;
        int64_t off = u - before;
        for (;;) {
            const int64_t t = request_tiles(p, load_request(p, b, rows));
            if (off < t) break;
            off -= t;
            ++b;
        }
        s_share.b = b;
        s_share.off = off;
    }
    __syncthreads();
    Share s = s_share;
    s.total = total;
    s.u = u;
    s.end = end;
    s.ctas = ctas;
    return s;
}

// One part of one item: tiles [t0, t1) of the nt of (b, h, row tile rt).
struct Part {
    Request r;
    int b, h, rt, t0, t1;
    int64_t item;  // the item's first tile on the line
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == r.nt; }
    __device__ __forceinline__ int tile(int i) const { return i < r.s1 ? i : r.w0 + (i - r.s1); }
};

// The share's next part; call while s.u < s.end.
__device__ __forceinline__ Part next_part(const AttnParams &p, Share &s, int rows) {
    Part x;
    for (;;) {
        x.r = load_request(p, s.b, rows);
        if (s.off < request_tiles(p, x.r)) break;
        s.off = 0;  // a share's next request is entered at its first tile
        ++s.b;
    }
    x.b = s.b;
    const int64_t i = s.off / x.r.nt;
    x.t0 = (int)(s.off - i * x.r.nt);
    x.h = (int)(i / x.r.rt);
    x.rt = (int)(i - (int64_t)x.h * x.r.rt);
    x.item = s.u - x.t0;
    const int64_t left = s.end - s.u;
    x.t1 = (int)min((int64_t)x.r.nt, x.t0 + left);
    s.u += x.t1 - x.t0;
    s.off += x.t1 - x.t0;
    return x;
}

// Lengths and pages of the requests, told by one warp for every gridDim.x-th request.
__device__ __forceinline__ void write_statuses(const AttnParams &p, int lane) {
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const Request r = load_request(p, b, 1);
        bool bad = false;
        if (r.n > 0) {
            const int bs = p.c.page_size, np = (r.len + bs - 1) / bs, ns = (r.sinks + bs - 1) / bs;
            const int32_t *t = p.table + (int64_t)b * p.ld_table;
            for (int i = lane; i < ns; i += 32) bad |= t[i] < 0 || t[i] >= p.c.num_pages;
            for (int i = r.low / bs + lane; i < np; i += 32) bad |= t[i] < 0 || t[i] >= p.c.num_pages;
        }
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0)
            p.status[b] = !r.ok ? SPEC_STATUS_BAD_LENGTH : (bad ? SPEC_STATUS_BAD_PAGE : SPEC_STATUS_OK);
    }
}

// ------------------------------------------------------------------ joining parts
// A part's slot: the first part of an item is its CTA's last part, every other part
// its CTA's first, so two slots a CTA are enough.
__device__ __forceinline__ float *slot_of(const AttnParams &p, int cta, bool first, int rows) {
    return p.partial + (int64_t)(2 * cta + (first ? 1 : 0)) * rows * (p.c.head_dim + 2);
}

// Output element (row r of the part's row tile, column d).
template <typename T>
__device__ __forceinline__ void store_out(const AttnParams &p, const Part &x, int row, int d, float v) {
    const int t = row / p.group, g = row - t * p.group;
    const int64_t at = ((int64_t)(x.r.row0 + t) * p.Hq + x.h * p.group + g) * p.c.head_dim + d;
    if constexpr (sizeof(T) == 2) ((uint16_t *)p.out)[at] = (uint16_t)pack_bf16x2(v, 0.f);
    else ((float *)p.out)[at] = v;
}
__device__ __forceinline__ void store_lse(const AttnParams &p, const Part &x, int row, float m, float l) {
    const int t = row / p.group, g = row - t * p.group;
    p.lse[(int64_t)(x.r.row0 + t) * p.Hq + x.h * p.group + g] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
}
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }

// 2^(a - m), 0 where the part a comes from saw nothing (a = -inf, whatever m is).
__device__ __forceinline__ float weight_of(float a, float m) { return a == kNegInf ? 0.f : exp2f(a - m); }

// Counts this CTA's part of a cut item in; true (in every thread) for the part that
// arrives last, which may then read the other parts.  NT threads call it, `bar` a
// named barrier of theirs.
template <int NT>
__device__ __forceinline__ bool arrive_last(const AttnParams &p, int first_cta, int parts, int *s_flag, int bar) {
    __threadfence();
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(NT) : "memory");
    if (threadIdx.x == 0) {
        const int before = atomicAdd(p.tickets + first_cta, 1);
        *s_flag = before == parts - 1;
        if (before == parts - 1) p.tickets[first_cta] = 0;  // for the next call
    }
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(NT) : "memory");
    const bool last = *s_flag != 0;
    if (last) __threadfence();
    return last;
}

// Joins the parts of an item in CTA order and writes its rows.  s_w: 2 * rows floats.
template <typename T, int NT>
__device__ void join_parts(const AttnParams &p, const Part &x, int rows, int nrows, int c0, int c1, float *s_w,
                           int bar) {
    const int D = p.c.head_dim, tid = threadIdx.x;
    for (int r = tid; r < nrows; r += NT) {
        float m = kNegInf, l = 0.f;
        for (int c = c0; c <= c1; ++c) {
            const float *s = slot_of(p, c, c == c0, rows) + (int64_t)rows * D;
            const float mc = __ldcg(s + r), lc = __ldcg(s + rows + r);
            const float mn = fmaxf(m, mc);
            l = l * weight_of(m, mn) + lc * weight_of(mc, mn);
            m = mn;
        }
        s_w[r] = m;
        s_w[rows + r] = inverse_sum(l);
        if (p.lse) store_lse(p, x, x.rt * rows + r, m, l);
    }
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(NT) : "memory");
    for (int i = tid; i < nrows * D; i += NT) {
        const int r = i / D, d = i - r * D;
        float o = 0.f;
        for (int c = c0; c <= c1; ++c) {
            const float *s = slot_of(p, c, c == c0, rows);
            o = fmaf(__ldcg(s + i), weight_of(__ldcg(s + (int64_t)rows * D + r), s_w[r]), o);
        }
        store_out<T>(p, x, x.rt * rows + r, d, o * s_w[rows + r]);
    }
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(NT) : "memory");
}

// ------------------------------------------------------------------ fp32 arithmetic kernel
// Four warps, each 32 tokens of a tile: a lane holds one token's scores of kSimtRows
// rows (its key row read 16 codes at a time, the queries broadcast from shared
// memory), then the warp walks its tokens with the lanes over the head's columns.
// Every warp keeps its own (m, l, o); they join in shared memory at the part's end.
constexpr int kSimtRows = 8, kSimtThreads = 128;

template <typename T, int ND>
__global__ void __launch_bounds__(kSimtThreads) attention_simt_kernel(AttnParams p) {
    constexpr int R = kSimtRows;
    __shared__ __align__(16) float s_q[R][128 * ND];
    __shared__ float s_p[4][32][R];
    __shared__ float s_m[4][R], s_l[4][R], s_w[2 * R];
    __shared__ __align__(16) float s_o[R][128 * ND];
    __shared__ int s_flag;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = p.c.head_dim, bs = p.c.page_size;
    if (warp == 0) write_statuses(p, lane);
    Share share = find_share<kSimtThreads>(p, R);
    while (share.u < share.end) {
        const Part x = next_part(p, share, R);
        const int nrows = min(R, x.r.n * p.group - x.rt * R);
        const int first = x.r.len - x.r.n;
        __syncthreads();  // the part before is done with shared memory
        for (int i = tid; i < R * D; i += kSimtThreads) {
            const int r = i / D, d = i - r * D;
            float v = 0.f;
            if (r < nrows) {
                const int row = x.rt * R + r, t = row / p.group, g = row - t * p.group;
                v = ld_elem<sizeof(T)>(p.q, (int64_t)(x.r.row0 + t) * p.ld_q + (int64_t)(x.h * p.group + g) * D + d) *
                    p.scale_log2;
            }
            s_q[r][d] = v;
        }
        __syncthreads();
        float m[R], l[R], o[R][4 * ND];
        int pos[R];  // the rows' positions; rows past the tile see nothing
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = kNegInf;
            l[r] = 0.f;
            pos[r] = r < nrows ? first + (x.rt * R + r) / p.group : -1;
#pragma unroll
            for (int e = 0; e < 4 * ND; ++e) o[r][e] = 0.f;
        }
        const int32_t *table = p.table + (int64_t)x.b * p.ld_table;
        for (int i = x.t0; i < x.t1; ++i) {
            const int j0 = x.tile(i) * kTile + warp * 32, j = j0 + lane;
            const bool held = j < x.r.len && (j >= x.r.low || j < x.r.sinks);
            int page = held ? table[j / bs] : -1;
            if (page >= p.c.num_pages) page = -1;
            const bool live = page >= 0;
            if (__ballot_sync(0xffffffffu, live) == 0) continue;
            const int64_t at = live ? (int64_t)page * p.c.page_stride + (int64_t)x.h * p.c.head_stride +
                                          (int64_t)(j % bs) * p.c.token_stride
                                    : 0;
            float ks = 0.f, vs = 0.f, s[R];
#pragma unroll
            for (int r = 0; r < R; ++r) s[r] = 0.f;
            if (live) {
                ks = __ldg(p.c.k_scale + (int64_t)page * p.c.num_heads + x.h);
                vs = __ldg(p.c.v_scale + (int64_t)page * p.c.num_heads + x.h);
                const char *kp = (const char *)p.c.k + at;
                for (int d = 0; d < D; d += 16) {
                    const uint4 q = __ldg((const uint4 *)(kp + d));
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 a = e4m3x2_to_float2(w[e] & 0xffffu), c = e4m3x2_to_float2(w[e] >> 16);
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const float4 f = *(const float4 *)&s_q[r][d + 4 * e];
                            s[r] = fmaf(a.x, f.x, fmaf(a.y, f.y, fmaf(c.x, f.z, fmaf(c.y, f.w, s[r]))));
                        }
                    }
                }
            }
            uint32_t sees = 0;  // rows that see this lane's token
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool see = live && j <= pos[r] && (p.window == 0 || j > pos[r] - p.window || j < p.sinks);
                sees |= see ? 1u << r : 0u;
                s[r] = see ? s[r] * ks : kNegInf;
                const float mn = fmaxf(m[r], warp_max(s[r]));  // a NaN score leaves the maximum alone
                const float ref = mn == kNegInf ? 0.f : mn;
                const float a = exp2f(m[r] - ref), w = see ? exp2f(s[r] - ref) : 0.f;
                m[r] = mn;
                l[r] = fmaf(l[r], a, warp_sum(w));
#pragma unroll
                for (int e = 0; e < 4 * ND; ++e) o[r][e] *= a;
                s_p[warp][lane][r] = w * vs;
            }
            __syncwarp();
            const uint32_t any = __ballot_sync(0xffffffffu, sees != 0);
            uint32_t all = sees;  // rows that see every token some row sees
            all = __reduce_and_sync(0xffffffffu, sees ? sees : 0xffffffffu);
            const uint32_t rows_in = (1u << nrows) - 1;
            const bool uniform = (all & rows_in) == rows_in;
            for (uint32_t todo = any; todo; todo &= todo - 1) {
                const int jj = __ffs(todo) - 1;
                const int64_t vat = __shfl_sync(0xffffffffu, at, jj);
                const uint32_t sj = __shfl_sync(0xffffffffu, sees, jj);
                const char *vp = (const char *)p.c.v + vat;
#pragma unroll
                for (int n = 0; n < ND; ++n) {
                    const int d = 128 * n + 4 * lane;
                    if (d < D) {
                        const uint32_t w = __ldg((const uint32_t *)(vp + d));
                        const float2 a = e4m3x2_to_float2(w & 0xffffu), c = e4m3x2_to_float2(w >> 16);
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            if (!uniform && !((sj >> r) & 1)) continue;  // 0 times a NaN is a NaN
                            const float f = s_p[warp][jj][r];
                            o[r][4 * n] = fmaf(f, a.x, o[r][4 * n]);
                            o[r][4 * n + 1] = fmaf(f, a.y, o[r][4 * n + 1]);
                            o[r][4 * n + 2] = fmaf(f, c.x, o[r][4 * n + 2]);
                            o[r][4 * n + 3] = fmaf(f, c.y, o[r][4 * n + 3]);
                        }
                    }
                }
            }
            __syncwarp();
        }
        // the four warps' sums join: references first, then warp after warp
        if (lane == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                s_m[warp][r] = m[r];
                s_l[warp][r] = l[r];
            }
        __syncthreads();
        float big[R];
#pragma unroll
        for (int r = 0; r < R; ++r) big[r] = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
        for (int w = 0; w < 4; ++w) {
            if (warp == w)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float f = weight_of(m[r], big[r]);
#pragma unroll
                    for (int n = 0; n < ND; ++n) {
                        const int d = 128 * n + 4 * lane;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float v = m[r] == kNegInf && l[r] == 0.f ? 0.f : o[r][4 * n + e] * f;
                            s_o[r][d + e] = w == 0 ? v : s_o[r][d + e] + v;
                        }
                    }
                }
            __syncthreads();
        }
        if (tid < R) {
            float mm = kNegInf, ll = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) mm = fmaxf(mm, s_m[w][tid]);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float f = s_m[w][tid] == kNegInf ? (s_l[w][tid] == 0.f ? 0.f : 1.f) : exp2f(s_m[w][tid] - mm);
                ll += s_l[w][tid] * f;
            }
            s_w[tid] = mm;
            s_w[R + tid] = ll;
        }
        __syncthreads();
        if (x.whole()) {
            for (int i = tid; i < nrows * D; i += kSimtThreads) {
                const int r = i / D, d = i - r * D;
                store_out<T>(p, x, x.rt * R + r, d, s_o[r][d] * inverse_sum(s_w[R + r]));
            }
            if (p.lse && tid < nrows) store_lse(p, x, x.rt * R + tid, s_w[tid], s_w[R + tid]);
        } else {
            float *slot = slot_of(p, blockIdx.x, x.t0 == 0, R);
            for (int i = tid; i < nrows * D; i += kSimtThreads) {
                const int r = i / D, d = i - r * D;
                slot[i] = s_o[r][d];
            }
            if (tid < nrows) {
                slot[R * D + tid] = s_w[tid];
                slot[R * D + R + tid] = s_w[R + tid];
            }
            const int c0 = cta_of(share.total, x.item, share.ctas);
            const int c1 = cta_of(share.total, x.item + x.r.nt - 1, share.ctas);
            if (arrive_last<kSimtThreads>(p, c0, c1 - c0 + 1, &s_flag, 1))
                join_parts<T, kSimtThreads>(p, x, R, nrows, c0, c1, s_w, 1);
        }
    }
}

}  // namespace
}  // namespace specv

using namespace specv;

extern "C" size_t spec_cache_attention_workspace_size(int num_query_heads, int num_heads, int head_dim, int dtype) {
    if (num_query_heads <= 0 || num_heads <= 0 || num_query_heads % num_heads || head_dim <= 0 || (head_dim & 15) ||
        head_dim > SPEC_KV_MAX_HEAD_DIM || (dtype != SPEC_BF16 && dtype != SPEC_F32))
        return 0;
    const size_t slot = sizeof(float) * kMaxRows * ((size_t)head_dim + 2);
    return sizeof(int) * kMaxCtas + 2 * kMaxCtas * slot;
}

extern "C" int spec_cache_attention(const spec_kv_cache *cache, const void *q, int dtype, int64_t ld_q,
                                    int num_query_heads, int n_tokens, int B, const int32_t *cu_query, int max_query,
                                    const int32_t *seq_len, const int32_t *page_table, int ld_table, float scale,
                                    int window, int sinks, void *out, float *out_lse, int32_t *out_status, void *ws,
                                    size_t ws_bytes, void *cuda_stream) {
    if (dtype != SPEC_BF16 && dtype != SPEC_F32) return SPEC_EINVAL;
    if (B < 0 || n_tokens < 0 || max_query < 0 || ld_table < 0 || num_query_heads <= 0 || window < 0 || sinks < 0)
        return SPEC_EINVAL;
    if (!(scale > 0.f) || !(scale * kLog2e < __builtin_huge_valf())) return SPEC_EINVAL;
    int rc = check_cache(cache);
    if (rc) return rc;
    if (num_query_heads % cache->num_heads) return SPEC_EINVAL;
    if (B == 0) return SPEC_OK;
    if (B > SPEC_MAX_BATCH) return SPEC_EUNSUPPORTED;
    if (!cu_query || !seq_len || !out_status || (ld_table > 0 && !page_table)) return SPEC_EINVAL;
    const int esz = dtype == SPEC_BF16 ? 2 : 4;
    if (n_tokens > 0 && (!q || !out || ld_q < (int64_t)num_query_heads * cache->head_dim)) return SPEC_EINVAL;
    if (((uintptr_t)q % esz) || ((uintptr_t)out % esz) || ((uintptr_t)out_lse & 3)) return SPEC_EINVAL;
    if ((int64_t)max_query * (num_query_heads / cache->num_heads) > 0x7fffffff - kMaxRows) return SPEC_EUNSUPPORTED;
    const size_t need = spec_cache_attention_workspace_size(num_query_heads, cache->num_heads, cache->head_dim, dtype);
    if (!ws || ws_bytes < need || ((uintptr_t)ws & 255)) return SPEC_EWORKSPACE;
    int dev = 0, sms = 0;
    if ((rc = kv_device_info(&dev, &sms))) return rc;
    if ((rc = kv_check_device_pointer(cache->k, dev))) return rc;
    AttnParams p = {};
    p.c = *cache;
    p.q = q;
    p.out = out;
    p.lse = out_lse;
    p.cu = cu_query;
    p.seq_len = seq_len;
    p.table = page_table;
    p.status = out_status;
    p.ld_q = ld_q;
    p.B = B;
    p.ld_table = ld_table;
    p.n_tokens = n_tokens;
    p.max_query = max_query;
    p.Hq = num_query_heads;
    p.group = num_query_heads / cache->num_heads;
    p.window = window < (1 << 30) ? window : (1 << 30);  // positions stay below 2^31
    p.sinks = window > 0 ? sinks : 0;
    p.scale_log2 = scale * kLog2e;
    p.tickets = (int *)ws;
    p.partial = (float *)((char *)ws + sizeof(int) * kMaxCtas);
    const cudaStream_t st = (cudaStream_t)cuda_stream;
    const int ctas = 2 * sms < kMaxCtas ? 2 * sms : kMaxCtas;
    if (cache->head_dim <= 128) {
        if (esz == 2) attention_simt_kernel<uint16_t, 1><<<ctas, kSimtThreads, 0, st>>>(p);
        else attention_simt_kernel<float, 1><<<ctas, kSimtThreads, 0, st>>>(p);
    } else {
        if (esz == 2) attention_simt_kernel<uint16_t, 2><<<ctas, kSimtThreads, 0, st>>>(p);
        else attention_simt_kernel<float, 2><<<ctas, kSimtThreads, 0, st>>>(p);
    }
    return launch_status();
}
