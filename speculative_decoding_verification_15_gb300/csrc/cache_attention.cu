// cache_attention.cu -- the verify step's attention over the 8-bit paged cache (sm_103a).
//
// Mathematics.  With log2 scores x_j = scale * log2(e) * (q . k_j) and a reference m,
//   out = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m),
// computed in one pass over the cache: each part of the tokens keeps (m, l, o) with
// l = sum 2^(x_j - m), o = sum 2^(x_j - m) v_j, and two parts join as
//   m = max(m1, m2), l = l1 2^(m1 - m) + l2 2^(m2 - m), o likewise
// (with a reference of its own, so that the values' scales do not cost it its range).
//
// Work split.  What has to be read is the cache, once: an item is (request, key head,
// row tile), its rows the queries of the request that share the key head (token-major:
// row = t * group + g), and its length is counted in tiles of kTile tokens.  All tiles
// of all items in order are one line that is cut into equal parts, one for each CTA,
// so long and short requests together, one long request alone and a full batch all
// load every SM alike; where items are few, an item takes whole CTAs instead.  A CTA
// whose part holds an item whole writes its output; an item cut by a boundary leaves
// these of each part in the workspace, and the part that arrives last (a counter;
// nobody waits) joins them in CTA order.
//
// Two kernels: bf16 queries with heads of up to 128 columns take the tensor cores; fp32
// queries, wider heads and a cache that no tensor map can describe take fp32 arithmetic
// (the verify batch of 64 requests below: 5420 us there, 128 us on the tensor cores).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "kv_common.cuh"
#include "tcgen05.cuh"

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
    bool q_vec;        // rows of q are 16-byte aligned
    uint64_t *tickets; // [kMaxCtas], zero between calls
    int *failed;       // not zero: a call on this workspace has failed
    float *partial;    // [2 * kMaxCtas][rows * (D + 3)]
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
           r.len <= min((int64_t)p.ld_table * p.c.page_size, (int64_t)0x7fffffff - 2 * kTile);
    if (!r.ok) r.n = r.len = 0;
    const int first = r.len - r.n;  // position of the first query
    r.low = p.window > 0 ? max(0, first - p.window + 1) : 0;
    r.sinks = min(p.sinks, r.low);
    r.w0 = r.low / kTile;
    r.s1 = min((r.sinks + kTile - 1) / kTile, r.w0);
    r.nt = max(1, r.s1 + (r.len + kTile - 1) / kTile - r.w0);
    r.rt = (int)(((uint32_t)r.n * p.group + rows - 1) / rows);  // the host keeps n * group below 2^31
    return r;
}

// Starting and finishing an item costs a CTA about as much as kItemCost tiles, so on the
// line an item is that much longer, ahead of its tiles -- where there are enough tiles
// to go round: with fewer than kTilesEach a CTA, spreading the tiles matters more.  With
// no such cost the verify batch measured below takes 149 us instead of 128.
constexpr int kItemCost = 3, kTilesEach = 4;
__device__ __forceinline__ int64_t request_items(const AttnParams &p, const Request &r) {
    return (int64_t)p.c.num_heads * r.rt;
}

// a / b for a >= 0, b > 0: most quotients here fit 32 bits, where a division is short.
__device__ __noinline__ int64_t quotient64(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return quotient64(a, b);
}

// A CTA's place on the line: [u, end), starting `off` units into request b.
// Only as many CTAs as there are units take part, so that no share among them is empty
// and the parts of a cut item are those of consecutive CTAs.
struct Share {
    int64_t total, u, end, off;
    int b, ctas, cost;  // cost: units of an item ahead of its tiles
    int each;           // > 0: every CTA has one part, of `each` tiles at most
};

__device__ __forceinline__ int64_t share_start(int64_t total, int cta, int ctas) {
    return quotient(total * cta, ctas);
}
// The CTA whose share holds unit u.
__device__ __forceinline__ int cta_of(int64_t total, int64_t u, int ctas) {
    return (int)quotient((u + 1) * ctas - 1, total);
}

// Few items: an item takes as many CTAs as it has runs of `each` tiles, and every CTA one
// part, where that keeps `each` within kEachTries - 1 tiles of a fair share of all tiles;
// cut by the line, most CTAs would have an end of one item and the start of the next,
// and pay for both.  256 items of 11 tiles: 32 us so, 39 on the line; 128 of 5: 16 us
// and 20; 192 of 20, on the line either way, 38 us.
constexpr int kEachTries = 4;

struct ShareScratch {  // shared memory of find_share
    int64_t tiles[20], items[20];
    int counts[20][kEachTries];
    Share share;
};

// Every thread of the CTA calls it (it synchronises); NT threads.
template <int NT>
__device__ __noinline__ Share find_share(const AttnParams &p, int rows, ShareScratch &scratch) {
    static_assert(NT / 32 <= 20, "sums a warp");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + NT - 1) / NT, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    int64_t tiles = 0, items = 0;
    for (int b = b0; b < b1; ++b) {
        const Request r = load_request(p, b, rows);
        const int64_t n = request_items(p, r);
        items += n;
        tiles += n * r.nt;
    }
    int64_t ti = tiles, it = items;  // sums of the threads up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, ti, o), z = __shfl_up_sync(0xffffffffu, it, o);
        if (lane >= o) {
            ti += y;
            it += z;
        }
    }
    if (lane == 31) {
        scratch.tiles[warp] = ti;
        scratch.items[warp] = it;
    }
    if (tid == 0) scratch.share.b = p.B;
    __syncthreads();
    int64_t all_tiles = 0, all_items = 0;
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) {
            ti += scratch.tiles[w];
            it += scratch.items[w];
        }
        all_tiles += scratch.tiles[w];
        all_items += scratch.items[w];
    }
    if (all_items <= gridDim.x) {
        const int fair = (int)min((all_tiles + gridDim.x - 1) / gridDim.x, (int64_t)1 << 30);
        int mine[kEachTries] = {}, upto[kEachTries];  // CTAs that this thread's requests take; and all up to it
        for (int b = b0; b < b1; ++b) {
            const Request r = load_request(p, b, rows);
            const int n = (int)request_items(p, r);
            if (n > 0)
#pragma unroll
                for (int j = 0; j < kEachTries; ++j) mine[j] += n * min(1 << 16, (r.nt - 1) / (fair + j) + 1);
        }
#pragma unroll
        for (int j = 0; j < kEachTries; ++j) {
            upto[j] = mine[j];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto[j], o);
                if (lane >= o) upto[j] += y;
            }
            if (lane == 31) scratch.counts[warp][j] = upto[j];
        }
        __syncthreads();
        for (int j = 0; j < kEachTries; ++j) {
            int all = 0, before = upto[j] - mine[j];
            for (int w = 0; w < NT / 32; ++w) {
                if (w < warp) before += scratch.counts[w][j];
                all += scratch.counts[w][j];
            }
            if (all > (int)gridDim.x) continue;
            const int cta = blockIdx.x;
            if (cta >= before && cta < before + mine[j]) {
                int b = b0, off = cta - before;
                for (;; ++b) {
                    const Request r = load_request(p, b, rows);
                    const int t = (int)request_items(p, r) * ((r.nt - 1) / (fair + j) + 1);
                    if (off < t) break;
                    off -= t;
                }
                scratch.share.b = b;
                scratch.share.off = off;
            }
            __syncthreads();
            Share s = scratch.share;
            s.u = 0;
            s.end = cta < all;
            s.each = fair + j;
            return s;
        }
    }
    const int cost = all_tiles >= (int64_t)kTilesEach * gridDim.x ? kItemCost : 0;
    const int64_t total = all_tiles + cost * all_items, sum = tiles + cost * items, before = ti + cost * it - sum;
    const int ctas = (int)min((int64_t)gridDim.x, total), cta = blockIdx.x;
    const int64_t u = cta < ctas ? share_start(total, cta, ctas) : 0;
    const int64_t end = cta < ctas ? share_start(total, cta + 1, ctas) : 0;
    if (u < end && u >= before && u < before + sum) {  // one thread: its requests hold unit u
        int b = b0;
        int64_t off = u - before;
        for (; b + 1 < b1; ++b) {
            const Request r = load_request(p, b, rows);
            const int64_t t = request_items(p, r) * (r.nt + cost);
            if (off < t) break;
            off -= t;
        }
        scratch.share.b = b;
        scratch.share.off = off;
    }
    __syncthreads();
    Share s = scratch.share;
    s.total = total;
    s.u = u;
    s.end = end;
    s.ctas = ctas;
    s.cost = cost;
    s.each = 0;
    return s;
}

// One part of one item: tiles [t0, t1) of the nt of (b, h, row tile rt).
struct Part {
    Request r;
    int b, h, rt, t0, t1;
    int nrows, pos0, pos1;  // rows of the row tile, positions of its first and last
    bool whole;
    int c0, c1;  // the CTAs that hold the item's first and last tile
    __device__ __forceinline__ int tile(int i) const { return i < r.s1 ? i : r.w0 + (i - r.s1); }
};

// The share's next part; b = -1 where there is none.
__device__ __noinline__ Part next_part(const AttnParams &p, Share &s, int rows) {
    Part x;
    x.b = -1;
    if (s.each > 0) {
        if (s.u >= s.end) return x;
        s.u = s.end;
        x.r = load_request(p, s.b, rows);
        const int k = (x.r.nt - 1) / s.each + 1, i = (int)s.off / k, j = (int)s.off - i * k;
        const int q = x.r.nt / k, more = x.r.nt - q * k;
        x.b = s.b;
        x.t0 = j * q + min(j, more);
        x.t1 = x.t0 + q + (j < more ? 1 : 0);
        x.h = i / x.r.rt;
        x.rt = i - x.h * x.r.rt;
        x.whole = k == 1;
        x.c0 = blockIdx.x - j;
        x.c1 = x.c0 + k - 1;
    } else {
        int64_t item = 0;
        for (;;) {
            if (s.u >= s.end) return x;
            x.r = load_request(p, s.b, rows);
            if (s.off >= request_items(p, x.r) * (x.r.nt + s.cost)) {
                s.off = 0;  // a share's next request is entered at its first unit
                ++s.b;
                continue;
            }
            const int units = x.r.nt + s.cost;
            const int64_t i = quotient(s.off, units);
            const int at = (int)(s.off - i * units), to = (int)min((int64_t)units, at + s.end - s.u);
            item = s.u - at;
            s.u += to - at;
            s.off += to - at;
            if (to <= s.cost) continue;  // none of its tiles are here
            x.b = s.b;
            x.t0 = max(0, at - s.cost);
            x.t1 = to - s.cost;
            x.h = (int)quotient(i, x.r.rt);
            x.rt = (int)(i - (int64_t)x.h * x.r.rt);
            break;
        }
        x.whole = x.t0 == 0 && x.t1 == x.r.nt;
        x.c0 = x.c1 = blockIdx.x;
        if (!x.whole) {
            x.c0 = cta_of(s.total, item + s.cost, s.ctas);
            x.c1 = cta_of(s.total, item + s.cost + x.r.nt - 1, s.ctas);
        }
    }
    const int row0 = x.rt * rows;
    x.nrows = min(rows, x.r.n * p.group - row0);
    x.pos0 = x.r.len - x.r.n + row0 / p.group;
    x.pos1 = x.r.len - x.r.n + (row0 + x.nrows - 1) / p.group;
    // tiles that start after the row tile's last position hold nothing for it; a part
    // keeps at least one tile, so that it has a result to join
    const int seen = x.pos1 < 0 ? 0 : (x.pos1 / kTile < x.r.w0 ? min(x.r.s1, x.pos1 / kTile + 1)
                                                               : x.r.s1 + x.pos1 / kTile - x.r.w0 + 1);
    x.t1 = max(x.t0 + 1, min(x.t1, seen));
    return x;
}

// Lengths and pages of the requests, told by one warp for every gridDim.x-th request.
__device__ __noinline__ void write_statuses(const AttnParams &p, int lane) {
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const Request r = load_request(p, b, 1);
        bool bad = false;
        if (r.n > 0) {
            const int bs = p.c.page_size, np = (r.len + bs - 1) / bs, ns = (r.sinks + bs - 1) / bs;
            const int32_t *t = p.table + (int64_t)b * p.ld_table;
            for (int i = lane; i < ns; i += 32) bad |= t[i] < 0 || t[i] >= p.c.num_pages;
#pragma unroll 8
            for (int i = r.low / bs + lane; i < np; i += 32) bad |= t[i] < 0 || t[i] >= p.c.num_pages;
        }
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0)
            p.status[b] = !r.ok ? SPEC_STATUS_BAD_LENGTH : (bad ? SPEC_STATUS_BAD_PAGE : SPEC_STATUS_OK);
    }
}

// A CTA that cannot answer for its parts fails the whole call: every request, whatever
// other CTAs wrote or have yet to write.  The word stays for the calls after this one,
// which may find what this one left behind.  NT threads call it.
template <int NT>
__device__ __noinline__ void fail_call(const AttnParams &p) {
    if (threadIdx.x == 0) *(volatile int *)p.failed = 1;
    __threadfence();
    __syncthreads();
    for (int b = threadIdx.x; b < p.B; b += NT) p.status[b] = SPEC_STATUS_INTERNAL;
}

// The thread that wrote a CTA's statuses looks at the word after them.  Either it sees
// the word, or its statuses come before those of the CTA that sets it.
__device__ __noinline__ void recheck_statuses(const AttnParams &p) {
    __threadfence();
    if (*(volatile int *)p.failed == 0) return;
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) p.status[b] = SPEC_STATUS_INTERNAL;
}

// ------------------------------------------------------------------ joining parts
template <int NT>
__device__ __forceinline__ void named_sync(int bar) {
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(NT) : "memory");
}

// A barrier of NT threads that tells whether any of them has x.
template <int NT>
__device__ __forceinline__ bool named_any(int bar, bool x) {
    uint32_t any;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n barrier.cta.red.or.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
                 : "=r"(any)
                 : "r"(bar), "n"(NT), "r"((uint32_t)x)
                 : "memory");
    return any != 0;
}

// A part's slot: the first part of an item is its CTA's last part, every other part
// its CTA's first, so two slots a CTA are enough.  It holds the R rows' sums o [R][D],
// the references m of their weights' sums, those sums l, and the references of o.
__device__ __forceinline__ float *slot_of(const AttnParams &p, int cta, bool first, int rows) {
    return p.partial + (int64_t)(2 * cta + (first ? 1 : 0)) * rows * (p.c.head_dim + 3);
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
// What o, with reference mo, is multiplied by to be divided by l with reference m.
__device__ __forceinline__ float output_factor(float mo, float m, float l) {
    return l == 0.f ? 0.f : exp2f(mo - m) / l;
}

// 2^(a - m), 0 where the part a comes from saw nothing (a = -inf, whatever m is).
__device__ __forceinline__ float weight_of(float a, float m) { return a == kNegInf ? 0.f : exp2f(a - m); }

// Counts this CTA's part of a cut item in; true (in every thread) for the part that
// arrives last, which may then read the other parts.  NT threads call it, `bar` a
// named barrier of theirs: it orders their stores before thread 0's release, and that
// thread's acquire before their loads.
// A counter holds, besides how many parts have arrived (low half), the sum of their
// numbers from 1: one that does not add up has not started at zero, and fails the call.
template <int NT>
__device__ __forceinline__ bool arrive_last(const AttnParams &p, int first_cta, int parts, int *s_flag, int bar, bool &failed) {
    named_sync<NT>(bar);
    if (threadIdx.x == 0) {
        const uint64_t mine = 1 + ((uint64_t)(blockIdx.x - first_cta + 1) << 32);
        const uint64_t all = parts + ((uint64_t)((uint32_t)parts * (parts + 1) / 2) << 32);
        uint64_t before;
        asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], %2;"
                     : "=l"(before)
                     : "l"(p.tickets + first_cta), "l"(mine)
                     : "memory");
        const bool last = before + mine == all, sound = last || (uint32_t)before < (uint32_t)parts - 1;
        *s_flag = last ? 1 : (sound ? 0 : 2);
        if (last) p.tickets[first_cta] = 0;  // for the next call
    }
    named_sync<NT>(bar);
    failed |= *s_flag == 2;
    return *s_flag == 1;
}

// Joins the parts of an item in CTA order and writes its rows: a warp takes two rows at
// a time, four columns a lane, with the statistics and sums of four parts in flight.
// ND: 128-column blocks of the head.
template <typename T, int NT, int R, int ND>
__device__ __noinline__ void join_parts(const AttnParams &p, const Part &x) {
    constexpr int kWarps = NT / 32, P = 4;
    const int D = p.c.head_dim, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nrows = x.nrows, parts = x.c1 - x.c0 + 1;
    const int64_t stride = 2 * (int64_t)R * (D + 3);  // from a CTA's slot to the next one's
    const float *slot0 = slot_of(p, x.c0, true, R), *slots = slot_of(p, x.c0, false, R);  // part 0; part c at c * stride
    for (int r0 = warp; r0 < nrows; r0 += 2 * kWarps) {
        float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f}, mo[2] = {kNegInf, kNegInf};
        float4 o[2][ND];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int n = 0; n < ND; ++n) o[k][n] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c0 = 0; c0 < parts; c0 += P) {
            float mc[2][P], lc[2][P], moc[2][P];
            float4 v[2][P][ND];
#pragma unroll
            for (int c = 0; c < P; ++c) {
                const float *s = c0 + c == 0 ? slot0 : slots + (c0 + c) * stride;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int r = r0 + k * kWarps;
                    const bool on = c0 + c < parts && r < nrows;
                    mc[k][c] = on ? __ldcg(s + R * D + r) : kNegInf;
                    lc[k][c] = on ? __ldcg(s + R * D + R + r) : 0.f;
                    moc[k][c] = on ? __ldcg(s + R * D + 2 * R + r) : kNegInf;
#pragma unroll
                    for (int n = 0; n < ND; ++n) {
                        const int d = 128 * n + 4 * lane;
                        v[k][c][n] = on && d < D ? __ldcg((const float4 *)(s + r * D + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float top = m[k], top_o = mo[k];
#pragma unroll
                for (int c = 0; c < P; ++c) {
                    top = fmaxf(top, mc[k][c]);
                    top_o = fmaxf(top_o, moc[k][c]);
                }
                l[k] *= weight_of(m[k], top);
                m[k] = top;
                const float keep = weight_of(mo[k], top_o);
                mo[k] = top_o;
#pragma unroll
                for (int n = 0; n < ND; ++n) {
                    o[k][n].x *= keep;
                    o[k][n].y *= keep;
                    o[k][n].z *= keep;
                    o[k][n].w *= keep;
                }
#pragma unroll
                for (int c = 0; c < P; ++c) {
                    l[k] = fmaf(lc[k][c], weight_of(mc[k][c], top), l[k]);
                    const float w = weight_of(moc[k][c], top_o);
#pragma unroll
                    for (int n = 0; n < ND; ++n) {
                        o[k][n].x = fmaf(v[k][c][n].x, w, o[k][n].x);
                        o[k][n].y = fmaf(v[k][c][n].y, w, o[k][n].y);
                        o[k][n].z = fmaf(v[k][c][n].z, w, o[k][n].z);
                        o[k][n].w = fmaf(v[k][c][n].w, w, o[k][n].w);
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = r0 + k * kWarps;
            if (r >= nrows) break;
            const float inv = output_factor(mo[k], m[k], l[k]);
            const int row = x.rt * R + r, t = row / p.group, g = row - t * p.group;
            const int64_t at = ((int64_t)(x.r.row0 + t) * p.Hq + x.h * p.group + g) * D;
            if (p.lse && lane == 0) store_lse(p, x, row, m[k], l[k]);
#pragma unroll
            for (int n = 0; n < ND; ++n) {
                const int d = 128 * n + 4 * lane;
                if (d >= D) break;
                const float4 f = make_float4(o[k][n].x * inv, o[k][n].y * inv, o[k][n].z * inv, o[k][n].w * inv);
                if constexpr (sizeof(T) == 2) {
                    *(uint2 *)((uint16_t *)p.out + at + d) = make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
                } else {
                    *(float4 *)((float *)p.out + at + d) = f;
                }
            }
        }
    }
}

// ------------------------------------------------------------------ fp32 arithmetic kernel
// Four warps, each 32 tokens of a tile: a lane holds one token's scores of kSimtRows
// rows (its key row read 16 codes at a time, the queries broadcast from shared
// memory), then the warp walks its tokens with the lanes over the head's columns.
// Every warp keeps its own (m, l, o); they join in shared memory at the part's end.
// Bound by instructions: two fp32 products of rows x tokens x columns and eight warp
// reductions a token block.  9 requests of 1 to 5 fp32 queries, 10 heads on 2 of 80
// columns, 40 to 1500 tokens: 30 us.
constexpr int kSimtRows = 8, kSimtThreads = 128;

template <typename T, int ND>
__global__ void __launch_bounds__(kSimtThreads) attention_simt_kernel(AttnParams p) {
    constexpr int R = kSimtRows;
    __shared__ __align__(16) float s_q[R][128 * ND];
    __shared__ float s_p[4][32][R];
    __shared__ float s_m[4][R], s_l[4][R], s_w[2 * R];
    __shared__ ShareScratch s_scratch;
    __shared__ __align__(16) float s_o[R][128 * ND];
    __shared__ int s_flag;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = p.c.head_dim, bs = p.c.page_size;
    if (warp == 0) write_statuses(p, lane);
    Share share = find_share<kSimtThreads>(p, R, s_scratch);
    bool failed = false;
    for (;;) {
        const Part x = next_part(p, share, R);
        if (x.b < 0) break;
        const int nrows = x.nrows, first = x.r.len - x.r.n;
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
            // rows that see every token some row sees
            const uint32_t all = __reduce_and_sync(0xffffffffu, sees ? sees : 0xffffffffu);
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
        if (x.whole) {
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
                slot[R * D + 2 * R + tid] = s_w[tid];
            }
            if (arrive_last<kSimtThreads>(p, x.c0, x.c1 - x.c0 + 1, &s_flag, 1, failed))
                join_parts<T, kSimtThreads, R, ND>(p, x);
        }
    }
    if (failed) fail_call<kSimtThreads>(p);  // the same in every thread
    else if (tid == 0) recheck_statuses(p);
}

// ------------------------------------------------------------------ tensor-core kernel
// bf16 queries, head sizes up to 128.  Both products run on the fifth-generation
// tensor cores straight from the e4m3 codes that the tiled copies bring to shared
// memory; nothing is converted on the way.  With the tokens as M:
//   S^T [128 tokens, R rows] = K [128, D] Q^T      (K's rows run along K)
//   O^T [128 >= D, R rows]  = V^T [D, 128] P^T     (V transposed by the operand's layout)
// so the rows of a tile, few in a verify step, are the products' narrow side and cost
// what they are, and a thread of the softmax owns one token in S^T and one column of
// the head in O^T: 16 rows of each.
//  - e4m3 keeps 4 significant bits, so Q and P are each the sum of two e4m3 terms.  The
//    terms lie side by side along N, so that a product is one instruction a step of 32
//    with 2 R columns (32 columns take 55 cycles, 64 take 69, 128 take 97), and their
//    results are added as they leave tensor memory.  A row of Q is scaled by a power of
//    two to a largest magnitude of 128 .. 256: a bf16 entry (8 bits) is then exact in two
//    terms down to 2^-9 of the row's largest, and off by 2^-17 of it at most below.
//  - What P V^T adds for token j is 2^x_j vs_j times its codes, vs_j the scale of its
//    value's page.  Two e4m3 terms of a number z of 0 .. 256 are off by 2^-8 of it, or by
//    2^-10 where that is more, so z has to be near 256 where it matters: z_j =
//    2^(8 + y_j - r) with y_j = x_j + log2(vs_j), r the largest y_j of the tokens of the
//    tile that the row sees.  Neither pages that a row does not see nor improbable ones
//    with large values then cost the others their bits, and a tail of small
//    probabilities next to one large one in another tile keeps its own.
//  - The weights' sum l needs 2^x_j = z_j 2^(r - 8) / vs_j.  That is one exponential for
//    both, while the tile's value scales lie within 2^kNearLog2 of each other; where they
//    do not, z_j may vanish while its weight does not, and l gets its own reference, the
//    tile's largest x_j, and its own exponentials.  (log2(vs_j) is counted from the
//    tile's largest, lt, so that it is 0 where all are equal.)
//  - So a row has two running references, m for l and mo for O, both in fp32; the
//    output is O 2^(mo - m) / l.
//  - A running reference moves only when a tile's is more than 2^64 above it, so sums
//    are rescaled at a part's first tile and hardly ever after.
//  - exp2 is the hardware's approximation, its error far below the rounding of P.
// Roles: R / 16 groups of 128 threads for the softmax and the sums, one warp that issues
// the products, one or two that copy.  The first copying warp also finds the CTA's parts
// and tells the others of each while it copies the one before (kParts places).  S^T and
// O^T are double-buffered: S^T of the next tile is multiplied while the softmax of this
// one runs, O^T of this one while the sums take the last.
//
// What bounds it: the chain of one tile through its softmax warps, from tensor memory
// through maxima, exponentials and two roundings to P and back, about 3200 cycles, of
// which two (two CTAs) are under way on an SM; the issue slots are half full, the
// tensor cores at an eighth, DRAM at two thirds.  R = 16 and 32 have two CTAs an SM
// (with one, the first two batches below take 158 and 112 us instead of 128 and 91),
// R = 64 has the shared memory and registers for one.  R is the smallest that holds a
// request's rows: 38 requests of 8192 tokens and 8 key heads of 128 take, with 8 rows,
// 103 us in R = 16, 109 in 32 and 175 in 64; with 32 rows 121 us in 32 and 189 in 64; with
// 64 rows 217 us in 64, 232 in 32 and 374 in 16.  The bytes alone take 94 us.
// Measured (a launch among others in a graph, codes read): 64 requests, 8 queries, 32
// query and 8 key heads of 128, 500 to 8000 tokens, pages of 64: 128 us, 4.4 TB/s.  Two
// requests of 120000 and 131071 tokens, one query, 64 query heads: 91 us, 5.7 TB/s.  256
// requests of 1 to 8 queries, 4 key heads of 64, 60 to 3000 tokens, pages of 16: 109 us,
// 1.9 TB/s.  One request of one query over 1004 tokens: 13.5 us.
// With probabilities rounded next to the largest value scale of the tile these three took
// 119, 89 and 107 us, and 64 rows 194, but a page far above the others cost those their
// probabilities.
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kSlotBytes = kTile * 128;  // a tile of keys or values
constexpr int kInfo = 8;                 // tiles whose scales are held at a time
constexpr float kRefStep = 64.f;         // how far (log2) a tile may pass the running reference
constexpr float kNearLog2 = 16.f;        // spread of a tile's value scales that one exponential serves

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
    unsigned long long d;
    asm("mul.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
    return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float redux_max(float x) {  // over the warp; a NaN counts as absent
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
    return m;
}
__device__ __forceinline__ uint32_t float2_to_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t half2_sub(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t half4_to_e4m3x4(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("{\n .reg .b16 t, u;\n cvt.rn.satfinite.e4m3x2.f16x2 t, %1;\n cvt.rn.satfinite.e4m3x2.f16x2 u, %2;\n"
        " mov.b32 %0, {t, u};\n}"
        : "=r"(r)
        : "r"(a), "r"(b));
    return r;
}
// Four floats as two words of e4m3 codes: the values, and what is left of them.
__device__ __forceinline__ void split_e4m3x4(float2 x, float2 y, uint32_t &first, uint32_t &rest) {
    const uint32_t a = float2_to_half2(x.x, x.y), b = float2_to_half2(y.x, y.y);
    uint32_t c, d;
    first = half4_to_e4m3x4(a, b);
    asm("{\n .reg .b16 t, u;\n mov.b32 {t, u}, %2;\n cvt.rn.f16x2.e4m3x2 %0, t;\n cvt.rn.f16x2.e4m3x2 %1, u;\n}"
        : "=r"(c), "=r"(d)
        : "r"(first));
    rest = half4_to_e4m3x4(half2_sub(a, c), half2_sub(b, d));  // exact before the rounding
}
// Waits for the phase of the given parity; false after kWaitNs.  These waits are a few
// hundred cycles long and on the path of every tile, so the thread polls: one that
// sleeps in the barrier is woken late.
__device__ __forceinline__ bool try_barrier(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done != 0;
}
__device__ __noinline__ bool poll_barrier(uint32_t bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t n = 1;; ++n) {
        if (try_barrier(bar, parity)) return true;
        if ((n & 255) == 0) {
            const uint64_t now = global_ns();
            if (t0 == 0) t0 = now;
            else if (now - t0 > kWaitNs) return false;
        }
    }
}

template <int R>
struct TcShape {
    static constexpr int kRowsG = 16;                     // rows of a softmax group
    static constexpr int kGroups = R / kRowsG;            // groups of 128 threads
    static constexpr int kSoft = 128 * kGroups;           // softmax threads
    static constexpr int kPerSM = R < 64 ? 2 : 1;         // CTAs an SM
    static constexpr int kSlots = R < 64 ? 5 : 10;
    static constexpr uint32_t kCols = 8 * R;              // S^T and O^T, two terms and two buffers each
};

// Softmax threads, the issuer of the products, W warps that copy.
template <int R, int W>
constexpr int kTcThreads = TcShape<R>::kSoft + 32 * (1 + W);

constexpr int kParts = 4;  // places for parts that have been told and are not done with
constexpr int kAllBar = 8, kLookBar = 9;  // named barriers of all softmax threads; group g's is 1 + g

template <int R>
struct TcShared {
    using C = TcShape<R>;
    uint8_t ring[C::kSlots][kSlotBytes];
    uint8_t q[2][R * 128];             // two terms, rows of 128 bytes, swizzled
    uint16_t q_raw[R][128];            // the next part's, as they are stored
    uint8_t p[2][R / 16][kTile * 16];  // two terms, blocks of 16 rows, a token's 16 bytes together
    uint64_t full[C::kSlots], empty[C::kSlots], s_full[2], p_full, o_full, q_full;
    uint64_t part_full[kParts], part_empty[kParts];
    Part part[kParts];                      // b < 0: no more
    // a tile's pages: the key's scale, log2 of the value's over the tile's largest and the
    // inverse of that (0 if the tile is far), whether it is far (1 or 0); log2 of the largest
    float4 page_info[kInfo][8];
    float lt[kInfo];
    int pages[2][8];                              // and its pages, for the copies of keys and of values
    // every softmax warp's own copy, by the tile's parity: 8 less the rows' references,
    // weights of the row sums and of O^T
    alignas(16) float nref[4 * C::kGroups][2][C::kRowsG];
    float beta[4 * C::kGroups][2][C::kRowsG], w[4 * C::kGroups][2][C::kRowsG];
    float red[2][4][R], red_far[4][R];
    float c[R];               // score factor of a row: scale * log2(e) / its power of two
    float m[R], l[R], mo[R];  // at a part's end
    // A row's first output element, by the part's number mod 3: written while the part
    // before runs, read as the part ends, by each warp in its own time.  Every warp passes
    // a barrier in the next part, so by the part after that, which may use the same place,
    // all have read.  (By the next part alone, one of a single tile, they may not have.)
    int64_t out_at[3][R];
    ShareScratch scratch;
    uint32_t tmem;
    int flag;
};

// The two terms' products of a tile, as loaded from tensor memory, into one.
template <int N>
__device__ __forceinline__ void add_terms(uint32_t (&a)[N], const uint32_t (&b)[N]) {
#pragma unroll
    for (int r = 0; r < N; r += 2) {
        const float2 f = fadd2(make_float2(__uint_as_float(a[r]), __uint_as_float(a[r + 1])),
                               make_float2(__uint_as_float(b[r]), __uint_as_float(b[r + 1])));
        a[r] = __float_as_uint(f.x);
        a[r + 1] = __float_as_uint(f.y);
    }
}

// Sum over the warp of each of N <= 32 values a lane: lane i gets value i (mod N).
template <int N>
__device__ __forceinline__ float warp_sum_scatter(float (&v)[N], int lane) {
#pragma unroll
    for (int s = N / 2; s > 0; s >>= 1) {
#pragma unroll
        for (int i = 0; i < s; ++i) {
            const bool up = lane & s;
            const float keep = up ? v[i + s] : v[i], send = up ? v[i] : v[i + s];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, s);
        }
    }
    float x = v[0];
#pragma unroll
    for (int s = N; s < 32; s <<= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    return x;
}

// A far tile's own work, out of the way of the others' registers: the warp's largest x
// = y - log2(value's scale) of each row, and each row's weight of this lane's token.
template <int NR>
__device__ __noinline__ void far_maxima(const float (&y)[NR], float lv, float *red, int lane) {
#pragma unroll 1
    for (int r = 0; r < NR; ++r) {
        const float f = redux_max(y[r] == kNegInf ? kNegInf : y[r] - lv);
        if (lane == 0) red[r] = f;
    }
    __syncwarp();
}
template <int NR>
__device__ __noinline__ void far_weights(float (&y)[NR], float lv, float x_ref, float x_beta) {
#pragma unroll 1
    for (int r = 0; r < NR; ++r) {
        const float x = y[r] == kNegInf ? kNegInf : y[r] - lv;
        y[r] = ex2_approx(x - __shfl_sync(0xffffffffu, x_ref, r)) * __shfl_sync(0xffffffffu, x_beta, r);
    }
}

// A part's queries: a thread takes kCols columns of one row.  start_queries, a tile
// ahead, starts their copy to shared memory, where only the same thread reads them;
// store_queries makes two e4m3 terms of each entry for the products.
template <int R>
struct QueryShape {
    static constexpr int kCols = R * 128 / TcShape<R>::kSoft, kPerRow = 128 / kCols;
};

template <int R>
__device__ __noinline__ void start_queries(const AttnParams &p, const Part &x, TcShared<R> &sm, int tid, int at) {
    constexpr int kCols = QueryShape<R>::kCols;
    const int row = tid / QueryShape<R>::kPerRow, c0 = (tid % QueryShape<R>::kPerRow) * kCols, D = p.c.head_dim;
    if (row >= x.nrows) return;
    const uint32_t grow = x.rt * R + row, t = grow / (uint32_t)p.group, head = x.h * p.group + (grow - t * p.group);
    if (c0 == 0) sm.out_at[at][row] = ((int64_t)(x.r.row0 + (int)t) * p.Hq + head) * D;
    const char *src = (const char *)p.q + ((int64_t)(x.r.row0 + (int)t) * p.ld_q + (int64_t)head * D + c0) * 2;
#pragma unroll
    for (int c = 0; c < kCols; c += 8) {
        if (c0 + c >= D) break;
        uint16_t *dst = &sm.q_raw[row][c0 + c];
        if (p.q_vec) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src + c * 2) : "memory");
        } else {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) dst[i] = __ldg((const unsigned short *)(src + c * 2) + i);
        }
    }
}

template <int R>
__device__ __noinline__ void store_queries(float scale_log2, int nrows, int D, TcShared<R> &sm, int tid) {
    constexpr int kCols = QueryShape<R>::kCols, kPerRow = QueryShape<R>::kPerRow;
    const int row = tid / kPerRow, c0 = (tid % kPerRow) * kCols;
    uint32_t raw[kCols / 2];
    asm volatile("cp.async.wait_all;" ::: "memory");
    uint32_t top = 0;  // magnitudes compare as integers; a NaN or an infinity has 0x7f80 or more
#pragma unroll
    for (int c = 0; c < kCols; c += 8) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (row < nrows && c0 + c < D) u = *(const uint4 *)&sm.q_raw[row][c0 + c];
        raw[c / 2] = u.x;
        raw[c / 2 + 1] = u.y;
        raw[c / 2 + 2] = u.z;
        raw[c / 2 + 3] = u.w;
    }
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) top = __vmaxu2(top, raw[i] & 0x7fff7fffu);
#pragma unroll
    for (int s = 1; s < kPerRow; s <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, s));
    top = max(top & 0xffffu, top >> 16);
    // the row's largest magnitude's exponent becomes 7; a row with a NaN or an infinity is NaN
    const bool bad = top >= 0x7f80u;
    const int e = max((int)(top >> 7) - 127, -110);
    const float up = __uint_as_float((uint32_t)(bad ? 127 : 134 - e) << 23);
    const float down = bad ? 1.f : __uint_as_float((uint32_t)(120 + e) << 23);
#pragma unroll
    for (int c = 0; c < kCols; c += 8) {
        uint32_t a[2], b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w0 = raw[c / 2 + 2 * i], w1 = raw[c / 2 + 2 * i + 1];
            split_e4m3x4(make_float2(bf16_lo(w0) * up, bf16_hi(w0) * up), make_float2(bf16_lo(w1) * up, bf16_hi(w1) * up), a[i], b[i]);
            if (bad) a[i] = 0x7f7f7f7fu;
        }
        const int col = c0 + c, at = row * 128 + (((col >> 4) ^ (row & 7)) << 4) + (col & 8);
        *(uint2 *)(sm.q[0] + at) = make_uint2(a[0], a[1]);
        *(uint2 *)(sm.q[1] + at) = make_uint2(b[0], b[1]);
    }
    if (c0 == 0) sm.c[row] = fmaxf(scale_log2 * down, 1.1754944e-38f);  // -inf times it stays -inf
    fence_async_shared();
    __syncwarp();
    if ((tid & 31) == 0) mbar_arrive(&sm.q_full);
}

template <int R, int W>
__global__ void __launch_bounds__(kTcThreads<R, W>, TcShape<R>::kPerSM)
    attention_tc_kernel(AttnParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using C = TcShape<R>;
    constexpr int NR = C::kRowsG, NS = C::kSlots;
    extern __shared__ __align__(1024) uint8_t raw[];
    TcShared<R> &sm = *reinterpret_cast<TcShared<R> *>(raw);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the warp's: roles branch on it
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&sm.full[i], 2);  // the copies, and the copier's word that the tile's scales are there
            mbar_init(&sm.empty[i], 1);
        }
        mbar_init(&sm.s_full[0], 2);  // the product, and the issuer's word for the tile's scales
        mbar_init(&sm.s_full[1], 2);
        mbar_init(&sm.p_full, C::kSoft / 32);
        mbar_init(&sm.o_full, 1);
        mbar_init(&sm.q_full, C::kSoft / 32);
        for (int i = 0; i < kParts; ++i) {
            mbar_init(&sm.part_full[i], 1);
            mbar_init(&sm.part_empty[i], W + C::kSoft / 32);  // the readers
        }
        mbar_init_fence();
    }
    if (warp == C::kSoft / 32 + 1) tmem_alloc(&sm.tmem, C::kCols);
    tc_fence_before();
    Share share = find_share<kTcThreads<R, W>>(p, R, sm.scratch);  // it synchronises the CTA
    tc_fence_after();
    const uint32_t tm = sm.tmem, tS = tm, tO = tm + 4 * R;  // a buffer: R columns of each term
    bool dead = false;    // a wait ran out: wait no more, finish, report
    bool failed = false;  // something else to report
    auto wait = [&](uint64_t *bar, int parity) {
        if (!try_barrier(smem_addr(bar), parity) && !dead && !poll_barrier(smem_addr(bar), parity)) dead = true;
        __syncwarp();
    };
    auto gone = [&] {
        dead = __any_sync(0xffffffffu, dead);
        return dead;
    };
    // The copying warps: a batch is the tiles whose pages fill a warp's lanes.
    const int bs = p.c.page_size, shift = 31 - __clz(kTile / bs), ppt = 1 << shift, batch = 32 >> shift;
    auto fetch_page = [&](const Part &x, int i0) {
        const int i = i0 + (lane >> shift);
        if (i >= x.t1) return -1;
        const int j = x.tile(i) * kTile + (lane & (ppt - 1)) * bs;
        if (j >= x.r.len || (j + bs <= x.r.low && j >= x.r.sinks)) return -1;
        const int page = p.table[(int64_t)x.b * p.ld_table + j / bs];
        return page < p.c.num_pages ? page : -1;
    };
    int sent = 0;  // past the last slot this warp filled
    auto copy_tile = [&](const CUtensorMap &map, int seq, int page, int h, int *pages) {
        const int slot = seq % NS, turn = seq / NS;
        if (turn > 0) wait(&sm.empty[slot], (turn - 1) & 1);
        if (gone()) return;
        sent = seq + 1;
        if (lane < ppt) pages[lane] = page >= 0 ? page : p.c.num_pages;  // past the map's end: reads as zeros
        __syncwarp();
        if (elect_one()) {
            mbar_arrive_expect_tx(&sm.full[slot], kSlotBytes);
#pragma unroll 4
            for (int i = 0; i < ppt; ++i)
                tma_load_4d(sm.ring[slot] + i * bs * 128, &map, 0, 0, h, pages[i], &sm.full[slot]);
        }
        __syncwarp();
    };
    // After a wait that ran out: none of this warp's copies may be in flight when the CTA ends.
    auto drain = [&] {
        if (gone())
            for (int i = max(0, sent - NS); i < sent; ++i)
                if (W == 1 || ((sent - i) & 1)) mbar_wait(&sm.full[i % NS], (i / NS) & 1, kWaitNs);
    };

    if (warp == C::kSoft / 32) {
        // ---------------------------------------------------------------- copies
        // Of the keys, and of the values if no second warp copies.  This warp also finds
        // the parts, and tells the others of the next one early in the last batch of each;
        // page ids and scales come a batch of 32 pages ahead.
        int g = 0, n = 0;  // tiles, parts told
        auto tell_part = [&](const Part &x) {
            const int at = n % kParts;
            if (n >= kParts) wait(&sm.part_empty[at], (n / kParts - 1) & 1);
            dead = __any_sync(0xffffffffu, dead);
            if (lane == 0) {
                sm.part[at] = x;
                mbar_arrive(&sm.part_full[at]);
            }
            ++n;
        };
        auto fetch_scale = [&](const float *s, const Part &x, int page) {
            return page >= 0 ? __ldg(s + (int64_t)page * p.c.num_heads + x.h) : 0.f;
        };
        Part x, xn = next_part(p, share, R);
        tell_part(xn);
        int i0 = 0, in = xn.t0, page = -1, page_n = -1;
        float ks = 0.f, vs = 0.f, ks_n = 0.f, vs_n = 0.f;
        float lv = 0.f, iv = 0.f, top = 0.f;
        bool far = false;
        if (xn.b >= 0) {
            page_n = fetch_page(xn, in);
            ks_n = fetch_scale(p.c.k_scale, xn, page_n);
            vs_n = fetch_scale(p.c.v_scale, xn, page_n);
        }
        while (xn.b >= 0 && !dead) {
            x = xn;
            i0 = in;
            page = page_n;
            ks = ks_n;
            vs = vs_n;
            for (int k = 0; k < batch && i0 + k < x.t1; ++k, ++g) {
                const int from = (k << shift) + (lane & (ppt - 1)), seq = 2 * g, slot = seq % NS;
                copy_tile(kmap, seq, __shfl_sync(0xffffffffu, page, from), x.h, sm.pages[0]);
                if (dead) break;
                if (k == 0) {  // the scales may still be on their way here
                    // Of this lane's page; those below the smallest normal number count as
                    // that, and a page that is not there has no weight.
                    const float lvs = page >= 0 ? log2f(fmaxf(vs, 1.1754944e-38f)) : -1e30f;
                    float low = page >= 0 ? lvs : 1e30f;
                    top = lvs;
                    for (int s = 1; s < ppt; s <<= 1) {  // over the pages of a tile
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
                        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, s));
                    }
                    far = top - low > kNearLog2;
                    lv = page >= 0 ? lvs - top : -1e30f;
                    iv = page >= 0 && !far ? exp2f(-lv) : 0.f;
                }
                const int at = g % kInfo;
                const float tks = __shfl_sync(0xffffffffu, ks, from), tlv = __shfl_sync(0xffffffffu, lv, from);
                const float tiv = __shfl_sync(0xffffffffu, iv, from), tlt = __shfl_sync(0xffffffffu, top, from);
                const float tfar = __shfl_sync(0xffffffffu, far ? 1.f : 0.f, from);
                if (lane < ppt) sm.page_info[at][lane] = make_float4(tks, tlv, tiv, tfar);
                if (lane == 0) sm.lt[at] = tlt;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.full[slot]);
                if constexpr (W == 1) {
                    copy_tile(vmap, seq + 1, __shfl_sync(0xffffffffu, page, from), x.h, sm.pages[0]);
                    if (dead) break;
                    if (lane == 0) mbar_arrive(&sm.full[(seq + 1) % NS]);
                }
                if (k == 0) {  // the next batch, of this part or of the next
                    if (i0 + batch < x.t1) {
                        in = i0 + batch;
                    } else {
                        xn = next_part(p, share, R);
                        tell_part(xn);
                        in = xn.t0;
                    }
                    page_n = xn.b >= 0 ? fetch_page(xn, in) : -1;
                }
                if (k == min(1, min(batch, x.t1 - i0) - 1)) {
                    ks_n = fetch_scale(p.c.k_scale, xn, page_n);
                    vs_n = fetch_scale(p.c.v_scale, xn, page_n);
                }
            }
        }
        drain();
    } else if (warp == C::kSoft / 32 + 2) {
        // ---------------------------------------------------------------- copies of values
        int g = 0;
        wait(&sm.part_full[0], 0);
        int page_n = !gone() && sm.part[0].b >= 0 ? fetch_page(sm.part[0], sm.part[0].t0) : -1;
        for (int n = 0; !gone() && sm.part[n % kParts].b >= 0; ++n) {
            const Part &x = sm.part[n % kParts], &next = sm.part[(n + 1) % kParts];
            const int t1 = x.t1, h = x.h;
            for (int i0 = x.t0; i0 < t1 && !dead; i0 += batch) {
                const int page = page_n;
                for (int k = 0; k < batch && i0 + k < t1; ++k, ++g) {
                    const int seq = 2 * g + 1, from = (k << shift) + (lane & (ppt - 1));
                    copy_tile(vmap, seq, __shfl_sync(0xffffffffu, page, from), h, sm.pages[1]);
                    if (dead) break;
                    if (lane == 0) mbar_arrive(&sm.full[seq % NS]);
                    if (k == 0) {  // pages of the next batch, of this part or of the next
                        if (i0 + batch < t1) {
                            page_n = fetch_page(x, i0 + batch);
                        } else {
                            wait(&sm.part_full[(n + 1) % kParts], ((n + 1) / kParts) & 1);
                            if (gone()) break;
                            page_n = next.b >= 0 ? fetch_page(next, next.t0) : -1;
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.part_empty[n % kParts]);
        }
        drain();
    } else if (warp == C::kSoft / 32 + 1) {
        // ---------------------------------------------------------------- products
        write_statuses(p, lane);  // while the first tile is on its way
        constexpr uint32_t iqk = fp8_idesc(2 * R, false, false), ipv = fp8_idesc(2 * R, true, true);
        const int ksteps = (p.c.head_dim + 31) / 32;
        const uint64_t dk = smem_desc(smem_addr(sm.ring), 16, 1024, 2), dq = smem_desc(smem_addr(sm.q), 16, 1024, 2);
        const uint64_t dv = smem_desc(smem_addr(sm.ring), 1024, 1024, 2);
        const uint64_t dp = smem_desc(smem_addr(sm.p), 128, kTile * 16, 0);
        auto scores = [&](int g) {
            const int seq = 2 * g, slot = seq % NS;
            wait(&sm.full[slot], (seq / NS) & 1);
            if (gone()) return;
            tc_fence_after();
            const uint64_t a = dk + slot * (kSlotBytes / 16);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < ksteps) mma_fp8(tS + (g & 1) * 2 * R, a + 2 * k, dq + 2 * k, iqk, k != 0);
                mma_commit(&sm.s_full[g & 1]);
                mma_commit(&sm.empty[slot]);
                mbar_arrive(&sm.s_full[g & 1]);  // passes the scales on: `full` acquired them
            }
            __syncwarp();
        };
        auto values = [&](int g) {
            const int seq = 2 * g + 1, slot = seq % NS;
            wait(&sm.full[slot], (seq / NS) & 1);
            wait(&sm.p_full, g & 1);
            if (gone()) return;
            tc_fence_after();
            const uint64_t a = dv + slot * (kSlotBytes / 16);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kTile / 32; ++k)
                    mma_fp8(tO + (g & 1) * 2 * R, a + 256 * k, dp + 32 * k, ipv, k != 0);
                mma_commit(&sm.o_full);
                mma_commit(&sm.empty[slot]);
            }
            __syncwarp();
        };
        int g = 0;
        for (int n = 0; !gone(); ++n) {
            const int at = n % kParts;
            wait(&sm.part_full[at], (n / kParts) & 1);
            if (gone() || __shfl_sync(0xffffffffu, sm.part[at].b, 0) < 0) break;
            const int tiles = __shfl_sync(0xffffffffu, sm.part[at].t1 - sm.part[at].t0, 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.part_empty[at]);
            wait(&sm.q_full, n & 1);
            scores(g);
            for (int i = 0; i < tiles; ++i, ++g) {
                if (i + 1 < tiles) scores(g + 1);
                values(g);
            }
        }
        if (lane == 0) recheck_statuses(p);  // while the last tile is on its way out
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- softmax and sums
        const int grp = tid >> 7, t128 = tid & 127, w4 = warp & 3, r0 = grp * NR, D = p.c.head_dim;
        const int bs_shift = 31 - __clz(p.c.page_size), bar = 1 + grp;
        const uint32_t lanes = (uint32_t)(32 * w4) << 16;
        // Every barrier phase is waited for once by a thread, before the arrival of that
        // thread without which the phase after it cannot end: parities never alias.
        wait(&sm.part_full[0], 0);
        int g = 0;
        bool more = !named_any<C::kSoft>(kAllBar, dead) && sm.part[0].b >= 0;  // the same in every thread
        if (more) {
            start_queries<R>(p, sm.part[0], sm, tid, 0);
            store_queries<R>(p.scale_log2, sm.part[0].nrows, D, sm, tid);
            named_sync<C::kSoft>(kAllBar);
        }
        int n3 = 0;  // n mod 3
        for (int n = 0; more; ++n, n3 = n3 == 2 ? 0 : n3 + 1) {
            const Part &x = sm.part[n % kParts], &next = sm.part[(n + 1) % kParts];
            const int t0 = x.t0, t1 = x.t1;
            // tiles within [clear_lo, clear_hi] hide no token from any row
            const int clear_hi = x.pos0, clear_lo = p.window > 0 ? max(0, x.pos1 - p.window + 1) : 0;
            float acc[NR], l[NR];
            float m_run = kNegInf, mo_run = kNegInf;  // lane r: row r's running references
            float alpha = 1.f, alpha_last = 1.f;      // lane r: what row r's O so far is multiplied by
            bool moved = false, moved_last = false;
#pragma unroll
            for (int r = 0; r < NR; ++r) acc[r] = l[r] = 0.f;
            auto add_values = [&](int gg, bool rescale, float alpha) {  // O^T of tile gg into the sums
                tc_fence_after();
                uint32_t o[NR], o1[NR];
                tmem_ld<NR>(tO + (gg & 1) * 2 * R + r0 + lanes, o);
                tmem_ld<NR>(tO + (gg & 1) * 2 * R + R + r0 + lanes, o1);
                tmem_wait_ld();
                add_terms<NR>(o, o1);
                if (rescale) {
#pragma unroll
                    for (int r = 0; r < NR; ++r) acc[r] *= __shfl_sync(0xffffffffu, alpha, r);
                }
#pragma unroll
                for (int r = 0; r < NR; r += 4) {
                    const float4 f = *(const float4 *)&sm.w[warp][gg & 1][r];
                    float2 a = make_float2(acc[r], acc[r + 1]), b = make_float2(acc[r + 2], acc[r + 3]);
                    a = ffma2(make_float2(__uint_as_float(o[r]), __uint_as_float(o[r + 1])), make_float2(f.x, f.y), a);
                    b = ffma2(make_float2(__uint_as_float(o[r + 2]), __uint_as_float(o[r + 3])), make_float2(f.z, f.w), b);
                    acc[r] = a.x;
                    acc[r + 1] = a.y;
                    acc[r + 2] = b.x;
                    acc[r + 3] = b.y;
                }
            };
            const bool idle = r0 >= x.nrows;  // none of this group's rows: it only keeps step
            for (int i = t0; i < t1; ++i, ++g) {
                const int buf = g & 1, inf = g % kInfo, j0 = x.tile(i) * kTile, j = j0 + t128;
                const bool masked = j0 + kTile - 1 > clear_hi || (j0 < clear_lo && j0 + kTile > p.sinks);
                if (i + 1 == t1) {
                    wait(&sm.part_full[(n + 1) % kParts], ((n + 1) / kParts) & 1);
                    if (!dead && next.b >= 0) start_queries<R>(p, next, sm, tid, n3 == 2 ? 0 : n3 + 1);
                }
                wait(&sm.s_full[buf], (g >> 1) & 1);
                if (idle) {
                    if (masked && C::kGroups > 1) named_sync<C::kSoft>(kLookBar);
                    if (i > t0) wait(&sm.o_full, (g - 1) & 1);
                    if (lane == 0) mbar_arrive(&sm.p_full);
                    continue;
                }
                const float4 info = sm.page_info[inf][t128 >> bs_shift];
                const bool far = info.w != 0.f;  // the same in every thread
                tc_fence_after();
                uint32_t s[NR], s1[NR];
                tmem_ld<NR>(tS + buf * 2 * R + r0 + lanes, s);
                tmem_ld<NR>(tS + buf * 2 * R + R + r0 + lanes, s1);
                tmem_wait_ld();
                add_terms<NR>(s, s1);
                float v[NR];  // y: log2 scores with the value's scale
                const float2 ks2 = make_float2(info.x, info.x), lv2 = make_float2(info.y, info.y);
#pragma unroll
                for (int r = 0; r < NR; r += 4) {
                    const float4 c = *(const float4 *)&sm.c[r0 + r];
                    const float2 f0 = fmul2(make_float2(__uint_as_float(s[r]), __uint_as_float(s[r + 1])), ks2);
                    const float2 f1 = fmul2(make_float2(__uint_as_float(s[r + 2]), __uint_as_float(s[r + 3])), ks2);
                    const float2 y0 = ffma2(f0, make_float2(c.x, c.y), lv2), y1 = ffma2(f1, make_float2(c.z, c.w), lv2);
                    v[r] = y0.x;
                    v[r + 1] = y0.y;
                    v[r + 2] = y1.x;
                    v[r + 3] = y1.y;
                }
                if (masked) {
                    // Some row does not see some token of the tile.  Rows are token-major,
                    // so the rows that see token j are an interval: from the first at a
                    // position >= j to the last at a position < j + window.
                    const int first = x.r.len - x.r.n, base = x.rt * R + r0;
                    const int lo = j - first <= 0 ? 0 : (j - first >= x.r.n ? NR : min(NR, max(0, (j - first) * p.group - base)));
                    int hi = min(NR, max(0, x.nrows - r0));
                    if (p.window > 0 && j >= p.sinks && j - first + p.window < x.r.n)
                        hi = min(hi, max(0, (j - first + p.window) * p.group - base));
                    const uint32_t below_hi = hi >= 32 ? 0xffffffffu : (1u << hi) - 1;
                    const uint32_t sees = lo >= hi ? 0u : below_hi & ~((1u << lo) - 1);
                    // 0 times a NaN is a NaN: a value row that some rows do not see is
                    // cleared if no row sees it, or if it holds a NaN, which then
                    // reaches the rows that see it through their probability
                    const bool any = j <= x.pos1 && (p.window == 0 || j > x.pos0 - p.window || j < p.sinks);
                    const bool all = j <= x.pos0 && (p.window == 0 || j > x.pos1 - p.window || j < p.sinks);
                    const int slot = (2 * g + 1) % NS;
                    wait(&sm.full[slot], ((2 * g + 1) / NS) & 1);
                    uint4 *row = (uint4 *)(sm.ring[slot] + t128 * 128);
                    bool spoilt = false;
                    if (any && !all) {
                        uint32_t nan = 0;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const uint4 q = row[(c + lane) & 7];
                            nan |= __vcmpeq4(q.x & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(q.y & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                                   __vcmpeq4(q.z & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(q.w & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        }
                        spoilt = nan != 0;
                    }
                    __syncwarp();
                    // one group clears; with two, both have looked before it does
                    if constexpr (C::kGroups > 1) named_sync<C::kSoft>(kLookBar);
                    if ((!any || spoilt) && grp == 0) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) row[(c + lane) & 7] = make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                    const float put = spoilt ? __int_as_float(0x7fffffff) : 0.f;
#pragma unroll
                    for (int r = 0; r < NR; ++r) v[r] = (sees >> r) & 1 ? v[r] + put : kNegInf;
                }
                // the tile's largest y of every row: over the warp, then over the four
                // warps, which each keep the rows' references for themselves (lane = row)
#pragma unroll
                for (int r = 0; r < NR; r += 4) {
                    const float4 f = make_float4(redux_max(v[r]), redux_max(v[r + 1]), redux_max(v[r + 2]), redux_max(v[r + 3]));
                    *(float4 *)&sm.red[buf][w4][r0 + r] = f;  // every lane the same: no branch
                }
                if (far) {  // and the largest x
                    float y[NR];
#pragma unroll
                    for (int r = 0; r < NR; ++r) y[r] = v[r];
                    far_maxima<NR>(y, sm.page_info[inf][t128 >> bs_shift].y, &sm.red_far[w4][r0], lane);
                }
                named_sync<128>(bar);
                float x_ref = 0.f, x_beta = 0.f;  // lane r, far: row r's largest x, its weight in l
                {
                    const int k = lane & (NR - 1), r = r0 + k;
                    const float mt = fmaxf(fmaxf(sm.red[buf][0][r], sm.red[buf][1][r]), fmaxf(sm.red[buf][2][r], sm.red[buf][3][r]));
                    const bool some = mt > kNegInf;
                    const float ref = some ? mt : 0.f, mo = some ? ref + sm.lt[inf] : kNegInf;
                    float mm = some ? ref : kNegInf;  // at most the tile's largest x
                    if (far && some)
                        mm = fmaxf(fmaxf(sm.red_far[0][r], sm.red_far[1][r]), fmaxf(sm.red_far[2][r], sm.red_far[3][r]));
                    const bool moves = mm > m_run + kRefStep, moves_o = mo > mo_run + kRefStep;  // also from -inf
                    moved_last = moved;
                    alpha_last = alpha;
                    moved = __any_sync(0xffffffffu, moves || moves_o);
                    if (moved) {
                        alpha = moves_o ? ex2_approx(mo_run - mo) : 1.f;  // 0 from -inf
                        mo_run = moves_o ? mo : mo_run;
                        const float alpha_l = moves ? ex2_approx(m_run - mm) : 1.f;
                        m_run = moves ? mm : m_run;
#pragma unroll
                        for (int r = 0; r < NR; ++r) l[r] *= __shfl_sync(0xffffffffu, alpha_l, r);
                    }
                    // with 16 rows, lanes 16 .. 31 write what lanes 0 .. 15 do
                    sm.nref[warp][buf][k] = 8.f - ref;
                    sm.beta[warp][buf][k] = some ? ex2_approx(ref - m_run - 8.f) : 1.f;
                    sm.w[warp][buf][k] = some ? ex2_approx(mo - mo_run - 8.f) : 1.f;
                    if (far) {
                        x_ref = some ? mm : 0.f;
                        x_beta = some ? ex2_approx(mm - m_run) : 1.f;
                    }
                    __syncwarp();
                }
                if (far) {
                    float y[NR];
#pragma unroll
                    for (int r = 0; r < NR; ++r) y[r] = v[r];
                    far_weights<NR>(y, sm.page_info[inf][t128 >> bs_shift].y, x_ref, x_beta);
#pragma unroll
                    for (int r = 0; r < NR; ++r) l[r] += y[r];
                    named_sync<128>(bar);  // every warp has read red_far
                }
                uint32_t first[NR / 4], rest[NR / 4];
                const float iv = sm.page_info[inf][t128 >> bs_shift].z;
                const float2 iv2 = make_float2(iv, iv);
#pragma unroll
                for (int r = 0; r < NR; r += 4) {
                    const float4 b = *(const float4 *)&sm.beta[warp][buf][r], f = *(const float4 *)&sm.nref[warp][buf][r];
                    float2 z[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int k = r + 2 * e;
                        z[e] = fadd2(make_float2(v[k], v[k + 1]), e ? make_float2(f.z, f.w) : make_float2(f.x, f.y));
                        z[e].x = ex2_approx(z[e].x);
                        z[e].y = ex2_approx(z[e].y);
                        const float2 ll = ffma2(fmul2(z[e], iv2), e ? make_float2(b.z, b.w) : make_float2(b.x, b.y), make_float2(l[k], l[k + 1]));
                        l[k] = ll.x;
                        l[k + 1] = ll.y;
                    }
                    split_e4m3x4(z[0], z[1], first[r / 4], rest[r / 4]);
                }
                if (i > t0) wait(&sm.o_full, (g - 1) & 1);  // the last tile's product has read P
#pragma unroll
                for (int k = 0; k < NR / 16; ++k) {
                    *(uint4 *)(sm.p[0][r0 / 16 + k] + t128 * 16) = make_uint4(first[4 * k], first[4 * k + 1], first[4 * k + 2], first[4 * k + 3]);
                    *(uint4 *)(sm.p[1][r0 / 16 + k] + t128 * 16) = make_uint4(rest[4 * k], rest[4 * k + 1], rest[4 * k + 2], rest[4 * k + 3]);
                }
                fence_async_shared();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full);
                if (i > t0) add_values(g - 1, moved_last, alpha_last);
            }
            // the next part (told before the last tile) sends its queries before this part's
            // last product is waited for
            // (every warp has the last scores here: the queries may go); after a wait that
            // ran out anywhere, this part is the CTA's last and the whole call has failed
            const bool lost = named_any<C::kSoft>(kAllBar, dead);
            more = !lost && next.b >= 0;
            if (more) store_queries<R>(p.scale_log2, next.nrows, D, sm, tid);
            wait(&sm.o_full, (g - 1) & 1);
            if (!idle) add_values(g - 1, moved, alpha);
            tc_fence_before();
            const float lt = warp_sum_scatter<NR>(l, lane);
            if (lane < NR) sm.red[0][w4][r0 + lane] = lt;
            named_sync<128>(bar);
            if (w4 == 0 && lane < NR) {
                const int r = r0 + lane;
                const float sum = sm.red[0][0][r] + sm.red[0][1][r] + sm.red[0][2][r] + sm.red[0][3][r];
                sm.m[r] = m_run;
                sm.mo[r] = mo_run;
                sm.l[r] = x.whole ? output_factor(mo_run, m_run, sum) : sum;
                if (p.lse && x.whole && r < x.nrows) store_lse(p, x, x.rt * R + r, m_run, sum);
            }
            named_sync<128>(bar);
            if (x.whole) {
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    if (r0 + r < x.nrows && t128 < D)
                        ((uint16_t *)p.out)[sm.out_at[n3][r0 + r] + t128] =
                            (uint16_t)pack_bf16x2(acc[r] * sm.l[r0 + r], 0.f);
            } else {
                float *slot = slot_of(p, blockIdx.x, x.t0 == 0, R);
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    if (r0 + r < x.nrows && t128 < D) slot[(r0 + r) * D + t128] = acc[r];
                if (t128 < NR && r0 + t128 < x.nrows) {
                    slot[R * D + r0 + t128] = sm.m[r0 + t128];
                    slot[R * D + R + r0 + t128] = sm.l[r0 + t128];
                    slot[R * D + 2 * R + r0 + t128] = sm.mo[r0 + t128];
                }
                if (arrive_last<C::kSoft>(p, x.c0, x.c1 - x.c0 + 1, &sm.flag, kAllBar, failed))
                    join_parts<uint16_t, C::kSoft, R, 1>(p, x);
            }
            __syncwarp();  // this warp reads the part no more
            if (lane == 0) mbar_arrive(&sm.part_empty[n % kParts]);
        }
    }
    tc_fence_before();
    const bool lost = __syncthreads_or(dead || failed);
    if (warp == C::kSoft / 32 + 1) tmem_free(tm, C::kCols);
    if (lost) fail_call<kTcThreads<R, W>>(p);
}

// ------------------------------------------------------------------ host
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 got = fn.load();
    if (!got) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn.store(got = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f));
        cudaGetLastError();
    }
    return got;
}

// The codes as a map {head_dim, page_size, heads, pages}: a box is one page of one head,
// its rows filled with zeros to 128 bytes and swizzled.
bool codes_map(const spec_kv_cache &c, const void *codes, CUtensorMap *map) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.num_heads,
                                (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.token_stride, (cuuint64_t)c.head_stride, (cuuint64_t)c.page_stride};
    const cuuint32_t box[4] = {128, (cuuint32_t)c.page_size, 1, 1}, one[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(codes), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int R, int W>
int launch_tc(const AttnParams &p, int dev, int sms, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
    using C = TcShape<R>;
    constexpr int bytes = (int)sizeof(TcShared<R>);
    static_assert(C::kPerSM * (bytes + 1024) <= 228 * 1024, "shared memory of an SM");
    static std::atomic<bool> set[64];
    if (!set[dev].load()) {
        const cudaError_t e = cudaFuncSetAttribute(attention_tc_kernel<R, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) {
            note_cuda_error((int)e);
            return SPEC_ECUDA;
        }
        set[dev].store(true);
    }
    const int ctas = C::kPerSM * sms < kMaxCtas ? C::kPerSM * sms : kMaxCtas;
    attention_tc_kernel<R, W><<<ctas, kTcThreads<R, W>, bytes, st>>>(p, kmap, vmap);
    return launch_status();
}

}  // namespace
}  // namespace specv

using namespace specv;

extern "C" size_t spec_cache_attention_workspace_size(int num_query_heads, int num_heads, int head_dim, int dtype) {
    if (num_query_heads <= 0 || num_heads <= 0 || num_query_heads % num_heads || head_dim <= 0 || (head_dim & 15) ||
        head_dim > SPEC_KV_MAX_HEAD_DIM || (dtype != SPEC_BF16 && dtype != SPEC_F32))
        return 0;
    const size_t slot = sizeof(float) * kMaxRows * ((size_t)head_dim + 3);
    return SPEC_CACHE_ATTENTION_COUNTERS + 2 * kMaxCtas * slot;
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
    if (((uintptr_t)q % esz) || ((uintptr_t)out & 15) || ((uintptr_t)out_lse & 3)) return SPEC_EINVAL;
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
    p.tickets = (uint64_t *)ws;
    static_assert(sizeof(uint64_t) * kMaxCtas + sizeof(int) <= SPEC_CACHE_ATTENTION_COUNTERS, "counters");
    p.failed = (int *)((char *)ws + SPEC_CACHE_ATTENTION_COUNTERS) - 1;
    p.partial = (float *)((char *)ws + SPEC_CACHE_ATTENTION_COUNTERS);
    const cudaStream_t st = (cudaStream_t)cuda_stream;
    p.q_vec = !((uintptr_t)q & 15) && !((ld_q * esz) & 15);
    // bf16 heads of up to 128 columns (one swizzled row of a tile): the tensor cores, in
    // row tiles of 16, 32 or 64
    alignas(64) CUtensorMap kmap, vmap;
    if (esz == 2 && cache->head_dim <= 128 && codes_map(*cache, cache->k, &kmap) && codes_map(*cache, cache->v, &vmap)) {
        const int64_t rows = (int64_t)max_query * p.group;
        // One warp's copies go one after another, about 5 cycles a row and 20 a copy, so
        // with small pages a second warp pays: 304 heads of 64 columns, 8192 tokens in
        // pages of 16, take 107 us with one and 84 with two.  It costs registers: in pages
        // of 64 the same takes 79 us with one and 84 with two.  With 32 rows there are none
        // to spare (128 us with one, 204 with two); with 64 and one CTA an SM there are
        // (222 us with one, 217 with two).
        if (rows > 32) return launch_tc<64, 2>(p, dev, sms, kmap, vmap, st);
        if (rows > 16) return launch_tc<32, 1>(p, dev, sms, kmap, vmap, st);
        if (cache->page_size > 32) return launch_tc<16, 1>(p, dev, sms, kmap, vmap, st);
        return launch_tc<16, 2>(p, dev, sms, kmap, vmap, st);
    }
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
