// prompt_attention.cu -- causal attention of packed prompts (sm_103a).
//
// Mathematics.  With log2 scores x_j = scale * log2(e) * (q . k_j), a row's output is
//   out = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m)
// for any reference m; one pass over the keys keeps (m, l, o) and multiplies l and o by
// 2^(m - m') when the reference moves to m'.
//
// Work split.  An item is (request, key head, row tile); a row tile's rows are queries of
// the request that share the key head, token-major: row = t * group + g, so that grouped
// heads read a key tile once and a diagonal tile wastes little.  A tile of keys that no row
// of the item sees is not visited; one that every row sees in full is not masked.
//
// fp32 queries, and bf16 where the tensor cores cannot serve (odd strides), take fp32
// arithmetic throughout: attention_rows_kernel.
#include <atomic>

#include "prompt_common.cuh"

namespace specv {
namespace {

// ------------------------------------------------------------------ fp32 arithmetic
// A CTA takes an item of R rows (16 threads down, 16 across: R / 16 rows and 4 keys a thread)
// and walks over tiles of 64 keys in shared memory.
constexpr int kRowsThreads = 256, kKeys = 64;

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) { return x; }
template <>
__device__ __forceinline__ float to_float(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

// ND: columns of the output in 32s.
template <typename T, int ND>
struct RowsShape {
    static constexpr int kEach = ND == 4 ? 8 : 4;  // rows a thread: two CTAs an SM up to 96 columns
    static constexpr int kRows = 16 * kEach;
    static constexpr int kStride = 32 * ND + 4;    // floats of a row: 16 bytes of skew
    static constexpr int kBytes = 4 * (kRows * kStride + 2 * kKeys * kStride + kRows * (kKeys + 4));
};

template <typename T, int ND, bool VEC>
__global__ void __launch_bounds__(kRowsThreads, ND <= 3 ? 2 : 1) attention_rows_kernel(PromptParams p, int levels) {
    using S = RowsShape<T, ND>;
    constexpr int E = S::kEach, R = S::kRows, LD = S::kStride, LP = kKeys + 4;
    extern __shared__ __align__(16) float rows_smem[];
    float *sq = rows_smem, *sk = sq + R * LD, *sv = sk + kKeys * LD, *sp = sv + kKeys * LD;
    __shared__ int found[2];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, lane = tid & 31, D = p.D;
    write_prompt_statuses(p, blockIdx.x * kRowsThreads + tid, gridDim.x * kRowsThreads);
    // Items, the heads of a row tile side by side.  Where that asks for few that do not exist,
    // the last row tiles of all requests come first, then the last but one (levels: row tiles
    // of the longest request): the longest items are not left to the end.  5 prompts of 60 to
    // 1700 tokens, 10 heads of 80: 487 us so, 570 request after request.
    for (int64_t item = blockIdx.x;; item += gridDim.x) {
        const int64_t whole = item / p.parts, which = whole / p.H;
        const int part = (int)(item - whole * p.parts), h = (int)(whole - which * p.H);
        int b, tile;
        if (levels > 0) {
            const int level = (int)(which / p.B);
            if (level >= levels) return;
            b = (int)(which - (int64_t)level * p.B);
            tile = levels - 1 - level;
            if (tile >= ((int64_t)load_prompt(p, b).n * p.group + R - 1) / R) continue;
        } else {
            // the request that holds row tile `which`; its last tiles, the longest, come first
            if (tid < 32) {
                int64_t before = 0;
                int at = -1, nth = 0;
                for (int b0 = 0; b0 < p.B && at < 0; b0 += 32) {
                    const int mine = b0 + lane < p.B ? (int)(((int64_t)load_prompt(p, b0 + lane).n * p.group + R - 1) / R) : 0;
                    int64_t upto = mine;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
                        if (lane >= o) upto += x;
                    }
                    const uint32_t past = __ballot_sync(0xffffffffu, before + upto > which);
                    if (past) {
                        const int w = __ffs(past) - 1;
                        at = b0 + w;
                        const int tiles = __shfl_sync(0xffffffffu, mine, w);
                        nth = tiles - 1 - (int)(which - before - (__shfl_sync(0xffffffffu, upto, w) - tiles));
                    }
                    before += __shfl_sync(0xffffffffu, upto, 31);
                }
                if (lane == 0) {
                    found[0] = at;
                    found[1] = nth;
                }
            }
            __syncthreads();
            b = found[0];
            tile = found[1];
            if (b < 0) return;
        }
        const Prompt r = load_prompt(p, b);
        const int first = tile * R, nrows = min(R, r.n * p.group - first);  // the host keeps n * group below 2^31
        const int off = r.m - r.n;  // position of query 0
        const int pos0 = off + first / p.group, pos1 = off + (first + nrows - 1) / p.group;
        const Span span = span_of<kKeys>(p, pos0, pos1);
        auto global_row = [&](int row) {  // of q and out, in elements without the row stride
            const int f = first + row;
            return make_int2(r.row0 + f / p.group, h * p.group + f % p.group);
        };
        for (int i = tid; i < R * (LD / 4); i += kRowsThreads) {
            const int row = i / (LD / 4), c = (i - row * (LD / 4)) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row < nrows && c < D) {
                const int2 g = global_row(row);
                const T *src = (const T *)p.q + g.x * p.ld_q + (int64_t)g.y * D + c;
                x = make_float4(to_float(src[0]), to_float(src[1]), to_float(src[2]), to_float(src[3]));
                x.x *= p.scale_log2, x.y *= p.scale_log2, x.z *= p.scale_log2, x.w *= p.scale_log2;
            }
            *(float4 *)(sq + row * LD + c) = x;
        }
        float m[E], l[E];
        float2 o[E][ND];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            m[e] = kNegInf;
            l[e] = 0.f;
#pragma unroll
            for (int c = 0; c < ND; ++c) o[e][c] = make_float2(0.f, 0.f);
        }
        int pos[E];  // a thread's rows: ty + 16 e
#pragma unroll
        for (int e = 0; e < E; ++e) pos[e] = ty + 16 * e < nrows ? off + (first + ty + 16 * e) / p.group : -1;
        // A tile of keys or values on its way to shared memory; rows past the request's are 0.
        const int d4 = D / 4;
        auto load_tile = [&](float *dst, const void *src, int64_t ld, int j0) {
            const T *rows = (const T *)src + (int64_t)(r.key0 + j0) * ld + (int64_t)h * D;
            const int have = r.m - j0;
            for (int x = tid; x < kKeys * d4; x += kRowsThreads) {
                const int row = (int)((uint32_t)x / (uint32_t)d4), c = (x - row * d4) * 4;
                const T *from = rows + (row < have ? row * ld + c : 0);  // in bounds: j0 < r.m
                float *to = dst + row * LD + c;
                if (sizeof(T) == 4 && VEC) {
                    const int bytes = row < have ? 16 : 0;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(to)), "l"(from), "r"(bytes) : "memory");
                } else {
                    const float4 y = make_float4(to_float(from[0]), to_float(from[1]), to_float(from[2]), to_float(from[3]));
                    *(float4 *)to = row < have ? y : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        auto arrived = [] { asm volatile("cp.async.wait_group 1;" ::: "memory"); };  // all but the last one sent
        const int i0 = (int)((int64_t)span.count * part / p.parts), i1 = (int)((int64_t)span.count * (part + 1) / p.parts);
        if (i0 < i1) load_tile(sk, p.k, p.ld_k, span.tile(i0) * kKeys);
        for (int i = i0; i < i1; ++i) {
            const int j0 = span.tile(i) * kKeys;
            const bool masked = j0 + kKeys - 1 > pos0 || (p.window > 0 && j0 <= pos1 - p.window && j0 + kKeys > p.sinks) || nrows < R;
            load_tile(sv, p.v, p.ld_v, j0);  // under way during the scores
            arrived();
            __syncthreads();
            // scores: pairs of columns summed side by side
            float2 s[E][4];
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int k = 0; k < 4; ++k) s[e][k] = make_float2(0.f, 0.f);
            for (int c = 0; c < D; c += 4) {
                float4 a[E], d[4];
#pragma unroll
                for (int e = 0; e < E; ++e) a[e] = *(const float4 *)(sq + (ty + 16 * e) * LD + c);
#pragma unroll
                for (int k = 0; k < 4; ++k) d[k] = *(const float4 *)(sk + (tx + 16 * k) * LD + c);
#pragma unroll
                for (int e = 0; e < E; ++e)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        s[e][k] = ffma2(make_float2(a[e].x, a[e].y), make_float2(d[k].x, d[k].y), s[e][k]);
                        s[e][k] = ffma2(make_float2(a[e].z, a[e].w), make_float2(d[k].z, d[k].w), s[e][k]);
                    }
            }
            __syncthreads();  // the keys have been read: the next ones' copy runs until the next scores
            if (i + 1 < i1) load_tile(sk, p.k, p.ld_k, span.tile(i + 1) * kKeys);
            else asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float x[4], top = kNegInf;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[k] = s[e][k].x + s[e][k].y;
                    if (masked && !visible(p, pos[e], j0 + tx + 16 * k)) x[k] = kNegInf;
                    top = fmaxf(top, x[k]);
                }
#pragma unroll
                for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                const float now = fmaxf(m[e], top), ref = now == kNegInf ? 0.f : now;
                const float alpha = ex2_approx(m[e] - ref);  // 0 from -inf
                m[e] = now;
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float y = ex2_approx(x[k] - ref);
                    sum += y;
                    sp[(ty + 16 * e) * LP + tx + 16 * k] = y;
                }
                l[e] = l[e] * alpha + sum;
#pragma unroll
                for (int c = 0; c < ND; ++c) {
                    o[e][c].x *= alpha;
                    o[e][c].y *= alpha;
                }
            }
            arrived();
            int strange = 0;  // values that are not finite
            if (masked) {
                __syncthreads();
                for (int x = tid; x < kKeys * d4; x += kRowsThreads) {
                    const int row = (int)((uint32_t)x / (uint32_t)d4);
                    const float4 d = *(const float4 *)(sv + row * LD + (x - row * d4) * 4);
                    strange |= !isfinite(d.x) || !isfinite(d.y) || !isfinite(d.z) || !isfinite(d.w);
                }
            }
            strange = __syncthreads_or(strange);
            if (strange) {  // a value that a row does not see must not meet its zero
                for (int k = 0; k < kKeys; ++k)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        if (!visible(p, pos[e], j0 + k)) continue;
                        const float y = sp[(ty + 16 * e) * LP + k];
#pragma unroll
                        for (int c = 0; c < ND; ++c) {
                            const float2 d = *(const float2 *)(sv + k * LD + tx * 2 + 32 * c);
                            o[e][c] = ffma2(make_float2(y, y), d, o[e][c]);
                        }
                    }
            } else {
                for (int k = 0; k < kKeys; k += 4) {
                    float4 y[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) y[e] = *(const float4 *)(sp + (ty + 16 * e) * LP + k);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        float2 d[ND];
#pragma unroll
                        for (int c = 0; c < ND; ++c) d[c] = *(const float2 *)(sv + (k + kk) * LD + tx * 2 + 32 * c);
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            const float f = kk == 0 ? y[e].x : kk == 1 ? y[e].y : kk == 2 ? y[e].z : y[e].w;
#pragma unroll
                            for (int c = 0; c < ND; ++c) o[e][c] = ffma2(make_float2(f, f), d[c], o[e][c]);
                        }
                    }
                }
            }
            __syncthreads();
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float sum = l[e];
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            const int row = ty + 16 * e;
            if (row >= nrows) continue;
            const int2 g = global_row(row);
            if (p.parts > 1) {  // unnormalised, with the reference and the sum
                const int64_t slot = ((int64_t)part * p.n_q + g.x) * p.Hq + g.y;
#pragma unroll
                for (int c = 0; c < ND; ++c)
                    if (tx * 2 + 32 * c < D) *(float2 *)(p.part_o + slot * D + tx * 2 + 32 * c) = o[e][c];
                if (tx == 0) p.part_ml[slot] = make_float2(m[e] == kNegInf ? 0.f : m[e], sum);
                continue;
            }
            const float f = sum == 0.f ? 0.f : 1.f / sum;  // a row that sees nothing: o is 0
            T *dst = (T *)p.out + ((int64_t)g.x * p.Hq + g.y) * D;
#pragma unroll
            for (int c = 0; c < ND; ++c) {
                const int col = tx * 2 + 32 * c;
                if (col >= D) continue;
                if (sizeof(T) == 2) *(uint32_t *)(dst + col) = pack_bf16x2(o[e][c].x * f, o[e][c].y * f);
                else *(float2 *)(dst + col) = make_float2(o[e][c].x * f, o[e][c].y * f);
            }
            if (p.lse && tx == 0) p.lse[(int64_t)g.x * p.Hq + g.y] = sum == 0.f ? kNegInf : (m[e] + log2f(sum)) * 0.6931471805599453f;
        }
        __syncthreads();
    }
}

template <typename T, int ND, bool VEC>
int launch_rows(const PromptParams &p, int dev, cudaStream_t st) {
    using S = RowsShape<T, ND>;
    static std::atomic<bool> set[64];
    if (!set[dev].load()) {
        const cudaError_t e = cudaFuncSetAttribute(attention_rows_kernel<T, ND, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
        if (e != cudaSuccess) {
            note_cuda_error((int)e);
            return SPEC_ECUDA;
        }
        set[dev].store(true);
    }
    // row tiles at most: every request's last one may be partial
    const int64_t tiles = ((int64_t)p.n_q * p.group + S::kRows - 1) / S::kRows + p.B;
    const int64_t levels = ((int64_t)p.max_query * p.group + S::kRows - 1) / S::kRows;
    const bool by_level = levels * p.B <= 4 * tiles;
    const int64_t items = (by_level ? levels * p.B : tiles) * p.H * p.parts;
    const unsigned grid = (unsigned)(items < 1 ? 1 : items < 1 << 20 ? items : 1 << 20);
    attention_rows_kernel<T, ND, VEC><<<grid, kRowsThreads, S::kBytes, st>>>(p, by_level ? (int)levels : 0);
    const int rc = launch_status();
    return rc || p.parts == 1 ? rc : launch_prompt_join(p, sizeof(T) == 2, st);
}

template <typename T, bool VEC>
int launch_rows_any(const PromptParams &p, int dev, cudaStream_t st) {
    if (p.D <= 64) return launch_rows<T, 2, VEC>(p, dev, st);
    if (p.D <= 96) return launch_rows<T, 3, VEC>(p, dev, st);
    if (p.D <= 128) return launch_rows<T, 4, VEC>(p, dev, st);
    if (p.D <= 192) return launch_rows<T, 6, VEC>(p, dev, st);
    return launch_rows<T, 8, VEC>(p, dev, st);
}

}  // namespace
}  // namespace specv

using namespace specv;

extern "C" size_t spec_prompt_attention_workspace_size(int n_query, int n_key, int B, int num_query_heads, int num_heads,
                                                       int head_dim, int dtype, int window, int sinks) {
    if ((dtype != SPEC_BF16 && dtype != SPEC_F32) || n_query <= 0 || n_key <= 0 || B <= 0 || num_query_heads <= 0 ||
        num_heads <= 0 || num_query_heads % num_heads || head_dim <= 0 || window < 0 || sinks < 0)
        return 0;
    if (dtype == SPEC_F32) {
        const int parts = rows_parts(n_query, n_key, B, num_query_heads / num_heads, num_heads, window, window > 0 ? sinks : 0);
        return parts > 1 ? (size_t)parts * n_query * num_query_heads * (head_dim + 2) * sizeof(float) : 0;
    }
    if (num_query_heads / num_heads > 128) return 0;
    return prompt_plan(n_query, n_key, B, num_query_heads / num_heads, num_heads, head_dim, window, window > 0 ? sinks : 0).bytes;
}

extern "C" int spec_prompt_attention(const void *q, const void *k, const void *v, int dtype, int64_t ld_q, int64_t ld_k,
                                     int64_t ld_v, int num_query_heads, int num_heads, int head_dim, int n_query,
                                     int n_key, int B, const int32_t *cu_query, int max_query, const int32_t *cu_key,
                                     float scale, int window, int sinks, void *out, float *out_lse, int32_t *out_status, void *ws,
                                     size_t ws_bytes, void *cuda_stream) {
    if (dtype != SPEC_BF16 && dtype != SPEC_F32) return SPEC_EINVAL;
    if (B < 0 || n_query < 0 || n_key < 0 || max_query < 0 || num_query_heads <= 0 || num_heads <= 0 || head_dim <= 0 ||
        window < 0 || sinks < 0 || num_query_heads % num_heads)
        return SPEC_EINVAL;
    if (!(scale > 0.f) || !(scale * kLog2e < __builtin_huge_valf())) return SPEC_EINVAL;
    if ((head_dim & 15) || head_dim > SPEC_KV_MAX_HEAD_DIM || num_heads > 65535) return SPEC_EUNSUPPORTED;
    if (B == 0) return SPEC_OK;
    if (B > SPEC_MAX_BATCH) return SPEC_EUNSUPPORTED;
    const int group = num_query_heads / num_heads;
    if ((int64_t)max_query * group > 0x7fffffff - 256 || n_key > 0x7fffffff - 1024) return SPEC_EUNSUPPORTED;
    if (!cu_query || !out_status || (!cu_key && n_key != n_query)) return SPEC_EINVAL;
    const int esz = dtype == SPEC_BF16 ? 2 : 4;
    const int64_t row = (int64_t)num_heads * head_dim;
    if (n_query > 0 && (!q || !out || ld_q < row * group)) return SPEC_EINVAL;
    if (n_key > 0 && (!k || !v || ld_k < row || ld_v < row)) return SPEC_EINVAL;
    if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v) % esz || ((uintptr_t)out & 15) || ((uintptr_t)out_lse & 3)) return SPEC_EINVAL;
    if (((uintptr_t)cu_query | (uintptr_t)cu_key | (uintptr_t)out_status) & 3) return SPEC_EINVAL;
    const size_t need = spec_prompt_attention_workspace_size(n_query, n_key, B, num_query_heads, num_heads, head_dim, dtype, window, sinks);
    if (need > 0 && (!ws || ws_bytes < need || ((uintptr_t)ws & 255))) return SPEC_EWORKSPACE;
    // items read queries, keys and values after others have written
    const size_t out_bytes = (size_t)n_query * num_query_heads * head_dim * esz;
    auto rows_bytes = [&](int n, int64_t ld, int64_t columns) { return n > 0 ? ((size_t)(n - 1) * ld + columns) * esz : 0; };
    if (overlap(out, out_bytes, q, rows_bytes(n_query, ld_q, row * group)) || overlap(out, out_bytes, k, rows_bytes(n_key, ld_k, row)) ||
        overlap(out, out_bytes, v, rows_bytes(n_key, ld_v, row)))
        return SPEC_EINVAL;
    int dev = 0, sms = 0, rc;
    if ((rc = kv_device_info(&dev, &sms))) return rc;
    if (n_query > 0 && (rc = kv_check_device_pointer(q, dev))) return rc;
    PromptParams p = {};
    p.q = q;
    p.k = k;
    p.v = v;
    p.out = out;
    p.lse = out_lse;
    p.cu_q = cu_query;
    p.cu_k = cu_key ? cu_key : cu_query;
    p.status = out_status;
    p.ld_q = ld_q;
    p.ld_k = ld_k;
    p.ld_v = ld_v;
    p.B = B;
    p.n_q = n_query;
    p.n_k = n_key;
    p.max_query = max_query;
    p.Hq = num_query_heads;
    p.H = num_heads;
    p.group = group;
    p.D = head_dim;
    p.window = window < n_key ? window : 0;  // one that is no shorter than the keys hides none
    p.sinks = p.window > 0 ? sinks : 0;
    p.scale_log2 = scale * kLog2e;
    p.parts = 1;
    if (need > 0) {
        p.parts = esz == 2 ? prompt_plan(n_query, n_key, B, group, num_heads, head_dim, p.window, p.sinks).parts
                           : rows_parts(n_query, n_key, B, group, num_heads, p.window, p.sinks);
        p.part_o = (float *)ws;
        p.part_ml = (float2 *)((char *)ws + (size_t)p.parts * n_query * num_query_heads * head_dim * sizeof(float));
    }
    const cudaStream_t st = (cudaStream_t)cuda_stream;
    if (esz == 2) {
        rc = launch_prompt_tc(p, dev, sms, st);
        return rc == SPEC_EUNSUPPORTED ? launch_rows_any<uint16_t, false>(p, dev, st) : rc;
    }
    const bool vec = !(((uintptr_t)k | (uintptr_t)v) & 15) && !((ld_k | ld_v) & 3);  // copies of 16 bytes
    return vec ? launch_rows_any<float, true>(p, dev, st) : launch_rows_any<float, false>(p, dev, st);
}
