// rotary.cu -- rotary positions of queries and keys, with one or several axes (sm_103a).
//
// Mathematics.  Pair i of a head's rotated columns is turned by the angle
//   a = position[axis_i] * freq_i:   (x, y) -> (x cos a - y sin a, y cos a + x sin a).
// The angle matters modulo a turn only, so it is kept in turns as a 64-bit fixed-point
// fraction: F_i = (freq_i / 2 pi) 2^64 modulo 2^64, and position * F_i in wrapping integer
// arithmetic is the phase, off by |position| 2^-64 turns (2^-33 at the farthest position).
// Its highest 32 bits, a signed number of half turns, go through sincospi in 32 bits.  A
// product in fp32 would be off by 2^-24 of an angle of up to 2^31 radians.
//
// Bound by memory: queries and keys are read and written once.  A CTA takes kTokens tokens;
// their sines and cosines are computed once each, into shared memory, while the first loads
// are under way; a thread keeps those of its 8 pairs in registers and walks over heads.
#include "kv_common.cuh"

namespace specv {
namespace {

constexpr int kThreads = 256, kTokens = 4, kMaxPairs = SPEC_KV_MAX_HEAD_DIM / 2;

struct RotaryParams {
    const void *src[2];
    void *dst[2];
    int64_t ld_src[2], ld_dst[2], ld_pos;
    const int32_t *position, *axis;
    const double *freq;
    int heads[2];
    int T, D, pairs, axes;
    bool adjacent;
    float scale;
};

// cos and sin of pair i at the token's positions, times the scale.
__device__ __forceinline__ float2 turn_of(const RotaryParams &p, int64_t token, int i) {
    const int a = p.axis ? min(max(p.axis[i], 0), p.axes - 1) : 0;
    const int pos = p.position[a * p.ld_pos + token];
    // turns a position, as a sum of two numbers: 1 / 2 pi to 106 bits
    const double f = p.freq[i], t = f * 0.15915494309189535, low = fma(f, 0.15915494309189535, -t) + f * -9.839338337591243e-18;
    const int64_t F = __double2ll_rn((t - rint(t) + low) * 18446744073709551616.0);
    const int hi = (int)(((uint64_t)(int64_t)pos * (uint64_t)F) >> 32);
    float s, c;
    sincospif((float)hi * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
    return make_float2(c * p.scale, s * p.scale);
}

__device__ __forceinline__ void load8_rw(const uint16_t *p, float (&x)[8]) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ void load8_rw(const float *p, float (&x)[8]) {
    asm volatile("ld.global.L1::no_allocate.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "l"(p));
    asm volatile("ld.global.L1::no_allocate.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]) : "l"(p + 4));
}
__device__ __forceinline__ void store8(uint16_t *p, const float (&x)[8]) {
    *(uint4 *)p = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    *(float4 *)p = make_float4(x[0], x[1], x[2], x[3]);
    *(float4 *)(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// Groups of 8 columns: a unit is 8 pairs, or 8 columns that are only copied.  Of a head's
// `units` the first `turning` rotate; ADJ: a unit is 16 consecutive columns, else 8 of each half.
template <typename T, bool ADJ>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryParams p, int heads_each) {
    __shared__ float4 turns[kTokens][4][kMaxPairs / 8];  // [token][two pairs][unit]
    const int half = p.pairs, turning = p.pairs / 8, units = turning + (p.D - 2 * p.pairs) / 8;
    const int64_t token0 = (int64_t)blockIdx.x * kTokens;
    const int tid = threadIdx.x, heads = p.heads[0] + p.heads[1];
    const int h0 = blockIdx.y * heads_each, h1 = min(heads, h0 + heads_each);
    const int slots = kThreads / units, u = tid % units, s = tid / units;
    const int groups = slots / kTokens;  // heads of a token under way at once (units <= 32: at least 2)
    const int token = s % kTokens, hg = s / kTokens;
    const bool works = hg < groups && token0 + token < p.T, turns_it = u < turning;
    const int c0 = turns_it ? (ADJ ? u * 16 : u * 8) : 2 * half + (u - turning) * 8, c1 = ADJ ? c0 + 8 : c0 + half;
    constexpr int U = sizeof(T) == 2 ? 4 : 2;  // heads in flight
    float a[U][8], b[U][8];
    auto at = [&](bool out, int h) {
        const int w = h >= p.heads[0];
        T *rows = (T *)(out ? (w ? p.dst[1] : p.dst[0]) : const_cast<void *>(w ? p.src[1] : p.src[0]));
        const int64_t ld = out ? (w ? p.ld_dst[1] : p.ld_dst[0]) : (w ? p.ld_src[1] : p.ld_src[0]);
        return rows + (token0 + token) * ld + (int64_t)(h - (w ? p.heads[0] : 0)) * p.D;
    };
    auto fetch = [&](int h) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (works && h + i * groups < h1) {
                const T *src = at(false, h + i * groups);
                load8_rw(src + c0, a[i]);
                if (turns_it) load8_rw(src + c1, b[i]);
            }
    };
    int h = h0 + hg;
    fetch(h);
    for (int i = tid; i < kTokens * p.pairs; i += kThreads) {
        const int t = i / p.pairs, k = i - t * p.pairs;
        if (token0 + t < p.T) ((float2 *)&turns[t][(k & 7) >> 1][k >> 3])[k & 1] = turn_of(p, token0 + t, k);
    }
    __syncthreads();
    if (!works) return;
    float c[8], d[8];
    if (turns_it)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 f = turns[token][i][u];
            c[2 * i] = f.x;
            d[2 * i] = f.y;
            c[2 * i + 1] = f.z;
            d[2 * i + 1] = f.w;
        }
    for (; h < h1; h += U * groups) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (h + i * groups >= h1) break;
            T *dst = at(true, h + i * groups);
            if (turns_it) {
                float y[8], z[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (ADJ) {
                        float *x = e < 4 ? a[i] : b[i], *o = e < 4 ? y : z;
                        const int k = 2 * (e & 3);
                        o[k] = x[k] * c[e] - x[k + 1] * d[e];
                        o[k + 1] = x[k + 1] * c[e] + x[k] * d[e];
                    } else {
                        y[e] = a[i][e] * c[e] - b[i][e] * d[e];
                        z[e] = b[i][e] * c[e] + a[i][e] * d[e];
                    }
                }
                store8(dst + c0, y);
                store8(dst + c1, z);
            } else {
                store8(dst + c0, a[i]);
            }
        }
        fetch(h + U * groups);
    }
}

// Any sizes and alignments: a thread takes one pair, or one column that is only copied.
template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_any_kernel(RotaryParams p) {
    __shared__ float2 turns[kTokens][kMaxPairs];
    const int64_t token0 = (int64_t)blockIdx.x * kTokens;
    const int tid = threadIdx.x, heads = p.heads[0] + p.heads[1], units = p.D - p.pairs;
    for (int i = tid; i < kTokens * p.pairs; i += kThreads) {
        const int t = i / p.pairs, k = i - t * p.pairs;
        if (token0 + t < p.T) turns[t][k] = turn_of(p, token0 + t, k);
    }
    __syncthreads();
    const int n = (int)min((int64_t)kTokens, p.T - token0) * heads * units;  // heads * units < 2^28
    auto value = [](const T *x) { return sizeof(T) == 2 ? __uint_as_float((uint32_t)*(const uint16_t *)x << 16) : *(const float *)x; };
    auto put = [](T *x, float f) {
        if (sizeof(T) == 2) *(uint16_t *)x = (uint16_t)pack_bf16x2(f, 0.f);
        else *(float *)x = f;
    };
    for (int i = tid; i < n; i += kThreads) {
        const int u = i % units, rest = i / units, h = rest % heads, t = rest / heads, w = h >= p.heads[0];
        const int64_t head = (int64_t)(h - (w ? p.heads[0] : 0)) * p.D;
        const T *src = (const T *)(w ? p.src[1] : p.src[0]) + (token0 + t) * (w ? p.ld_src[1] : p.ld_src[0]) + head;
        T *dst = (T *)(w ? p.dst[1] : p.dst[0]) + (token0 + t) * (w ? p.ld_dst[1] : p.ld_dst[0]) + head;
        if (u < p.pairs) {
            const int c0 = p.adjacent ? 2 * u : u, c1 = p.adjacent ? 2 * u + 1 : u + p.pairs;
            const float x = value(src + c0), y = value(src + c1);
            const float2 cs = turns[t][u];
            put(dst + c0, x * cs.x - y * cs.y);
            put(dst + c1, y * cs.x + x * cs.y);
        } else {
            dst[u + p.pairs] = src[u + p.pairs];
        }
    }
}

}  // namespace
}  // namespace specv

using namespace specv;

extern "C" int spec_rotary(const void *q, const void *k, int dtype, int64_t ld_q, int64_t ld_k, int num_query_heads,
                           int num_heads, int head_dim, int n_tokens, const int32_t *position, int64_t ld_position,
                           int num_axes, const double *freq, const int32_t *axis, int pairs, int adjacent, float scale,
                           void *out_q, void *out_k, int64_t ld_out_q, int64_t ld_out_k, void *cuda_stream) {
    if (dtype != SPEC_BF16 && dtype != SPEC_F32) return SPEC_EINVAL;
    if (n_tokens < 0 || num_query_heads <= 0 || num_heads < 0 || head_dim <= 0 || pairs < 0 || num_axes <= 0) return SPEC_EINVAL;
    if (2 * (int64_t)pairs > head_dim || !(scale - scale == 0.f)) return SPEC_EINVAL;
    if (head_dim > SPEC_KV_MAX_HEAD_DIM || (int64_t)num_query_heads + num_heads > 65535) return SPEC_EUNSUPPORTED;
    if (n_tokens == 0) return SPEC_OK;
    const int esz = dtype == SPEC_BF16 ? 2 : 4;
    const int64_t row_q = (int64_t)num_query_heads * head_dim, row_k = (int64_t)num_heads * head_dim;
    if (!q || !out_q || !position || (pairs > 0 && !freq) || (num_axes > 1 && !axis)) return SPEC_EINVAL;
    if (num_heads > 0 && (!k || !out_k || ld_k < row_k || ld_out_k < row_k)) return SPEC_EINVAL;
    if (ld_q < row_q || ld_out_q < row_q || (num_axes > 1 && ld_position < n_tokens)) return SPEC_EINVAL;
    if (((uintptr_t)q | (uintptr_t)out_q | (num_heads ? (uintptr_t)k | (uintptr_t)out_k : 0)) % esz) return SPEC_EINVAL;
    if (((uintptr_t)position | (uintptr_t)axis) & 3 || (uintptr_t)freq & 7) return SPEC_EINVAL;
    int dev = 0, sms = 0, rc;
    if ((rc = kv_device_info(&dev, &sms))) return rc;
    if ((rc = kv_check_device_pointer(q, dev))) return rc;
    RotaryParams p = {};
    p.src[0] = q;
    p.src[1] = k;
    p.dst[0] = out_q;
    p.dst[1] = out_k;
    p.ld_src[0] = ld_q;
    p.ld_src[1] = ld_k;
    p.ld_dst[0] = ld_out_q;
    p.ld_dst[1] = ld_out_k;
    p.ld_pos = num_axes > 1 ? ld_position : 0;
    p.position = position;
    p.axis = num_axes > 1 ? axis : nullptr;
    p.freq = freq;
    p.heads[0] = num_query_heads;
    p.heads[1] = num_heads;
    p.T = n_tokens;
    p.D = head_dim;
    p.pairs = pairs;
    p.axes = num_axes;
    p.adjacent = adjacent != 0;
    p.scale = scale;
    const cudaStream_t st = (cudaStream_t)cuda_stream;
    const int blocks = (n_tokens + kTokens - 1) / kTokens, heads = num_query_heads + num_heads;
    bool vec = !((pairs & 7) | ((head_dim - 2 * pairs) & 7));
    for (int w = 0; w < (num_heads ? 2 : 1); ++w)
        vec = vec && !(((uintptr_t)p.src[w] | (uintptr_t)p.dst[w]) & 15) && !(((p.ld_src[w] | p.ld_dst[w]) * esz) & 15);
    if (!vec) {
        if (esz == 2) rotary_any_kernel<uint16_t><<<blocks, kThreads, 0, st>>>(p);
        else rotary_any_kernel<float><<<blocks, kThreads, 0, st>>>(p);
        return launch_status();
    }
    // few tokens: the heads are split over CTAs too, down to one round of loads a thread
    const int units = pairs / 8 + (head_dim - 2 * pairs) / 8, groups = kThreads / units / kTokens;
    int each = heads;
    while (each > groups && (int64_t)blocks * ((heads + each - 1) / each) < 2 * sms) each = (each + 1) / 2;
    const dim3 grid(blocks, (heads + each - 1) / each);
    if (esz == 2 && adjacent) rotary_kernel<uint16_t, true><<<grid, kThreads, 0, st>>>(p, each);
    else if (esz == 2) rotary_kernel<uint16_t, false><<<grid, kThreads, 0, st>>>(p, each);
    else if (adjacent) rotary_kernel<float, true><<<grid, kThreads, 0, st>>>(p, each);
    else rotary_kernel<float, false><<<grid, kThreads, 0, st>>>(p, each);
    return launch_status();
}
