// rotary.cu -- rotary positions of queries and keys, with one or several axes (sm_103a).
//
// Mathematics.  Pair i of a head's rotated columns is turned by the angle
//   a = position[axis_i] * freq_i:   (x, y) -> (x cos a - y sin a, y cos a + x sin a).
// The angle matters modulo a turn only, so it is kept in turns as a 64-bit fixed-point
// fraction: F_i = (freq_i / 2 pi) 2^64 modulo 2^64, and position * F_i in wrapping integer
// arithmetic is the phase, off by |position| 2^-64 turns (2^-33 at the farthest position).
// Its highest 32 bits, less the nearest quarter turn, go through sincospi in 32 bits.  A
// product in fp32 would be off by 2^-24 of an angle of up to 2^31 radians.
//
// Bound by memory: queries and keys are read and written once.  Few tokens: short CTAs of kTokens
// tokens, whose sines and cosines are computed once each, into shared memory, while the first loads
// are under way; a thread keeps those of its 8 pairs in registers for all its heads (8 tokens of 40
// heads: 2.8 us).  From 16 tokens an SM on: warps that stay and copy their next tokens, or shares
// of them, asynchronously (16411 tokens of 40 heads: 57 us, 5.9 TB/s).  Sizes and addresses that
// 16-byte words do not fit go pair by pair.
#include <atomic>

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

// (freq / 2 pi) 2^64 modulo 2^64, cut to an integer: the 53-bit mantissa times the 128 highest
// bits of 1 / 2 pi.  Integer instructions: those on doubles are few to a cycle on this chip
// (with them 16411 tokens of 40 heads took 95 us).
__device__ __forceinline__ uint64_t turns_a_position(double freq) {
    constexpr uint64_t hi = 0x28be60db9391054aull, lo = 0x7f09d5f47d4d3770ull;  // 2^128 / 2 pi
    const uint64_t bits = (uint64_t)__double_as_longlong(freq);
    const int exponent = (int)(bits >> 52 & 0x7ff) - 1023, shift = 116 - exponent;
    const uint64_t m = (bits & 0xfffffffffffffull) | 1ull << 52;
    const uint64_t w1 = __umul64hi(m, lo) + m * hi, w2 = __umul64hi(m, hi) + (w1 < m * hi ? 1 : 0);
    uint64_t f = 0;
    if (shift >= 128) f = shift < 192 ? w2 >> (shift - 128) : 0;
    else if (shift >= 64) f = shift == 64 ? w1 : w1 >> (shift - 64) | w2 << (128 - shift);
    else if (shift >= 0) f = shift == 0 ? m * lo : m * lo >> shift | w1 << (64 - shift);
    return bits >> 63 ? 0 - f : f;
}
// The scale of a pair's turn: NaN where the frequency is not a number, infinite, or 2^64 and more
// (there those 128 bits no longer hold the angle at every position).
__device__ __forceinline__ float scale_at(double freq, float scale) {
    return fabs(freq) < 18446744073709551616.0 ? scale : __int_as_float(0x7fffffff);
}

// cos and sin, times the scale, of a phase of 2^-32 turns.  The nearest quarter turn is taken off
// as an integer: what becomes a float is an eighth of a turn at most and loses 2^-28 turns (half a
// turn would lose 2^-26).
__device__ __forceinline__ float2 turn(uint32_t phase, float scale) {
    const uint32_t quarter = phase + 0x20000000u;  // its number in the two highest bits
    const int rest = (int)(phase - (quarter & 0xc0000000u));
    float s, c;
    sincospif((float)rest * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
    const bool odd = quarter & 0x40000000u;
    const uint32_t x = __float_as_uint(odd ? s : c) ^ ((quarter ^ quarter << 1) & 0x80000000u);
    const uint32_t y = __float_as_uint(odd ? c : s) ^ (quarter & 0x80000000u);
    return make_float2(__uint_as_float(x) * scale, __uint_as_float(y) * scale);
}

// cos and sin of pair i at the token's positions, times the scale.
__device__ __forceinline__ float2 turn_of(const RotaryParams &p, int64_t token, int i) {
    const int a = p.axis ? min(max(p.axis[i], 0), p.axes - 1) : 0;
    const int pos = p.position[a * p.ld_pos + token];
    return turn((uint32_t)(((uint64_t)(int64_t)pos * turns_a_position(p.freq[i])) >> 32), scale_at(p.freq[i], p.scale));
}

// 8 columns of a unit: one 16-byte word of bf16, or two of fp32 that lie `words` columns apart,
// so that neighbouring lanes always touch neighbouring words.
__device__ __forceinline__ void load8_rw(const uint16_t *p, int, float (&x)[8]) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ void load8_rw(const float *p, int words, float (&x)[8]) {
    asm volatile("ld.global.L1::no_allocate.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "l"(p));
    asm volatile("ld.global.L1::no_allocate.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]) : "l"(p + words));
}
__device__ __forceinline__ void store8(uint16_t *p, int, const float (&x)[8]) {
    *(uint4 *)p = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float *p, int words, const float (&x)[8]) {
    *(float4 *)p = make_float4(x[0], x[1], x[2], x[3]);
    *(float4 *)(p + words) = make_float4(x[4], x[5], x[6], x[7]);
}

// 8 pairs: (a[e], b[e]), or neighbours in a and then in b.
template <bool ADJ>
__device__ __forceinline__ void turn8(const float (&a)[8], const float (&b)[8], const float (&c)[8], const float (&d)[8],
                                      float (&y)[8], float (&z)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (ADJ) {
            const float *x = e < 4 ? a : b;
            float *o = e < 4 ? y : z;
            const int k = 2 * (e & 3);
            o[k] = x[k] * c[e] - x[k + 1] * d[e];
            o[k + 1] = x[k + 1] * c[e] + x[k] * d[e];
        } else {
            y[e] = a[e] * c[e] - b[e] * d[e];
            z[e] = b[e] * c[e] + a[e] * d[e];
        }
    }
}

// Groups of 8 columns: a unit is 8 of the first half of the rotated columns and 8 of the
// second (8 pairs either way: one of each half, or neighbours), or 8 that are only copied.
// Of a head's `units` the first `turning` rotate.
struct Unit {
    int c0, words;  // the first group's first word, and how far its words lie apart
    bool turns;     // with a second group c0 + pairs
};
template <typename T>
__device__ __forceinline__ Unit unit_at(const RotaryParams &p, int u, int turning, int units) {
    constexpr int W = 16 / sizeof(T);  // columns of a word
    if (u < turning) return {u * W, turning * W, true};
    return {2 * p.pairs + (u - turning) * W, (units - turning) * W, false};
}
// Pair k is number `e` of unit `u`: where its cosine and sine go.
template <typename T, bool ADJ>
__device__ __forceinline__ int place_of(int k, int pairs, int turning) {
    constexpr int W = 16 / sizeof(T);
    const int column = ADJ ? 2 * k : k, second = column >= pairs, c = column - second * pairs;
    const int word = c / W, v = word / turning, u = word - v * turning;
    const int e = ADJ ? second * 4 + (v * W + c % W) / 2 : v * W + c % W;
    return ((e >> 1) * (kMaxPairs / 8) + u) * 2 + (e & 1);
}

template <typename T>
constexpr int kHeadsEach = sizeof(T) == 2 ? 4 : 2;  // heads a thread has in flight: all it takes
template <typename T, bool ADJ>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryParams p, int heads_each) {
    __shared__ float4 turns[kTokens][4][kMaxPairs / 8];  // [token][two pairs][unit]
    const int turning = p.pairs / 8, units = turning + (p.D - 2 * p.pairs) / 8;
    const int64_t token0 = (int64_t)blockIdx.x * kTokens;
    const int tid = threadIdx.x, heads = p.heads[0] + p.heads[1];
    const int h0 = blockIdx.y * heads_each, h1 = min(heads, h0 + heads_each);
    const int slots = kThreads / units, u = tid % units, s = tid / units;
    const int groups = slots / kTokens;  // heads of a token under way at once (units <= 32: at least 2)
    const int token = s % kTokens, hg = s / kTokens;
    const bool works = hg < groups && token0 + token < p.T;
    const Unit x = unit_at<T>(p, u, turning, units);
    constexpr int U = kHeadsEach<T>;
    float a[U][8], b[U][8];
    auto at = [&](bool out, int h) {
        const int w = h >= p.heads[0];
        T *rows = (T *)(out ? (w ? p.dst[1] : p.dst[0]) : const_cast<void *>(w ? p.src[1] : p.src[0]));
        const int64_t ld = out ? (w ? p.ld_dst[1] : p.ld_dst[0]) : (w ? p.ld_src[1] : p.ld_src[0]);
        return rows + (token0 + token) * ld + (int64_t)(h - (w ? p.heads[0] : 0)) * p.D;
    };
    const int h = h0 + hg;
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (works && h + i * groups < h1) {
            const T *src = at(false, h + i * groups);
            load8_rw(src + x.c0, x.words, a[i]);
            if (x.turns) load8_rw(src + x.c0 + p.pairs, x.words, b[i]);
        }
    for (int i = tid; i < kTokens * p.pairs; i += kThreads) {
        const int t = i / p.pairs, k = i - t * p.pairs;
        if (token0 + t < p.T) ((float2 *)turns[t])[place_of<T, ADJ>(k, p.pairs, turning)] = turn_of(p, token0 + t, k);
    }
    __syncthreads();
    if (!works) return;
    float c[8], d[8];
    if (x.turns)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 f = turns[token][i][u];
            c[2 * i] = f.x;
            d[2 * i] = f.y;
            c[2 * i + 1] = f.z;
            d[2 * i + 1] = f.w;
        }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        if (h + i * groups >= h1) break;
        T *dst = at(true, h + i * groups);
        if (!x.turns) {
            store8(dst + x.c0, x.words, a[i]);
            continue;
        }
        float y[8], z[8];
        turn8<ADJ>(a[i], b[i], c, d, y, z);
        store8(dst + x.c0, x.words, y);
        store8(dst + x.c0 + p.pairs, x.words, z);
    }
}

// Many tokens: warps that stay, each taking every W-th share of a token.  A lane copies its
// units of the next share (and the one after, with two ahead) into its own places of shared memory
// asynchronously while it turns this one's, so a warp's loads never wait for its stores, and
// needs no barrier but its own copies' completion.  The frequencies of a lane's pairs stay in
// registers.
template <typename T>
__device__ __forceinline__ void read8(const uint4 *s, float (&x)[8]) {  // places 32 apart: a lane's own
    if constexpr (sizeof(T) == 2) {
        const uint4 v = s[0];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = s[32 * i];
            x[4 * i] = __uint_as_float(v.x);
            x[4 * i + 1] = __uint_as_float(v.y);
            x[4 * i + 2] = __uint_as_float(v.z);
            x[4 * i + 3] = __uint_as_float(v.w);
        }
    }
}

constexpr int kStreamSmem = 200 * 1024;
// Units of a share of a token (all are full warps but the last), and the bytes of a warp's
// place for one: a lane's units, two groups of 8 columns each.
__host__ __device__ inline int share_units(int heads, int units, int shares) {
    return ((heads * units + shares - 1) / shares + 31) / 32 * 32;
}
__host__ __device__ inline int stream_slot(int heads, int units, int shares, int esz) {
    return share_units(heads, units, shares) * 2 * 8 * esz;
}

template <typename T, bool ADJ>
__global__ void __launch_bounds__(512) rotary_stream_kernel(RotaryParams p, int stages, int shares) {
    extern __shared__ __align__(16) uint8_t stream_smem[];
    __shared__ float4 turns[16][4][kMaxPairs / 8];
    constexpr int V = sizeof(T) / 2;  // 16-byte words of 8 columns
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int turning = p.pairs / 8, units = turning + (p.D - 2 * p.pairs) / 8;
    const int heads = p.heads[0] + p.heads[1], per = share_units(heads, units, shares);
    const int slot = stream_slot(heads, units, shares, sizeof(T));
    uint4 *place = (uint4 *)(stream_smem + (size_t)warp * stages * slot) + lane;
    const int step_h = 32 / units, step_u = 32 - step_h * units;
    auto each_unit = [&](int share, auto f) {  // of the lane: f(whether it is the first, head, unit)
        int i = share * per + lane, h = i / units, u = i - h * units;
        const int end = min(heads * units, (share + 1) * per);
        for (bool start = true; i < end; i += 32, start = false) {
            f(start, h, u);
            h += step_h;
            u += step_u;
            if (u >= units) {
                u -= units;
                ++h;
            }
        }
    };
    const int64_t items = (int64_t)p.T * shares;  // (token, share)
    auto fetch = [&](int64_t item, int stage) {
        if (item < items) {
            const int64_t token = item / shares;
            uint32_t at = smem_addr(place) + stage * slot;
            const T *rq = (const T *)p.src[0] + token * p.ld_src[0], *rk = (const T *)p.src[1] + token * p.ld_src[1] - (int64_t)p.heads[0] * p.D;
            each_unit((int)(item - token * shares), [&](bool, int h, int u) {
                const Unit x = unit_at<T>(p, u, turning, units);
                const T *src = (h < p.heads[0] ? rq : rk) + (int64_t)h * p.D + x.c0;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + v * 512), "l"(src + v * x.words) : "memory");
                if (x.turns)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + (V + v) * 512), "l"(src + p.pairs + v * x.words) : "memory");
                at += 2 * V * 512;
            });
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // the lane's pairs, 32 apart
    constexpr int kPairsEach = kMaxPairs / 32;
    uint64_t F[kPairsEach];
    float scale[kPairsEach];
    int place_k[kPairsEach];
    const int32_t *row[kPairsEach];
#pragma unroll
    for (int i = 0; i < kPairsEach; ++i) {
        const int k = lane + 32 * i;
        F[i] = k < p.pairs ? turns_a_position(p.freq[k]) : 0;
        scale[i] = k < p.pairs ? scale_at(p.freq[k], p.scale) : 0.f;
        place_k[i] = k < p.pairs ? place_of<T, ADJ>(k, p.pairs, turning) : 0;
        row[i] = p.position + (k < p.pairs && p.axis ? min(max(p.axis[k], 0), p.axes - 1) : 0) * p.ld_pos;
    }
    const int64_t first = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp, step = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int i = 0; i < stages - 1; ++i) fetch(first + i * step, i);
    const bool fixed = step_u == 0;  // a lane's units are one of every head it visits
    int stage = 0;
    for (int64_t item = first; item < items; item += step) {
        const int64_t token = item / shares;
        fetch(item + (stages - 1) * step, stage == 0 ? stages - 1 : stage - 1);
        __syncwarp();  // the last item's turns have been read
#pragma unroll
        for (int i = 0; i < kPairsEach; ++i) {
            const int k = lane + 32 * i;
            if (k >= p.pairs) break;
            ((float2 *)turns[warp])[place_k[i]] = turn((uint32_t)(((uint64_t)(int64_t)row[i][token] * F[i]) >> 32), scale[i]);
        }
        __syncwarp();
        if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
        else asm volatile("cp.async.wait_group 1;" ::: "memory");
        const uint4 *at = (const uint4 *)((const uint8_t *)place + stage * slot);
        T *wq = (T *)p.dst[0] + token * p.ld_dst[0], *wk = (T *)p.dst[1] + token * p.ld_dst[1] - (int64_t)p.heads[0] * p.D;
        float c[8], d[8];
        each_unit((int)(item - token * shares), [&](bool start, int h, int u) {
            const Unit x = unit_at<T>(p, u, turning, units);
            T *dst = (h < p.heads[0] ? wq : wk) + (int64_t)h * p.D + x.c0;
            float a[8], b[8], y[8], z[8];
            read8<T>(at, a);
            if (x.turns) {
                read8<T>(at + V * 32, b);
                if (!fixed || start)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 f = turns[warp][i][u];
                        c[2 * i] = f.x;
                        d[2 * i] = f.y;
                        c[2 * i + 1] = f.z;
                        d[2 * i + 1] = f.w;
                    }
                turn8<ADJ>(a, b, c, d, y, z);
                store8(dst, x.words, y);
                store8(dst + p.pairs, x.words, z);
            } else {
                store8(dst, x.words, a);
            }
            at += 2 * V * 32;
        });
        stage = stage + 1 == stages ? 0 : stage + 1;
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

template <typename T, bool ADJ>
int launch_stream(const RotaryParams &p, int sms, int dev, int stages, int shares, int warps, int slot, cudaStream_t st) {
    static std::atomic<bool> set[64];
    if (!set[dev].load()) {
        const cudaError_t e = cudaFuncSetAttribute(rotary_stream_kernel<T, ADJ>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem);
        if (e != cudaSuccess) {
            note_cuda_error((int)e);
            return SPEC_ECUDA;
        }
        set[dev].store(true);
    }
    rotary_stream_kernel<T, ADJ><<<sms, warps * 32, warps * stages * slot, st>>>(p, stages, shares);
    return launch_status();
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
    if (!q || !out_q || !position || (pairs > 0 && (!freq || (num_axes > 1 && !axis)))) return SPEC_EINVAL;
    if (num_heads > 0 && (!k || !out_k || ld_k < row_k || ld_out_k < row_k)) return SPEC_EINVAL;
    if (ld_q < row_q || ld_out_q < row_q || (num_axes > 1 && ld_position < n_tokens && ld_position != 0)) return SPEC_EINVAL;
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
    const int blocks = (int)(((int64_t)n_tokens + kTokens - 1) / kTokens), heads = num_query_heads + num_heads;
    bool vec = !((pairs & 7) | ((head_dim - 2 * pairs) & 7));
    for (int w = 0; w < (num_heads ? 2 : 1); ++w)
        vec = vec && !(((uintptr_t)p.src[w] | (uintptr_t)p.dst[w]) & 15) && !(((p.ld_src[w] | p.ld_dst[w]) * esz) & 15);
    if (!vec) {
        if (esz == 2) rotary_any_kernel<uint16_t><<<blocks, kThreads, 0, st>>>(p);
        else rotary_any_kernel<float><<<blocks, kThreads, 0, st>>>(p);
        return launch_status();
    }
    const int units = pairs / 8 + (head_dim - 2 * pairs) / 8;
    // Many tokens, whole or in shares so small that 16 warps have two places each in shared
    // memory (9000 tokens of 72 heads: 61 us in halves, 76 whole; 16411 of 40: 57 and 61), three
    // where that leaves 16 warps.
    int shares = 1;
    while (shares < 4 && (int64_t)stream_slot(heads, units, shares, esz) * 2 * 16 > kStreamSmem) shares *= 2;
    const int slot = stream_slot(heads, units, shares, esz);
    if ((int64_t)slot * 2 * 4 <= kStreamSmem && n_tokens >= 16 * sms) {
        const int stages = slot * 3 * 16 <= kStreamSmem ? 3 : 2;
        const int fit = kStreamSmem / (slot * stages), warps = fit < 16 ? fit : 16;
        if (esz == 2 && adjacent) return launch_stream<uint16_t, true>(p, sms, dev, stages, shares, warps, slot, st);
        if (esz == 2) return launch_stream<uint16_t, false>(p, sms, dev, stages, shares, warps, slot, st);
        if (adjacent) return launch_stream<float, true>(p, sms, dev, stages, shares, warps, slot, st);
        return launch_stream<float, false>(p, sms, dev, stages, shares, warps, slot, st);
    }
    // as many heads a CTA as its threads take in one go, in equal shares; with few tokens fewer
    const int groups = kThreads / units / kTokens;
    const int most = groups * (esz == 2 ? kHeadsEach<uint16_t> : kHeadsEach<float>), split = (heads + most - 1) / most;
    int each = (heads + split - 1) / split;
    while (each > groups && (int64_t)blocks * ((heads + each - 1) / each) < 2 * sms) each = (each + 1) / 2;
    const dim3 grid(blocks, (heads + each - 1) / each);
    if (esz == 2 && adjacent) rotary_kernel<uint16_t, true><<<grid, kThreads, 0, st>>>(p, each);
    else if (esz == 2) rotary_kernel<uint16_t, false><<<grid, kThreads, 0, st>>>(p, each);
    else if (adjacent) rotary_kernel<float, true><<<grid, kThreads, 0, st>>>(p, each);
    else rotary_kernel<float, false><<<grid, kThreads, 0, st>>>(p, each);
    return launch_status();
}
