// kv_common.cuh -- what the 8-bit paged cache's kernels share (sm_103a): the cache's
// view, e4m3 conversions and the host-side checks.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "spec_common.cuh"
#include "spec_verify.h"

namespace specv {

// ------------------------------------------------------------------ e4m3
// Conversions are the hardware's (cvt): two codes to two halves (exact, every e4m3
// value is a half), two floats to two codes (nearest even, saturating at 448; a NaN
// gives the NaN code).  The first operand of a pair is its high half.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
    uint32_t h;
    asm("{\n .reg .b16 t;\n cvt.u16.u32 t, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}" : "=r"(h) : "r"(two));
    return h;
}

__device__ __forceinline__ float2 half2_to_float2(uint32_t h) {
    float2 f;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.f32.f16 %0, lo;\n cvt.f32.f16 %1, hi;\n}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) { return half2_to_float2(e4m3x2_to_half2(two)); }

__device__ __forceinline__ uint32_t float2_to_e4m3x2(float lo, float hi) {
    uint32_t r;
    asm("{\n .reg .b16 t;\n cvt.rn.satfinite.e4m3x2.f32 t, %2, %1;\n cvt.u32.u16 %0, t;\n}"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r;
}

// ------------------------------------------------------------------ rows of bf16 or fp32
// Eight consecutive elements as floats.  VEC: 16-byte aligned.
template <int ESZ, bool VEC>
__device__ __forceinline__ void load8(const void *p, float (&x)[8]) {
    if constexpr (ESZ == 2 && VEC) {
        const uint4 v = ld_stream_v4(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    } else if constexpr (ESZ == 4 && VEC) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = ld_stream_v4((const uint4 *)p + i);
            x[4 * i] = __uint_as_float(v.x);
            x[4 * i + 1] = __uint_as_float(v.y);
            x[4 * i + 2] = __uint_as_float(v.z);
            x[4 * i + 3] = __uint_as_float(v.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = ld_elem<ESZ>(p, i);
    }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ------------------------------------------------------------------ host
int kv_device_info(int *dev, int *sms);             // verify.cu: the current device and its SM count
int kv_check_device_pointer(const void *p, int dev);  // verify.cu: p lies on dev, or is managed memory

// What every entry point asks of a cache description.
inline int check_cache(const spec_kv_cache *c) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return SPEC_EINVAL;
    if (c->num_pages <= 0 || c->num_heads <= 0 || c->head_dim <= 0) return SPEC_EINVAL;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return SPEC_EUNSUPPORTED;
    if ((c->head_dim & 15) || c->head_dim > SPEC_KV_MAX_HEAD_DIM || c->num_heads > 65535) return SPEC_EUNSUPPORTED;
    const int64_t smallest = c->head_dim, largest = (int64_t)1 << 40;
    const int64_t strides[3] = {c->page_stride, c->head_stride, c->token_stride};
    for (int64_t s : strides)
        if (s < smallest || (s & 15) || s >= largest) return SPEC_EINVAL;
    if (((uintptr_t)c->k | (uintptr_t)c->v) & 15) return SPEC_EINVAL;
    if (((uintptr_t)c->k_scale | (uintptr_t)c->v_scale) & 3) return SPEC_EINVAL;
    return SPEC_OK;
}

inline int launch_status() {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return SPEC_OK;
    note_cuda_error((int)e);
    return SPEC_ECUDA;
}

}  // namespace specv
