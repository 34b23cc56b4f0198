// kv_cache.cu -- the 8-bit paged key/value cache: writing and reading back (sm_103a).
#include <type_traits>

#include "kv_common.cuh"

namespace specv {
namespace {

// n / d as the high half of a product: exact for n * d < 2^32, with m = ceil(2^32 / d), d > 1.
struct Divisor {
    uint32_t d, m;
};
inline Divisor divisor(uint32_t d) { return {d, d > 1 ? (uint32_t)((((uint64_t)1 << 32) + d - 1) / d) : 0u}; }
__device__ __forceinline__ uint32_t quotient(uint32_t n, const Divisor &v) { return v.d > 1 ? __umulhi(n, v.m) : n; }

struct KvParams {
    spec_kv_cache c;
    const void *src[2];  // append: new keys, values; rows ld[i] elements apart
    int64_t ld[2];
    void *dst[2];  // gather: keys, values out
    const int32_t *cu, *start, *table;
    int32_t *status;
    int B, ld_table, n_tokens, max_new;
    Divisor per_token, per_head, per_row;  // vectors of 8 of a head, of 16 of a head, of 16 of a row
};

constexpr int kExpMin = -100, kExpMax = 119;  // exponents of a written scale

// The exponent of the smallest power of two 2^e with amax <= 448 * 2^e = 1.75 * 2^(8+e):
// the exponent field less 8, one more where the mantissa is above 1.75.
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, kExpMin), kExpMax);  // zero and denormals have exponent field 0: the lowest
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// q, a rounded quotient or product, for rounding to e4m3 as the exact one, which is larger
// by a number of `rest`'s sign: rounding twice goes wrong only where q is a tie between
// two codes (its low 19 bits are then zero) and the exact one is not.
__device__ __forceinline__ float off_tie(float q, float rest) {
    const uint32_t u = __float_as_uint(q);
    if ((u & 0x7ffffu) || rest == 0.f || !(fabsf(q) < 500.f) || q == 0.f) return q;
    return __uint_as_float((rest > 0.f) == (q > 0.f) ? u + 1 : u - 1);
}
// x / s for rounding to e4m3, s any positive number.  (It is at least 2^kExpMin; below
// 2^-40 both are scaled so that the remainder does not underflow.)
__device__ __noinline__ float quotient_for_e4m3(float x, float s) {
    const float up = s < 0x1p-40f ? 0x1p60f : 1.f;
    x *= up;
    s *= up;
    const float q = x / s;
    return off_tie(q, fmaf(-q, s, x));
}
// A power of two whose inverse is a normal number.
__device__ __forceinline__ bool power_of_two(float x) { return (__float_as_uint(x) & 0x7fffffu) == 0 && x < 0x1p126f; }

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __int_as_float(0x7f800000); }

// Request b's new tokens, or false where its offsets or lengths are not usable.
__device__ __forceinline__ bool request_range(const KvParams &p, int b, int &row0, int &n, int &from) {
    row0 = p.cu[b];
    const int row1 = p.cu[b + 1];
    from = p.start ? p.start[b] : 0;
    n = row1 - row0;
    return row0 >= 0 && row1 >= row0 && row1 <= p.n_tokens && n <= p.max_new && from >= 0 &&
           (int64_t)from + n <= min((int64_t)p.ld_table * p.c.page_size, (int64_t)0x7fffffff);
}

// ------------------------------------------------------------------ append
// One CTA per touched page, head and keys | values: the page's scale is one number for
// all of its tokens, so a CTA sees all of them.  Reading the new entries twice (first
// for their largest magnitude, then to round them) costs nothing in DRAM: at most
// 128 x 256 elements, the first kHeld vectors a thread held in registers, the rest
// read again out of L1.  A page is at most 4096 vectors of 8 and in a verify step one
// or a few tokens, so a CTA is small: 128 threads.  64 requests of 8 tokens, 8 heads of
// 128, bf16, take 4.0 us in a graph, launch and three dependent reads; 6 prompts of 700
// to 8000 tokens, 4 heads of 96, fp32, 18.4 us, 4 TB/s of reading and writing (15.0 us
// where the rows lie in L2): a short CTA waits for its rows with nothing else to do.
constexpr int kHeld = 4, kAppendThreads = 128;

template <int ESZ, bool VEC>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(KvParams p) {
    const int b = blockIdx.z >> 1, kv = blockIdx.z & 1, h = blockIdx.y, j = blockIdx.x, tid = threadIdx.x;
    const int bs = p.c.page_size, D = p.c.head_dim;
    int row0, n, from;
    const bool ok = request_range(p, b, row0, n, from);
    const int first_page = from / bs;
    if (j == 0 && h == 0 && kv == 0) {  // this CTA also answers for the request
        int st = ok ? SPEC_STATUS_OK : SPEC_STATUS_BAD_LENGTH;
        bool bad = false;
        if (ok && n > 0)
            for (int i = first_page + tid; i <= (from + n - 1) / bs; i += kAppendThreads) {
                const int page = p.table[(int64_t)b * p.ld_table + i];
                bad |= page < 0 || page >= p.c.num_pages;
            }
        bad = __syncthreads_or(bad);
        if (bad) st = SPEC_STATUS_BAD_PAGE;
        if (tid == 0) p.status[b] = st;
    }
    if (!ok) return;
    const int64_t p0 = (int64_t)(first_page + j) * bs;  // the page's first position
    if (p0 >= (int64_t)from + n || n == 0) return;
    const int page = p.table[(int64_t)b * p.ld_table + first_page + j];
    if (page < 0 || page >= p.c.num_pages) return;
    const int slot0 = j == 0 ? from - (int)p0 : 0;                       // tokens kept, then new ones
    const int m = (int)min((int64_t)bs, (int64_t)from + n - p0) - slot0;  // new tokens of this page
    const int src_row = row0 + (int)(p0 + slot0 - from);

    const char *src = (const char *)p.src[kv] + ((int64_t)src_row * p.ld[kv] + (int64_t)h * D) * ESZ;
    const int64_t src_step = p.ld[kv] * ESZ;
    const uint32_t vpt = D >> 3;
    const int nvec = m * (int)vpt;  // vectors of 8 elements, at most 128 * 32
    auto read = [&](int v, float(&x)[8]) {
        const uint32_t t = quotient(v, p.per_token);
        load8<ESZ, VEC>(src + (int64_t)t * src_step + (v - t * vpt) * (8 * ESZ), x);
    };
    float held[kHeld][8];
    float amax = 0.f;  // the largest magnitude, an infinity included, a NaN not
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int v = tid + i * kAppendThreads;
        if (v < nvec) read(v, held[i]);
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        if (tid + i * kAppendThreads >= nvec) break;
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(held[i][e]));
    }
    for (int v = tid + kHeld * kAppendThreads; v < nvec; v += kAppendThreads) {
        float x[8];
        read(v, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
    }
    __shared__ float s_max[kAppendThreads / 32];
    float *scale_at = (kv ? p.c.v_scale : p.c.k_scale) + (int64_t)page * p.c.num_heads + h;
    const float had = slot0 > 0 ? *scale_at : 0.f;
    auto block_max = [&](float a) {
        a = warp_max(a);
        if ((tid & 31) == 0) s_max[tid >> 5] = a;
        __syncthreads();  // also: every thread has read the present scale
        a = s_max[0];
#pragma unroll
        for (int w = 1; w < kAppendThreads / 32; ++w) a = fmaxf(a, s_max[w]);
        return a;
    };
    amax = block_max(amax);
    const bool infinite = !finite(amax);
    if (infinite) {  // rare: again, over the finite entries
        amax = 0.f;
        for (int v = tid; v < nvec; v += kAppendThreads) {
            float x[8];
            read(v, x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (finite(x[e])) amax = fmaxf(amax, fabsf(x[e]));
        }
        __syncthreads();
        amax = block_max(amax);
    }
    const float scale = fmaxf(exp2_int(scale_exponent(amax)), had);
    if (tid == 0) *scale_at = scale;

    char *codes = (char *)(kv ? p.c.v : p.c.k) + (int64_t)page * p.c.page_stride + (int64_t)h * p.c.head_stride;
    // A scale that this kernel wrote is a power of two, and multiplying by its inverse
    // rounds nothing; one kept from another writer of the cache may be any number.
    const float inv = 1.f / scale;
    auto put = [&](auto exact, int v, const float(&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float a = x[2 * e] * inv, c = x[2 * e + 1] * inv;
            if constexpr (!exact.value) {
                a = quotient_for_e4m3(x[2 * e], scale);
                c = quotient_for_e4m3(x[2 * e + 1], scale);
            }
            if (infinite) {  // an infinity becomes a NaN: inf - inf
                a = finite(x[2 * e]) ? a : x[2 * e] - x[2 * e];
                c = finite(x[2 * e + 1]) ? c : x[2 * e + 1] - x[2 * e + 1];
            }
            w[e] = float2_to_e4m3x2(a, c);
        }
        const uint32_t t = quotient(v, p.per_token);
        *(uint2 *)(codes + (int64_t)(slot0 + (int)t) * p.c.token_stride + (v - t * vpt) * 8) =
            make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    };
    auto put_all = [&](auto exact) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int v = tid + i * kAppendThreads;
            if (v < nvec) put(exact, v, held[i]);
        }
        for (int v = tid + kHeld * kAppendThreads; v < nvec; v += kAppendThreads) {
            float x[8];
            read(v, x);
            put(exact, v, x);
        }
    };
    if (power_of_two(scale)) put_all(std::true_type{});
    else put_all(std::false_type{});
    if (slot0 > 0 && scale > had) {  // the kept tokens, in the grown scale
        const float ratio = had / scale;
        const bool exact = power_of_two(had);
        const int kept = slot0 * (D >> 4);
        for (int v = tid; v < kept; v += kAppendThreads) {
            const uint32_t t = quotient(v, p.per_head);
            uint4 *at = (uint4 *)(codes + (int64_t)t * p.c.token_stride + (v - t * (D >> 4)) * 16);
            uint4 q = *at;
            uint32_t *w = &q.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 a = e4m3x2_to_float2(w[e] & 0xffffu), c = e4m3x2_to_float2(w[e] >> 16);
                float p[4] = {a.x * ratio, a.y * ratio, c.x * ratio, c.y * ratio};
                if (!exact) {
                    const float f[4] = {a.x, a.y, c.x, c.y};
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = off_tie(p[i], fmaf(f[i], ratio, -p[i]));
                }
                w[e] = float2_to_e4m3x2(p[0], p[1]) | (float2_to_e4m3x2(p[2], p[3]) << 16);
            }
            *at = q;
        }
    }
}

// ------------------------------------------------------------------ gather
// A CTA takes a few output rows (every head, keys and values): one thread a row finds
// the row's request by bisection of the offsets, its page and slot; then all threads
// stream 16 codes at a time.  The first ceil(B / 8) CTAs instead answer for the
// requests' lengths and pages, one warp a request.  Bound by DRAM writes: 16 prompts of
// 2000 to 8000 tokens, 8 heads of 128, read back as bf16 take 80 us, 6.1 TB/s (95 us
// with two 16-byte stores for each 32 bytes); three short ends of caches 3.0 us.
constexpr int kGatherThreads = 256, kGatherRows = 32;

// 16 values (32 bytes of bf16, 64 of fp32).  WIDE: 32-byte aligned, and stored 32 bytes
// at a time, so that a thread writes whole sectors.
template <bool WIDE>
__device__ __forceinline__ void store32(void *dst, const uint32_t (&w)[8]) {
    if constexpr (WIDE) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        __stcs((uint4 *)dst, make_uint4(w[0], w[1], w[2], w[3]));
        __stcs((uint4 *)dst + 1, make_uint4(w[4], w[5], w[6], w[7]));
    }
}

template <int ESZ, bool WIDE>
__device__ __forceinline__ void store16(void *dst, uint4 q, float scale) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    float f[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = e4m3x2_to_float2(w[i] & 0xffffu), c = e4m3x2_to_float2(w[i] >> 16);
        f[4 * i] = a.x * scale;
        f[4 * i + 1] = a.y * scale;
        f[4 * i + 2] = c.x * scale;
        f[4 * i + 3] = c.y * scale;
    }
    uint32_t o[8];
    if constexpr (ESZ == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
        store32<WIDE>(dst, o);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(f[8 * h + i]);
            store32<WIDE>((char *)dst + 32 * h, o);
        }
    }
}

template <int ESZ, bool WIDE>
__global__ void __launch_bounds__(kGatherThreads) kv_gather_kernel(KvParams p, int rows_per, int check_blocks) {
    const int tid = threadIdx.x, lane = tid & 31, bs = p.c.page_size, D = p.c.head_dim, H = p.c.num_heads;
    if ((int)blockIdx.x < check_blocks) {
        const int b = blockIdx.x * (kGatherThreads / 32) + (tid >> 5);
        if (b >= p.B) return;
        int row0, n, from;
        if (!request_range(p, b, row0, n, from)) {
            if (lane == 0) p.status[b] = SPEC_STATUS_BAD_LENGTH;
            return;
        }
        bool bad = false;
        if (n > 0)
            for (int i = from / bs + lane; i <= (from + n - 1) / bs; i += 32) {
                const int page = p.table[(int64_t)b * p.ld_table + i];
                bad |= page < 0 || page >= p.c.num_pages;
            }
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) p.status[b] = bad ? SPEC_STATUS_BAD_PAGE : SPEC_STATUS_OK;
        return;
    }
    __shared__ int s_page[kGatherRows], s_slot[kGatherRows];
    const int r0 = (blockIdx.x - check_blocks) * rows_per, nr = min(rows_per, p.n_tokens - r0);
    if (tid < nr) {
        const int r = r0 + tid;
        int lo = 0, hi = p.B;  // the last b in [0, B] with cu[b] <= r
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.cu[mid] <= r) lo = mid;
            else hi = mid - 1;
        }
        int page = -2, slot = 0, row0, n, from;  // -2: no request's row
        if (lo < p.B && p.cu[lo] <= r && request_range(p, lo, row0, n, from) && r < row0 + n) {
            const int pos = from + r - row0;
            page = p.table[(int64_t)lo * p.ld_table + pos / bs];
            if (page < 0 || page >= p.c.num_pages) page = -1;
            slot = pos % bs;
        }
        s_page[tid] = page;
        s_slot[tid] = slot;
    }
    __syncthreads();
    const int vph = D >> 4, vpr = vph * H, total = nr * vpr;
    constexpr int U = 4;  // loads in flight a thread
    for (int v0 = tid; v0 < total; v0 += U * kGatherThreads) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const char *codes = (const char *)(kv ? p.c.v : p.c.k);
            const float *scales = kv ? p.c.v_scale : p.c.k_scale;
            uint4 q[U];
            float s[U];
            int page[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int v = v0 + u * kGatherThreads;
                page[u] = -2;
                if (v >= total) continue;
                const int r = nr > 1 ? quotient(v, p.per_row) : 0, i = v - r * vpr, h = quotient(i, p.per_head), c = i - h * vph;
                page[u] = s_page[r];
                if (page[u] >= 0) {
                    q[u] = ld_stream_v4(codes + (int64_t)page[u] * p.c.page_stride + (int64_t)h * p.c.head_stride +
                                        (int64_t)s_slot[r] * p.c.token_stride + c * 16);
                    s[u] = __ldg(scales + (int64_t)page[u] * H + h);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (page[u] == -2) continue;
                const int v = v0 + u * kGatherThreads;
                if (page[u] < 0) {
                    q[u] = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
                    s[u] = 1.f;
                }
                // rows, heads and 16-element vectors are contiguous in the output
                store16<ESZ, WIDE>((char *)p.dst[kv] + ((int64_t)r0 * vpr + v) * 16 * ESZ, q[u], s[u]);
            }
        }
    }
}

}  // namespace
}  // namespace specv

using namespace specv;

extern "C" int spec_kv_append(const spec_kv_cache *cache, const void *k, const void *v, int dtype, int64_t ld_k,
                              int64_t ld_v, int n_tokens, int B, const int32_t *cu_new, int max_new,
                              const int32_t *cached_len, const int32_t *page_table, int ld_table,
                              int32_t *out_status, void *cuda_stream) {
    if (dtype != SPEC_BF16 && dtype != SPEC_F32) return SPEC_EINVAL;
    if (B < 0 || n_tokens < 0 || max_new < 0 || ld_table < 0) return SPEC_EINVAL;
    int rc = check_cache(cache);
    if (rc) return rc;
    if (B == 0) return SPEC_OK;
    if (B > SPEC_MAX_BATCH) return SPEC_EUNSUPPORTED;
    if (!cu_new || !cached_len || !out_status || (ld_table > 0 && !page_table)) return SPEC_EINVAL;
    const int64_t row = (int64_t)cache->num_heads * cache->head_dim;
    const int esz = dtype == SPEC_BF16 ? 2 : 4;
    if (n_tokens > 0 && (!k || !v || ld_k < row || ld_v < row)) return SPEC_EINVAL;
    if (((uintptr_t)k % esz) || ((uintptr_t)v % esz)) return SPEC_EINVAL;
    int dev = 0, sms = 0;
    if ((rc = kv_device_info(&dev, &sms))) return rc;
    if ((rc = kv_check_device_pointer(cache->k, dev))) return rc;
    KvParams p = {};
    p.c = *cache;
    p.src[0] = k;
    p.src[1] = v;
    p.ld[0] = ld_k;
    p.ld[1] = ld_v;
    p.cu = cu_new;
    p.start = cached_len;
    p.table = page_table;
    p.status = out_status;
    p.B = B;
    p.ld_table = ld_table;
    p.n_tokens = n_tokens;
    p.max_new = max_new;
    p.per_token = divisor(cache->head_dim / 8);
    p.per_head = divisor(cache->head_dim / 16);
    // pages max_new tokens can touch, whatever slot the first one has
    const int bs = cache->page_size;
    const int pages = (int)(((int64_t)max_new + bs - 2) / bs) + 1;
    const dim3 grid(pages, cache->num_heads, 2 * B);
    const bool vec = !(((uintptr_t)k | (uintptr_t)v) & 15) && !((ld_k * esz) & 15) && !((ld_v * esz) & 15);
    const cudaStream_t s = (cudaStream_t)cuda_stream;
    if (esz == 2 && vec) kv_append_kernel<2, true><<<grid, kAppendThreads, 0, s>>>(p);
    else if (esz == 2) kv_append_kernel<2, false><<<grid, kAppendThreads, 0, s>>>(p);
    else if (vec) kv_append_kernel<4, true><<<grid, kAppendThreads, 0, s>>>(p);
    else kv_append_kernel<4, false><<<grid, kAppendThreads, 0, s>>>(p);
    return launch_status();
}

extern "C" int spec_kv_gather(const spec_kv_cache *cache, int B, const int32_t *cu_out, int n_out,
                              const int32_t *first, const int32_t *page_table, int ld_table, void *out_k,
                              void *out_v, int dtype, int32_t *out_status, void *cuda_stream) {
    if (dtype != SPEC_BF16 && dtype != SPEC_F32) return SPEC_EINVAL;
    if (B < 0 || n_out < 0 || ld_table < 0) return SPEC_EINVAL;
    int rc = check_cache(cache);
    if (rc) return rc;
    if (B == 0) return SPEC_OK;
    if (B > SPEC_MAX_BATCH) return SPEC_EUNSUPPORTED;
    if (!cu_out || !out_status || (ld_table > 0 && !page_table)) return SPEC_EINVAL;
    if (n_out > 0 && (!out_k || !out_v)) return SPEC_EINVAL;
    if (((uintptr_t)out_k | (uintptr_t)out_v) & 15) return SPEC_EINVAL;
    int dev = 0, sms = 0;
    if ((rc = kv_device_info(&dev, &sms))) return rc;
    if ((rc = kv_check_device_pointer(cache->k, dev))) return rc;
    KvParams p = {};
    p.c = *cache;
    p.dst[0] = out_k;
    p.dst[1] = out_v;
    p.cu = cu_out;
    p.start = first;
    p.table = page_table;
    p.status = out_status;
    p.B = B;
    p.ld_table = ld_table;
    p.n_tokens = n_out;
    p.max_new = 0x7fffffff;
    p.per_head = divisor(cache->head_dim / 16);
    p.per_row = divisor((uint32_t)cache->num_heads * (cache->head_dim / 16));
    // about 1024 vectors of 16 codes a CTA, keys and values each
    const int vpr = cache->num_heads * (cache->head_dim / 16);
    int rows = 1024 / vpr;
    rows = rows < 1 ? 1 : (rows > kGatherRows ? kGatherRows : rows);
    const int check = (B + 7) / 8;
    const unsigned grid = (unsigned)(check + (n_out + (int64_t)rows - 1) / rows);
    const cudaStream_t s = (cudaStream_t)cuda_stream;
    const bool wide = !(((uintptr_t)out_k | (uintptr_t)out_v) & 31);
    if (dtype == SPEC_BF16 && wide) kv_gather_kernel<2, true><<<grid, kGatherThreads, 0, s>>>(p, rows, check);
    else if (dtype == SPEC_BF16) kv_gather_kernel<2, false><<<grid, kGatherThreads, 0, s>>>(p, rows, check);
    else if (wide) kv_gather_kernel<4, true><<<grid, kGatherThreads, 0, s>>>(p, rows, check);
    else kv_gather_kernel<4, false><<<grid, kGatherThreads, 0, s>>>(p, rows, check);
    return launch_status();
}
