// page_plan.cu -- block tables and slot maps of the paged cache, built on the GPU (sm_103a).
//
// Integers only.  A request that keeps keep_b tokens and gets new_b more needs
//   need_b = ceil((keep_b + new_b) / page_size)
// pages and holds held_b: it gives back its pages need_b .. held_b - 1, or takes as many as
// it lacks.  With exclusive sums over the requests, in order,
//   G_b = pages given before b,   K_b = pages taken before b,   cu_b = tokens before b,
// the free list is a stack of `count` ids: given page number k goes to place count + k, and
// with `all` pages taken in this call, taken page number j comes from place
//   base + j,   base = count + given - all.
// So every page that moves has one source and one destination, and one pass moves them all:
// the thread of given page k writes it to the free list, or straight to its taker.
//
// One cluster of CTAs does it in one launch: every CTA computes the sums over the requests
// for itself (12 bytes a request), the moves and then the tokens are split over all threads
// of the cluster, and a cluster barrier lies between the two, after which the tables are
// read back.  Small batches take one CTA; many tokens a kernel of their own on all SMs.
//
// Bound by latency: a launch, three dependent reads and the barriers; then by the 12 bytes a
// token that are written.
#include <atomic>

#include "kv_common.cuh"

namespace specv {
namespace {

struct PlanParams {
    int32_t *free, *count, *table, *held;
    const int32_t *keep, *fresh;
    int32_t *cu, *seq_len, *position, *status;
    int64_t *slot;
    int num_pages, page_size, shift, B, width, n_out;
    bool rows_apart;  // the tokens' slots are another kernel's
};

constexpr int kRowsEach = 8;  // rows of a thread

// Inclusive sum of two 64-bit numbers over the CTA's threads; the totals in *a_all, *b_all.
template <int NT>
__device__ __forceinline__ void block_sums(int64_t &a, int64_t &b, int64_t *a_all, int64_t *b_all, int64_t (*part)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
    if (lane == 31) {
        part[warp][0] = a;
        part[warp][1] = b;
    }
    __syncthreads();
    // every warp sums the others' totals for itself
    int64_t x = lane < NT / 32 ? part[lane][0] : 0, y = lane < NT / 32 ? part[lane][1] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
            x += u;
            y += v;
        }
    }
    const int64_t xa = __shfl_sync(0xffffffffu, x, warp > 0 ? warp - 1 : 0);
    const int64_t yb = __shfl_sync(0xffffffffu, y, warp > 0 ? warp - 1 : 0);
    if (warp > 0) {
        a += xa;
        b += yb;
    }
    *a_all = __shfl_sync(0xffffffffu, x, NT / 32 - 1);
    *b_all = __shfl_sync(0xffffffffu, y, NT / 32 - 1);
}

// The last i of [lo, n) with sums[i] <= x, for sums that do not decrease and sums[lo] <= x.
template <typename T>
__device__ __forceinline__ int last_at_most(const T *sums, int n, T x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Slots and positions of rows r, r + 32, .. (kRowsEach of them): the request of the first one
// by bisection, then onwards; the table's entries are fetched together.
template <typename S>
__device__ __forceinline__ void place_rows(const PlanParams &p, int64_t r, const int32_t *cu, const S *state) {
    int pos[kRowsEach], page[kRowsEach];
    const int64_t all = p.B > 0 ? cu[p.B] : 0;
    int b = r < all ? last_at_most(cu, p.B, (int32_t)r) : 0;
#pragma unroll
    for (int i = 0; i < kRowsEach; ++i) {
        const int64_t at = r + i * 32;
        pos[i] = page[i] = -1;
        if (at < all) {
            while (cu[b + 1] <= at) ++b;
            pos[i] = p.keep[b] + (int)(at - cu[b]);
            if (state[b] == SPEC_STATUS_OK) page[i] = __ldcg(p.table + (int64_t)b * p.width + (pos[i] >> p.shift));
        }
    }
#pragma unroll
    for (int i = 0; i < kRowsEach; ++i) {
        const int64_t at = r + i * 32;
        if (at >= p.n_out) break;
        p.slot[at] = page[i] < 0 ? -1 : ((int64_t)page[i] << p.shift) | (pos[i] & (p.page_size - 1));
        p.position[at] = pos[i];
    }
}

// Shared memory: cu [B + 1] and, for each request, its first given and taken page and its
// status.  Sums of pages stay below 2^31 where they are used (the host keeps B * width so).
template <int NT>
__global__ void __launch_bounds__(NT) page_plan_kernel(PlanParams p, int ctas) {
    extern __shared__ int32_t raw[];
    int32_t *cu = raw, *given = cu + p.B + 1, *taken = given + p.B + 1;
    uint8_t *state = (uint8_t *)(taken + p.B + 1);
    __shared__ int64_t part[2][32][2];
    const int tid = threadIdx.x, rank = blockIdx.x;
    const int per = (p.B + NT - 1) / NT, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);

    // ---- sums over the requests
    const int64_t room = min((int64_t)p.width << p.shift, (int64_t)0x7fffffff);  // a length is an int32
    int64_t rows = 0, none = 0, all_rows, unused;
    for (int b = b0; b < b1; ++b) rows += max(0, p.fresh[b]);
    int64_t at = rows;
    block_sums<NT>(at, none, &all_rows, &unused, part[0]);
    at -= rows;
    int64_t give = 0, take = 0;
    for (int b = b0; b < b1; ++b) {
        const int keep = p.keep[b], fresh = p.fresh[b], held = p.held[b];
        cu[b] = (int)min(at, (int64_t)0x7fffffff);
        at += max(0, fresh);
        const bool bad = keep < 0 || fresh < 0 || held < 0 || held > p.width || (int64_t)keep + fresh > room ||
                         keep > (int64_t)held << p.shift || at > p.n_out;
        const int need = bad ? held : (int)(((int64_t)keep + fresh + p.page_size - 1) >> p.shift);
        state[b] = bad ? SPEC_STATUS_BAD_LENGTH : SPEC_STATUS_OK;
        given[b] = max(0, held - need);
        taken[b] = max(0, need - held);
        give += given[b];
        take += taken[b];
    }
    if (tid == 0) cu[p.B] = (int)min(all_rows, (int64_t)0x7fffffff);
    int64_t G = give, K = take, all_given, all_wanted;
    block_sums<NT>(G, K, &all_given, &all_wanted, part[1]);
    G -= give;
    K -= take;
    const int count = min(max(*p.count, 0), p.num_pages);
    const int64_t have = count + all_given;
    // requests are served in order: from the first one that the list cannot serve on, those
    // that need pages get none (so those served are a prefix of the takers, and the sums of
    // pages taken before a served request count served ones alone)
    __shared__ int served;
    if (tid == 0) served = 0;
    __syncthreads();
    int mine = 0;
    for (int b = b0; b < b1; ++b) {
        const int g = given[b], k = taken[b];
        given[b] = (int)G;
        taken[b] = (int)min(K, (int64_t)0x7fffffff);
        G += g;
        K += k;
        if (k > 0) {
            if (K > have) state[b] = SPEC_STATUS_NO_PAGES;
            else mine = (int)K;
        }
    }
    if (mine > 0) atomicMax(&served, mine);
    if (tid == 0) given[p.B] = (int)all_given;
    __syncthreads();
    const int all = served, moved = (int)all_given;
    const int64_t base = have - all;
    if (tid == 0) taken[p.B] = all;
    const int first = rank * NT + tid, step = ctas * NT;
    for (int b = first; b <= p.B; b += step) {
        p.cu[b] = cu[b];
        if (b < p.B) {
            p.status[b] = state[b];
            p.seq_len[b] = state[b] == SPEC_STATUS_OK ? p.keep[b] + p.fresh[b] : p.keep[b];
        }
    }

    // ---- pages change hands
    auto enter = [&](int j, int id) {  // taken page j
        const int b = last_at_most(taken, p.B, j);
        p.table[(int64_t)b * p.width + p.held[b] + (j - taken[b])] = id;
    };
    for (int64_t j = first; j < moved; j += step) {
        const int k = (int)j, b = last_at_most(given, p.B, k);
        const int need = (int)(((int64_t)p.keep[b] + p.fresh[b] + p.page_size - 1) >> p.shift);
        int32_t *entry = p.table + (int64_t)b * p.width + need + (k - given[b]);
        const int id = *entry;
        *entry = -1;
        const int64_t place = (int64_t)count + k;
        if (place >= base) enter((int)(place - base), id);
        else if (place < p.num_pages) p.free[place] = id;
    }
    for (int64_t j = first; j < min((int64_t)all, count - base); j += step) enter((int)j, p.free[base + j]);

    // ---- the tables are whole: what the requests hold, and the tokens' slots
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (rank == 0) {
        for (int b = tid; b < p.B; b += NT)
            if (state[b] == SPEC_STATUS_OK) p.held[b] = (int)(((int64_t)p.keep[b] + p.fresh[b] + p.page_size - 1) >> p.shift);
        if (tid == 0) *p.count = (int)min(base, (int64_t)p.num_pages);
    }
    if (p.rows_apart) return;
    const int lane = tid & 31;
    for (int64_t r0 = (int64_t)(first - lane) * kRowsEach; r0 < p.n_out; r0 += (int64_t)step * kRowsEach)
        place_rows(p, r0 + lane, cu, state);
}

// Many tokens: all SMs, after the tables are whole.
constexpr int kRowsThreads = 128;
__global__ void __launch_bounds__(kRowsThreads) page_rows_kernel(PlanParams p) {
    const int64_t warp = ((int64_t)blockIdx.x * kRowsThreads + threadIdx.x) >> 5;
    place_rows(p, warp * 32 * kRowsEach + (threadIdx.x & 31), p.cu, p.status);
}

template <int NT>
int launch(const PlanParams &p, int ctas, size_t smem, int dev, cudaStream_t st) {
    static std::atomic<bool> set[64];
    if (!set[dev].load()) {
        const cudaError_t e = cudaFuncSetAttribute(page_plan_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 13 * SPEC_MAX_BATCH + 64);
        if (e != cudaSuccess) {
            note_cuda_error((int)e);
            return SPEC_ECUDA;
        }
        set[dev].store(true);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, page_plan_kernel<NT>, p, ctas);
    if (e != cudaSuccess) {
        cudaGetLastError();
        note_cuda_error((int)e);
        return SPEC_ECUDA;
    }
    return launch_status();
}

}  // namespace
}  // namespace specv

using namespace specv;

extern "C" int spec_kv_plan(int32_t *free_pages, int32_t *free_count, int num_pages, int page_size, int32_t *page_table,
                            int ld_table, int32_t *held, int B, const int32_t *keep_len, const int32_t *new_len,
                            int n_out, int32_t *out_cu, int32_t *out_seq_len, int64_t *out_slot,
                            int32_t *out_position, int32_t *out_status, void *cuda_stream) {
    if (B < 0 || n_out < 0 || ld_table < 0 || num_pages <= 0) return SPEC_EINVAL;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return SPEC_EUNSUPPORTED;
    if (B > SPEC_MAX_BATCH || (int64_t)B * ld_table > 0x7fffffff) return SPEC_EUNSUPPORTED;
    if (!free_pages || !free_count || !out_cu || (n_out > 0 && (!out_slot || !out_position))) return SPEC_EINVAL;
    if (B > 0 && (!held || !keep_len || !new_len || !out_seq_len || !out_status || (ld_table > 0 && !page_table)))
        return SPEC_EINVAL;
    if (((uintptr_t)free_pages | (uintptr_t)free_count | (uintptr_t)page_table | (uintptr_t)held | (uintptr_t)keep_len |
         (uintptr_t)new_len | (uintptr_t)out_cu | (uintptr_t)out_seq_len | (uintptr_t)out_position | (uintptr_t)out_status) & 3)
        return SPEC_EINVAL;
    if ((uintptr_t)out_slot & 7) return SPEC_EINVAL;
    // What is written must overlap nothing else: threads still read the lengths when others write.
    const size_t rows = 4 * (size_t)B;
    const struct {
        const void *p;
        size_t bytes;
    } used[] = {{free_pages, 4 * (size_t)num_pages}, {free_count, 4}, {page_table, rows * ld_table}, {held, rows},
                {out_cu, rows + 4}, {out_seq_len, rows}, {out_slot, 8 * (size_t)n_out}, {out_position, 4 * (size_t)n_out},
                {out_status, rows}, {keep_len, rows}, {new_len, rows}};
    for (int i = 0; i < 9; ++i)
        for (int j = i + 1; j < 11; ++j)
            if (overlap(used[i].p, used[i].bytes, used[j].p, used[j].bytes)) return SPEC_EINVAL;
    int dev = 0, sms = 0, rc;
    if ((rc = kv_device_info(&dev, &sms))) return rc;
    if ((rc = kv_check_device_pointer(free_pages, dev))) return rc;
    PlanParams p = {};
    p.free = free_pages;
    p.count = free_count;
    p.table = page_table;
    p.held = held;
    p.keep = keep_len;
    p.fresh = new_len;
    p.cu = out_cu;
    p.seq_len = out_seq_len;
    p.position = out_position;
    p.status = out_status;
    p.slot = out_slot;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.shift = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
    p.B = B;
    p.width = ld_table;
    p.n_out = n_out;
    const size_t smem = (size_t)3 * 4 * (B + 1) + B;
    const cudaStream_t st = (cudaStream_t)cuda_stream;
    // one CTA while few tokens are to be placed and few pages can move
    if (B <= 256 && n_out <= 2048 && (int64_t)B * ld_table <= 32768) return launch<256>(p, 1, smem, dev, st);
    // Two calls for 4096 requests, 110000 and 750000 tokens: 60 us with the rows in the cluster's
    // own CTAs (16 of them), 44 apart; 47 with clusters of 8, the portable size.
    p.rows_apart = n_out > 16384;
    rc = launch<1024>(p, B <= 1024 ? 4 : 8, smem, dev, st);
    if (rc || !p.rows_apart) return rc;
    constexpr int each = kRowsThreads * kRowsEach;
    page_rows_kernel<<<(unsigned)(((int64_t)n_out + each - 1) / each), kRowsThreads, 0, st>>>(p);
    return launch_status();
}
