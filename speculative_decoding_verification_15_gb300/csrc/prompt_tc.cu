// prompt_tc.cu -- prompt attention on the tensor cores (bf16).
//
// An item is a key head's two row tiles of up to 128 rows (queries of consecutive tokens,
// the group's heads of each) and the tiles of 128 keys that one of them sees.  For each key
// tile and row tile
//   S = Q K^T     operands in shared memory, fp32 in tensor memory,
//   P = 2^(S - m) rounded to bf16, by 128 threads, a row each, back into S's columns,
//   O += P V      P from tensor memory, V from shared memory, fp32 in tensor memory.
// The two row tiles take turns: while one's exponentials are computed the tensor cores work
// for the other.  The reference m of a row moves only when a log2 score exceeds it by more
// than 8 (weights stay below 2^8 and keep their relative precision, sums included), so O is
// rarely rescaled.
//
// P's rounding to bf16 (2^-8 of each weight at most) is of the size of the output's own; it
// lets both products run at the bf16 rate.  Everything else is fp32.  P in two terms takes half as
// many products again: 24 packed prompts 599 -> 860 us, one of 24571 tokens 1476 -> 2158, for outputs
// that are off by 0.0016 (relative 2-norm) instead of 0.0021.
//
// Roles: 8 warps of softmax (4 a row tile), one that issues products, one that copies
// (tensor maps: queries {D, group, heads, tokens}, keys and values {D, heads, tokens}, in
// panels of 64 columns, zeros past D), one that finds the items, one that watches the others.
//
// Order.  CTAs stay, and items go to them longest first, forth and back (CTA c takes numbers
// c, 2 n - 1 - c, 2 n + c, ..): costs fall along the order, so the sums are nearly equal
// without a counter.  Where the host sees fewer items than SMs over many keys, items are cut
// along the keys into parts of equal length, whose sums prompt_join_kernel joins in order.
//
// Bound by the chain scores, maximum, exponentials, weights of two warps a scheduler (1720
// TFLOP/s on one prompt of 16384 tokens with 16 heads of 128 columns, 990 on 8 prompts of 4500
// with 16 heads of 64 that share 4 key heads), and with short items by their starts and ends (some
// 3 us a pair of row tiles); long calls by power (clocks of 1.7 to 1.8 GHz).
//
// What a row does not see has weight 0, but 0 times a NaN or an infinity is NaN.  A CTA marks its
// items with a row that is not finite, and does them again when all are done, with care: what is
// not finite in the values of a tile that hides some key from some row is taken out of it in
// shared memory before the products.  A third round adds that to the rows that see it.  So such
// values cost their items' time again, however long their rows are (24571 tokens, 16 heads, NaN
// behind the last one: 1.7 ms; 1.4 without, 658 when rows were repaired key by key).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <type_traits>

#include "prompt_common.cuh"
#include "tcgen05.cuh"

namespace specv {
namespace {

constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kKeys = 128, kRows = 128, kPanel = 128 * 128;  // bytes of 64 columns of 128 rows
constexpr int kThreads = 384, kSoftWarps = 8;
constexpr int kMmaWarp = 8, kCopyWarp = 9, kFindWarp = 10, kWatchWarp = 11;
constexpr int kItems = 3;         // places for items that have been told and are not done with
constexpr int kMarks = 1024;      // of items to be done again, by their number modulo this
constexpr int kWorking = kThreads - 32;  // all but the watching warp
constexpr int kSortedBatch = 128; // requests whose items are put in order of length
constexpr float kRefStep = 8.f;   // log2: how far a score may exceed the reference

// What a CTA's waits go by: whether it has failed, and the pieces of tiles copied and the items told
// so far.
struct Watch {
    int failed;
    uint32_t pieces, items;
};

// Polls: these waits are on the path of every tile, so they look at no clock.  One warp watches over
// the others: two seconds without a copy or a new item, and all waits end.  (A wait may last a whole
// item, and an item of 200 million keys takes longer than that; millions of items without keys copy
// nothing.)
__device__ __forceinline__ bool try_barrier(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done != 0;
}
__device__ __forceinline__ bool poll_barrier(uint32_t bar, uint32_t parity, volatile Watch *watch) {
    for (uint32_t n = 1;; ++n) {
        if (try_barrier(bar, parity)) return true;
        if ((n & 255) == 0 && watch->failed) return false;
    }
}
// The watching warp's: done() becomes true, or fails the CTA.
template <typename F>
__device__ __forceinline__ bool watch_until(volatile Watch *watch, F done) {
    uint64_t t0 = 0;
    uint32_t before = 0;
    while (!done()) {
        const uint64_t now = global_ns();
        const uint32_t seen = watch->pieces + watch->items;  // neither falls
        if (t0 == 0 || seen != before) t0 = now;
        before = seen;
        if (watch->failed || now - t0 > kWaitNs) {
            watch->failed = 1;
            return false;
        }
    }
    return true;
}

// Key tiles of an item, as indexes into a list: tiles [0, s1) and [w0, ...).  A row tile's
// own are indexes [0, its s1) and [w, e).
struct Tiles {
    int s1, w0, count;
    struct Sub {
        int s1, w, e;
        __device__ __forceinline__ bool active(int i) const { return i < s1 || (i >= w && i < e); }
        __device__ __forceinline__ int count(int i0, int i1) const {  // of indexes i0 .. i1 - 1
            return max(0, min(s1, i1) - i0) + max(0, min(e, i1) - max(w, i0));
        }
    } sub[2];
    __device__ __forceinline__ int tile(int i) const { return i < s1 ? i : w0 + (i - s1); }
};

struct Item {
    int b;                            // -1: no more
    int row0, n, key0, off, tok0, h;  // off: position of query 0; tok0: first token of the first row tile
    int part, parts, i0, i1;          // its part of the tiles: indexes i0 .. i1 - 1
    Tiles t;
};

__device__ __forceinline__ Tiles tiles_of(const PromptParams &p, const Item &x, int tokens, int subs) {
    Tiles t;
    Span s[2];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        const int first = x.tok0 + a * tokens, end = min(x.n, first + tokens);
        s[a] = a < subs && first < end ? span_of<kKeys>(p, x.off + first, x.off + end - 1) : Span{0, 0, 0};
    }
    const bool one = s[0].count > 0, two = s[1].count > 0;
    t.w0 = one ? (two ? min(s[0].w0, s[1].w0) : s[0].w0) : s[1].w0;
    t.s1 = min(max(s[0].s1, s[1].s1), t.w0);
    t.count = 0;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        t.sub[a].s1 = s[a].s1;
        t.sub[a].w = s[a].count > 0 ? t.s1 + s[a].w0 - t.w0 : 0;
        t.sub[a].e = t.sub[a].w + s[a].count - s[a].s1;
        t.count = max(t.count, t.sub[a].e);
    }
    return t;
}

// Whether some row of the row tiles that visit tile i does not see one of its keys.
__device__ __forceinline__ bool hides(const PromptParams &p, const Item &x, int tokens, int i) {
    const int j0 = x.t.tile(i) * kKeys;
    bool some = false;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        const int first = x.tok0 + a * tokens, last = min(x.n, first + tokens) - 1;
        some |= x.t.sub[a].active(i) && (j0 + kKeys - 1 > x.off + first || (p.window > 0 && j0 <= x.off + last - p.window && j0 + kKeys > p.sinks));
    }
    return some;
}

// ------------------------------------------------------------------ the order of the items
// One warp.  A pair is an item without its head: (request, pair t of its row tiles), its
// level the tiles up to its last query.  Up to kSortedBatch requests: highest level first,
// with counts in closed form; numbers are asked for in rising order, so the level falls by a
// few steps at a time (and by bisection where it has far to go).  More requests: request
// after request, each one's last pairs first.
struct Finder {
    static constexpr int kEach = kSortedBatch / 32;
    uint32_t tokens;               // of a pair
    int n[kEach], off[kEach];      // a lane's requests
    int row0[kEach], key0[kEach];
    int before, upto;              // sorted: pairs above the current level, and down to it
    int64_t passed;                // not sorted: pairs of the requests below b0
    int64_t total;                 // pairs in all
    int each, b0, level;           // each: requests a lane really has, at most
    int parts[kEach];              // cut: of a lane's requests
    bool sorted;

    __device__ __forceinline__ int pairs_of(int n) const { return (int)(((uint32_t)n + tokens - 1) / tokens); }
    // The first pair of a request that is at least `level` tiles long (>= 1).
    __device__ __forceinline__ int first_at(int n, int off, int level) const {
        if (level <= 1) return 0;
        const int64_t x = (int64_t)(level - 1) * kKeys + 1 - off;  // tokens it takes
        if (x > n) return pairs_of(n);
        if (x <= tokens) return 0;
        return (int)(((uint32_t)x + tokens - 1) / tokens) - 1;
    }
    __device__ __forceinline__ int at_least(int level) const {
        int c = 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            if (k < each) c += pairs_of(n[k]) - first_at(n[k], off[k], level);
        return __reduce_add_sync(0xffffffffu, c);
    }
    __device__ __forceinline__ void start(const PromptParams &p, int pair_tokens, int lane) {
        tokens = pair_tokens;
        each = (p.B + 31) / 32;
        sorted = p.B <= kSortedBatch;
        b0 = before = upto = 0;
        passed = total = 0;
        int longest = 1;
        if (sorted) {
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                n[k] = off[k] = row0[k] = key0[k] = 0;
                const int b = k * 32 + lane;
                if (b < p.B) {
                    const Prompt r = load_prompt(p, b);
                    n[k] = r.n;
                    off[k] = r.m - r.n;
                    row0[k] = r.row0;
                    key0[k] = r.key0;
                    if (r.n > 0) longest = max(longest, (r.m + kKeys - 1) / kKeys);
                    total += pairs_of(r.n);
                }
            }
        } else {
            for (int b = lane; b < p.B; b += 32) total += pairs_of(load_prompt(p, b).n);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        sorted = sorted && total < 1 << 30;  // more only where offsets overlap
        level = __reduce_max_sync(0xffffffffu, longest) + 1;
    }
    // Items in parts (few requests, p.parts > 1): request after request; in each, head by head
    // and part by part all pairs, which read the same keys at the same time.  Every part is of
    // about `unit` tiles, so that all cost alike: the unit is the one of six whose rounds over
    // the CTAs take least.  Returns the number of items.
    __device__ __forceinline__ int64_t cut(const PromptParams &p, int ctas) {
        constexpr int kFixed = 6;  // tiles that an item's start and end cost
        int tiles[kEach];
        int64_t all = 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int first = (pairs_of(n[k]) - 1) * (int)tokens;  // of the last pair
            tiles[k] = n[k] > 0 ? max(1, span_of<kKeys>(p, off[k] + first, off[k] + n[k] - 1).count) : 0;
            all += (int64_t)pairs_of(n[k]) * tiles[k];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        static_assert(kEach == 4, "tiles of a lane's requests");
        const int longest = __reduce_max_sync(0xffffffffu, max(max(tiles[0], tiles[1]), max(tiles[2], tiles[3])));
        int64_t least = 0, count = 0;
        int unit = 0;
        for (int rounds = 1; rounds <= 6; ++rounds) {
            const int64_t fair = (all * p.H + (int64_t)rounds * ctas - 1) / ((int64_t)rounds * ctas);
            const int u = (int)max(max(fair, (int64_t)4), (int64_t)(longest + p.parts - 1) / p.parts);
            int64_t items = 0;
#pragma unroll
            for (int k = 0; k < kEach; ++k) items += (int64_t)pairs_of(n[k]) * ((tiles[k] + u - 1) / u);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) items += __shfl_xor_sync(0xffffffffu, items, o);
            items *= p.H;
            const int64_t time = (items + ctas - 1) / ctas * (u + kFixed);
            if (unit == 0 || time < least) {
                least = time;
                unit = u;
                count = items;
            }
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) parts[k] = (tiles[k] + unit - 1) / unit;
        return count;
    }
    // Item i of these (i below their number).
    __device__ __forceinline__ Item find_part(const PromptParams &p, int64_t i, int lane) {
        Item x;
        x.b = -1;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if (k >= each || x.b >= 0) continue;
            const int pairs = pairs_of(n[k]);
            const int64_t mine = (int64_t)pairs * parts[k] * p.H;
            int64_t s = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += y;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, s > i);
            if (past) {
                const int w = __ffs(past) - 1;
                const int64_t rest = i - __shfl_sync(0xffffffffu, s - mine, w);
                const int np = __shfl_sync(0xffffffffu, pairs, w), nparts = __shfl_sync(0xffffffffu, parts[k], w);
                const int which = (int)(rest / np);
                x.b = k * 32 + w;
                x.tok0 = (np - 1 - (int)(rest - (int64_t)which * np)) * (int)tokens;
                x.h = which / nparts;
                x.part = which - x.h * nparts;
                x.parts = nparts;
                x.row0 = __shfl_sync(0xffffffffu, row0[k], w);
                x.n = __shfl_sync(0xffffffffu, n[k], w);
                x.key0 = __shfl_sync(0xffffffffu, key0[k], w);
                x.off = __shfl_sync(0xffffffffu, off[k], w);
            } else {
                i -= __shfl_sync(0xffffffffu, s, 31);
            }
        }
        return x;
    }
    // Pair number r of the order (r < total, rising from call to call).
    __device__ __forceinline__ Item find(const PromptParams &p, int64_t r, int lane) {
        Item x;
        x.b = -1;
        if (sorted) {
            for (int steps = 0; upto <= r && steps < 4; ++steps) {
                before = upto;
                upto = at_least(--level);
            }
            if (upto <= r) {
                int lo = 1, hi = level;  // at_least(lo) > r >= at_least(hi)
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (at_least(mid) > r) lo = mid;
                    else hi = mid;
                }
                level = lo;
                before = at_least(lo + 1);
                upto = at_least(lo);
            }
            int rest = (int)r - before;
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                if (k >= each || x.b >= 0) continue;
                const int t0 = first_at(n[k], off[k], level), mine = first_at(n[k], off[k], level + 1) - t0;
                int s = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, s, o);
                    if (lane >= o) s += y;
                }
                const uint32_t past = __ballot_sync(0xffffffffu, s > rest);
                if (past) {
                    const int w = __ffs(past) - 1;
                    x.b = k * 32 + w;
                    x.tok0 = __shfl_sync(0xffffffffu, t0 + rest - (s - mine), w) * (int)tokens;
                    x.row0 = __shfl_sync(0xffffffffu, row0[k], w);
                    x.n = __shfl_sync(0xffffffffu, n[k], w);
                    x.key0 = __shfl_sync(0xffffffffu, key0[k], w);
                    x.off = __shfl_sync(0xffffffffu, off[k], w);
                } else {
                    rest -= __shfl_sync(0xffffffffu, s, 31);
                }
            }
            return x;
        }
        for (;;) {
            Prompt q = {0, 0, 0, 0, false};
            if (b0 + lane < p.B) q = load_prompt(p, b0 + lane);
            const int mine = pairs_of(q.n);
            int64_t s = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += y;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, passed + s > r);
            if (past || b0 >= p.B) {
                const int w = past ? __ffs(past) - 1 : 0;
                if (past) x.b = b0 + w;
                const int64_t start = passed + __shfl_sync(0xffffffffu, s - mine, w);
                x.tok0 = (__shfl_sync(0xffffffffu, mine, w) - 1 - (int)(r - start)) * (int)tokens;
                x.row0 = __shfl_sync(0xffffffffu, q.row0, w);
                x.n = __shfl_sync(0xffffffffu, q.n, w);
                x.key0 = __shfl_sync(0xffffffffu, q.key0, w);
                x.off = __shfl_sync(0xffffffffu, q.m - q.n, w);
                return x;
            }
            passed += __shfl_sync(0xffffffffu, s, 31);
            b0 += 32;
        }
    }
};

// ------------------------------------------------------------------ shared memory
// Heads of up to 128 columns (NP panels of 64): two row tiles, whose S and O fill tensor
// memory; a ring of tiles K0 V0 K1 V1 ..  (Up to 64 columns P
// would have room beside S and the next S could be computed while the last weights are: 378 us
// instead of 363 on 8 prompts of 4500 tokens, 16 heads.)  Wider heads: O takes half of tensor memory, so one
// row tile with two buffers of S, and the next tile's S is computed during the exponentials;
// the ring holds halves of tiles (64 keys) in the order K0 K1 V0 K2 V1 ..
template <int NP>
struct PromptShared {
    static constexpr bool kWide = NP > 2;
    static constexpr int kSubs = kWide ? 1 : 2;
    static constexpr int kRingKeys = kWide ? 64 : 128, kPieces = kKeys / kRingKeys;
    static constexpr int kRingPanel = kRingKeys * 128, kRingBytes = NP * kRingPanel;
    static constexpr int kStages = NP == 1 ? 10 : NP == 3 ? 7 : 5;
    uint8_t q[kSubs][NP * kPanel];
    uint8_t ring[kStages][kRingBytes];
    uint64_t full[kStages], empty[kStages], q_full, q_empty, s_full[2], p_full[2][2], o_full[2], drain;
    uint64_t item_full[kItems], item_empty[kItems], finished, raw;
    Item items[kItems];
    uint32_t redo[kMarks / 32], redo_any;  // items to be done again
    uint32_t tmem;
    Watch watch;
};

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The n lowest bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t bits_below(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1; }

__device__ __forceinline__ void store_v8(void *dst, const uint32_t *w) {  // 32-byte aligned
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Which of keys j0 .. j0 + 31 have values that are not finite, a bit each, and in `all` those that
// have nothing but NaN (one warp, a key a lane).
__device__ __forceinline__ uint32_t strange_keys(const PromptParams &p, const Item &x, int j0, int lane, uint32_t *all) {
    const int key = x.key0 + j0 + lane;
    bool some = false, only = true;
    if (key < p.n_k) {
        const uint4 *v = (const uint4 *)((const uint16_t *)p.v + (int64_t)key * p.ld_v + (int64_t)x.h * p.D);
#pragma unroll 2
        for (int c = 0; c < p.D / 8; ++c) {
            const uint4 y = v[c];
            const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                some |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
                only &= (w[e] & 0x7fffu) > 0x7f80u && (w[e] & 0x7fffffffu) >= 0x7f810000u;
            }
        }
    }
    *all = __ballot_sync(0xffffffffu, some && only);
    return __ballot_sync(0xffffffffu, some);
}

// Values of KEYS keys in `panels` panels: what is not finite becomes 0 (one warp).
template <int KEYS>
__device__ __forceinline__ void take_out(uint8_t *values, int panels, int lane) {
#pragma unroll 1
    for (int w = lane; w < panels * KEYS * 32; w += 32) {
        uint32_t *two = (uint32_t *)values + w;
        const uint32_t x = *two, lo = (x & 0x7f80u) == 0x7f80u ? 0u : 0xffffu, hi = (x & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u;
        if ((lo | hi) != 0xffffffffu) *two = x & (lo | hi);
    }
    fence_async_shared();  // the products read them next
}

// What was taken out of an item's tiles, added to the rows that see it, which have been written (a
// warp's 32 rows, a lane each, at position pos, -1 for rows that do not count; a weight is
// positive, so an infinity times it is that infinity).
__device__ __forceinline__ void put_back(const PromptParams &p, const Item &x, int tokens, const Tiles::Sub &sub, int pos, int lane,
                                         int64_t row) {
    const int64_t slot = ((int64_t)x.part * p.n_q * p.Hq + row) * p.D;
    auto add = [&](int c, float z) {
        if (p.parts > 1) {
            p.part_o[slot + c] += z;
        } else {
            uint16_t *o = (uint16_t *)p.out + row * p.D + c;
            *o = (uint16_t)pack_bf16x2(__uint_as_float((uint32_t)*o << 16) + z, 0.f);
        }
    };
    bool gone = false;  // the row is NaN throughout
#pragma unroll 1
    for (int t = x.i0 * 4; t < x.i1 * 4; ++t) {  // 32 keys at a time
        if (!hides(p, x, tokens, t >> 2) || !sub.active(t >> 2)) {
            t |= 3;
            continue;
        }
        const int j0 = x.t.tile(t >> 2) * kKeys + (t & 3) * 32;
        uint32_t all;
#pragma unroll 1
        for (uint32_t left = strange_keys(p, x, j0, lane, &all); left; left &= left - 1) {
            const int e = __ffs(left) - 1;
            const bool sees = !gone && visible(p, pos, j0 + e);
            if (!__any_sync(0xffffffffu, sees)) continue;  // also keys behind the request's last
            const bool only = all >> e & 1;
            gone |= sees && only;
            const uint16_t *v = (const uint16_t *)p.v + (int64_t)(x.key0 + j0 + e) * p.ld_v + (int64_t)x.h * p.D;
#pragma unroll 1
            for (int c = 0; c < p.D; ++c) {
                const float z = ld_elem<2>(v, c);
                if (sees && !isfinite(z)) add(c, z);
            }
        }
    }
}

__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 56;"); }
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 224;"); }

template <int NP>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_tc_kernel(const PromptParams p, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, int tokens, int subs) {
    using SM = PromptShared<NP>;
    constexpr int NS = SM::kStages;
    constexpr bool kWide = SM::kWide;
    extern __shared__ __align__(1024) uint8_t raw[];
    SM &sm = *reinterpret_cast<SM *>(raw);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 1);
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sm.s_full[a], 1);
            mbar_init(&sm.p_full[a][0], 4);
            mbar_init(&sm.p_full[a][1], 4);
            mbar_init(&sm.o_full[a], 1);
        }
        mbar_init(&sm.drain, 1);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sm.item_full[i], 1);
            mbar_init(&sm.item_empty[i], 2 + kSoftWarps);
        }
        mbar_init(&sm.finished, kThreads / 32 - 1);
        mbar_init(&sm.raw, 1);
        sm.redo_any = 0;
        sm.watch.failed = 0;
        sm.watch.pieces = sm.watch.items = 0;
        mbar_init_fence();
    }
    if (tid < kMarks / 32) sm.redo[tid] = 0;
    if (warp == kMmaWarp) tmem_alloc(&sm.tmem, 512);
    tc_fence_before();
    // Statuses: the first CTA's alone, at its start.  One that fails overwrites them seconds after its
    // own start, which is not before the first one's; a late one of the others writes none.
    if (blockIdx.x == 0) write_prompt_statuses(p, tid, kThreads);
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sm.tmem;  // S of the two row tiles (or its two buffers) at 0 and 128, O from 256
    bool dead = false;            // a wait ran out: end
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!dead && !try_barrier(smem_addr(bar), parity)) dead = !poll_barrier(smem_addr(bar), parity, &sm.watch);
        dead = __any_sync(0xffffffffu, dead);
    };
    int told = 0;  // items taken
    auto take = [&](Item &x) {
        const int at = told % kItems;
        wait(&sm.item_full[at], (told / kItems) & 1);
        x = sm.items[at];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.item_empty[at]);
        ++told;
        return !dead && x.b >= 0;
    };
    // Every working warp's items are done.  Whether there is a second round, of the marked items with
    // care, and a third, in which what was taken out of their tiles is put back.  (What one warp
    // alone knows, that it ended early, all learn at the barrier.)
    int round = 0;
    auto another_round = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.finished);
        uint32_t ended;
        asm volatile(
            "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
            : "=r"(ended)
            : "r"(dead ? 1u : 0u), "n"(kWorking)
            : "memory");
        tc_fence_after();
        if (__builtin_expect(ended || round == 2 || !((volatile uint32_t &)sm.redo_any), 1)) return false;
        ++round;
        return true;
    };

    // Softmax rows live in registers: 256 threads x 224 + 128 x 56 is what 384 were launched with
    // (8 prompts of 4500 tokens, 16 heads of 64: 345 us; 350 with 216 and 72, 356 with 208 and 88).
    if (warp == kFindWarp) {
        // ---------------------------------------------------------------- items
        fewer_registers();
        do {
            Finder f;
            f.start(p, tokens * subs, lane);
            const bool cut = p.parts > 1;
            const int64_t total = cut ? f.cut(p, gridDim.x) : f.total * p.H;
            uint32_t number = 0;
            for (int64_t turn = 0;; ++turn) {
                const int64_t i = turn * gridDim.x + ((turn & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
                const bool last = turn * gridDim.x >= total;
                if (i >= total && !last) continue;
                if (__builtin_expect(round > 0 && !last, 0)) {
                    const uint32_t at = number++ % kMarks;
                    if (!(((volatile uint32_t *)sm.redo)[at / 32] >> (at % 32) & 1)) continue;
                }
                Item x;
                x.b = -1;
                if (!last) {
                    if (cut) {
                        x = f.find_part(p, i, lane);
                    } else {
                        const int64_t r = i / p.H;
                        x = f.find(p, r, lane);
                        x.h = (int)(i - r * p.H);
                        x.part = 0;
                        x.parts = 1;
                    }
                    x.t = tiles_of(p, x, tokens, subs);
                    x.i0 = (int)((int64_t)x.t.count * x.part / x.parts);
                    x.i1 = (int)((int64_t)x.t.count * (x.part + 1) / x.parts);
                }
                const int at = told % kItems;
                if (told >= kItems) wait(&sm.item_empty[at], (told / kItems - 1) & 1);
                if (dead) break;
                if (lane == 0) {
                    ((volatile Watch *)&sm.watch)->items = told + 1;
                    sm.items[at] = x;
                    mbar_arrive(&sm.item_full[at]);
                }
                ++told;
                if (last) break;
            }
        } while (another_round());
    } else if (warp == kCopyWarp) {
        // ---------------------------------------------------------------- copies
        fewer_registers();
        int sent = 0, nq = 0, raws = 0;
        auto copy_items = [&](auto careful) {
            Item x;
            while (take(x)) {
                const Tiles &t = x.t;
                if (x.i0 >= x.i1 || (careful && round == 2)) continue;
                auto copy_tile = [&](bool values, int i) {
                    const int key = x.key0 + t.tile(i) * kKeys;
                    const bool care = careful && values && hides(p, x, tokens, i);
                    for (int part = 0; part < SM::kPieces; ++part) {
                        const int slot = sent % NS;
                        if (sent >= NS) wait(&sm.empty[slot], (sent / NS - 1) & 1);
                        if (dead) return;
                        if (elect_one()) {
                            ((volatile Watch *)&sm.watch)->pieces = sent + 1;
                            uint64_t *bar = care ? &sm.raw : &sm.full[slot];
                            mbar_arrive_expect_tx(bar, SM::kRingBytes);
                            for (int c = 0; c < NP; ++c)
                                tma_load_3d(sm.ring[slot] + c * SM::kRingPanel, values ? &vmap : &kmap, 64 * c, x.h,
                                            key + part * SM::kRingKeys, bar);
                        }
                        __syncwarp();
                        ++sent;
                        if (care) {
                            wait(&sm.raw, raws++ & 1);
                            if (!dead) take_out<SM::kRingKeys>(sm.ring[slot], NP, lane);
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sm.full[slot]);
                        }
                    }
                };
                copy_tile(false, x.i0);  // the ring is free before the last item's queries are
                if (dead) break;
                if (nq > 0) wait(&sm.q_empty, (nq - 1) & 1);
                if (dead) break;
                if (elect_one()) {
                    const uint32_t bytes = (uint32_t)tokens * p.group * 128 * NP;
                    const bool one = t.sub[0].count(x.i0, x.i1) > 0, two = t.sub[1].count(x.i0, x.i1) > 0;  // wide: no second one
                    mbar_arrive_expect_tx(&sm.q_full, (one ? bytes : 0) + (two ? bytes : 0));
#pragma unroll
                    for (int a = 0; a < SM::kSubs; ++a)
                        if (a == 0 ? one : two)
                            for (int c = 0; c < NP; ++c)
                                tma_load_4d(sm.q[a] + c * kPanel, &qmap, 64 * c, 0, x.h, x.row0 + x.tok0 + a * tokens, &sm.q_full);
                }
                __syncwarp();
                ++nq;
                for (int i = x.i0; i < x.i1 && !dead; ++i) {
                    if (!kWide && i > x.i0) copy_tile(false, i);
                    if (kWide && i + 1 < x.i1) copy_tile(false, i + 1);
                    if (!dead) copy_tile(true, i);
                }
            }
        };
        do {
            if (round == 0) copy_items(std::false_type());
            else copy_items(std::true_type());
            // none of the copies may be in flight when the CTA ends
            for (int i = max(0, sent - NS); i < sent; ++i) mbar_wait(&sm.full[i % NS], (i / NS) & 1, kWaitNs);
            if (nq > 0) mbar_wait(&sm.q_full, (nq - 1) & 1, kWaitNs);
            if (raws > 0) mbar_wait(&sm.raw, (raws - 1) & 1, kWaitNs);
        } while (another_round());
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------- products
        fewer_registers();
        const uint32_t idesc_s = bf16_idesc(SM::kRingKeys, false), idesc_o = bf16_idesc(p.D, true);
        const uint64_t dq = smem_desc(smem_addr(sm.q), 16, 1024, 2), dk = smem_desc(smem_addr(sm.ring), 16, 1024, 2);
        const uint64_t dv = smem_desc(smem_addr(sm.ring), SM::kRingPanel, 1024, 2);
        const int steps = p.D / 16;
        int got = 0, nq = 0, np[2] = {0, 0};  // ring slots, query tiles, tiles of weights used
        do {
            Item x;
            while (take(x)) {
                const Tiles &t = x.t;
                const int i0 = x.i0, i1 = x.i1;
                if (i0 >= i1 || round == 2) continue;
                int done[2] = {0, 0};
                wait(&sm.q_full, nq & 1);
                ++nq;
                if constexpr (kWide) {
                    for (int i = i0 - 1; i < i1 && !dead; ++i) {
                        if (i + 1 < i1) {  // S of tile i + 1, in the buffer that the tile's number says
                            const int buf = (np[0] + (i < i0 ? 0 : 1)) & 1;
                            for (int part = 0; part < SM::kPieces && !dead; ++part, ++got) {
                                const int slot = got % NS;
                                wait(&sm.full[slot], (got / NS) & 1);
                                if (dead) break;
                                tc_fence_after();
                                if (elect_one()) {
                                    const uint64_t k = dk + (uint64_t)(slot * (SM::kRingBytes >> 4));
#pragma unroll
                                    for (int s = 0; s < NP * 4; ++s)
                                        if (s < steps)
                                            mma_bf16(tm + buf * 128 + part * SM::kRingKeys, dq + (s >> 2) * (kPanel >> 4) + (s & 3) * 2,
                                                     k + (s >> 2) * (SM::kRingPanel >> 4) + (s & 3) * 2, idesc_s, s > 0);
                                    mma_commit(&sm.empty[slot]);
                                    if (part + 1 == SM::kPieces) mma_commit(&sm.s_full[buf]);
                                    if (part + 1 == SM::kPieces && i + 2 == i1) mma_commit(&sm.q_empty);
                                }
                                __syncwarp();
                            }
                        }
                        if (i < i0) continue;
                        for (int part = 0; part < SM::kPieces && !dead; ++part, ++got) {
                            const int slot = got % NS;
                            wait(&sm.full[slot], (got / NS) & 1);
                            wait(&sm.p_full[np[0] & 1][part], (np[0] >> 1) & 1);
                            if (dead) break;
                            tc_fence_after();
                            if (elect_one()) {
                                const uint64_t v = dv + (uint64_t)(slot * (SM::kRingBytes >> 4));
#pragma unroll
                                for (int k = 0; k < SM::kRingKeys / 16; ++k)
                                    mma_bf16_ta(tm + 256, tm + (np[0] & 1) * 128 + part * (SM::kRingKeys / 2) + k * 8, v + k * 128, idesc_o,
                                                i > i0 || part > 0 || k > 0);
                                mma_commit(&sm.empty[slot]);
                                if (part + 1 == SM::kPieces) mma_commit(&sm.o_full[0]);
                            }
                            __syncwarp();
                        }
                        ++np[0];
                    }
                } else {
                    for (int i = i0 - 1; i < i1 && !dead; ++i) {
                        // the ring holds K0 V0 K1 V1 ..: tile i's values, then tile i + 1's keys
                        const int sv = got + 2 * (i - i0) + 1, sk = got + 2 * (i - i0) + 2;
                        if (i >= i0) wait(&sm.full[sv % NS], (sv / NS) & 1);
                        tc_fence_after();
#pragma unroll
                        for (int a = 0; a < 2; ++a) {
                            const uint32_t tS = tm + a * 128, tO = tm + 256 + a * 128;
                            const bool now = i >= i0 && t.sub[a].active(i), next = i + 1 < i1 && t.sub[a].active(i + 1);
                            auto scores = [&] {  // of tile i + 1
                                wait(&sm.full[sk % NS], (sk / NS) & 1);
                                if (dead) return;
                                tc_fence_after();
                                if (elect_one()) {
                                    const uint64_t q = dq + (uint64_t)(a * (NP * kPanel >> 4)), k = dk + (uint64_t)((sk % NS) * (SM::kRingBytes >> 4));
#pragma unroll
                                    for (int s = 0; s < NP * 4; ++s)
                                        if (s < steps) {
                                            const uint64_t at = (s >> 2) * (kPanel >> 4) + (s & 3) * 2;
                                            mma_bf16(tS, q + at, k + at, idesc_s, s > 0);
                                        }
                                    mma_commit(&sm.s_full[a]);
                                }
                                __syncwarp();
                            };
#pragma unroll
                            for (int part = 0; part < 2; ++part) {
                                if (now) {
                                    wait(&sm.p_full[a][part], np[a] & 1);
                                    if (dead) break;
                                    tc_fence_after();
                                    if (elect_one()) {
                                        const uint64_t v = dv + (uint64_t)((sv % NS) * (SM::kRingBytes >> 4));
#pragma unroll
                                        for (int k = part * 4; k < part * 4 + 4; ++k)
                                            mma_bf16_ta(tO, tS + k * 8, v + k * 128, idesc_o, done[a] > 0 || k > 0);
                                        if (part > 0) mma_commit(&sm.o_full[a]);
                                    }
                                    __syncwarp();
                                }
                                if (next && part == 1) scores();
                                if (dead) break;
                            }
                            if (dead) break;
                            if (now) {
                                ++np[a];
                                ++done[a];
                            }
                        }
                        if (dead) break;
                        if (elect_one()) {
                            if (i >= i0) mma_commit(&sm.empty[sv % NS]);
                            if (i + 1 < i1) mma_commit(&sm.empty[sk % NS]);
                            if (i + 2 == i1) mma_commit(&sm.q_empty);
                        }
                        __syncwarp();
                    }
                    got += 2 * (i1 - i0);
                }
            }
            // no product may be under way when the tensor memory is freed
            if (elect_one()) mma_commit(&sm.drain);
            __syncwarp();
            mbar_wait(&sm.drain, round & 1, kWaitNs);
        } while (another_round());
    } else if (warp == kWatchWarp) {
        fewer_registers();
        for (int r = 0; r < 3; ++r) {
            const bool over = watch_until(&sm.watch, [&] { return mbar_try_wait(&sm.finished, r & 1); });
            if (!over || !(volatile uint32_t &)sm.redo_any) break;
        }
    } else if (warp < kSoftWarps) {
        // ---------------------------------------------------------------- softmax
        more_registers();
        const int a = warp >> 2, w4 = warp & 3, r = w4 * 32 + lane;
        const uint32_t lanes = (uint32_t)(w4 * 32) << 16, tO = tm + 256 + a * 128 + lanes;
        const float scale = p.scale_log2;
        const float2 scale2 = make_float2(scale, scale);
        const int tok_r = r / p.group, head_r = r - tok_r * p.group;
        const int tok_w0 = __shfl_sync(0xffffffffu, tok_r, 0), tok_w1 = __shfl_sync(0xffffffffu, tok_r, 31);
        const bool wide = ((uintptr_t)p.out & 31) == 0;
        int ns = 0;  // tiles of scores
        do {
            Item x;
            while (take(x)) {
                const int first = x.tok0 + a * tokens, have = min(tokens, x.n - first);
                if (a >= subs || have <= 0) continue;
                const int list_s1 = x.t.s1, list_step = x.t.w0 - list_s1;  // of the list of tiles
                const auto sub = a == 0 ? x.t.sub[0] : x.t.sub[1];
                const int todo = sub.count(x.i0, x.i1), token = first + tok_r;
                const bool mine = tok_r < have;  // also false for rows past the last whole token
                const int pos = mine ? x.off + token : -1;
                // positions of the warp's first and last row that counts
                const int wp0 = x.off + first + tok_w0, wp1 = x.off + first + min(have - 1, tok_w1);
                float m = kNegInf, ref = 0.f;  // the reference (log2) and what is subtracted
                float2 l[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                int done = 0;
                for (int i = x.i0; done < todo && !dead; ++i) {
                    if (!sub.active(i)) continue;
                    const int j0 = (i < list_s1 ? i : i + list_step) * kKeys;
                    const uint32_t tS = tm + (kWide ? ns & 1 : a) * 128 + lanes;
                    if (kWide) wait(&sm.s_full[ns & 1], (ns >> 1) & 1);
                    else wait(&sm.s_full[a], ns & 1);
                    ++ns;
                    if (dead) break;
                    tc_fence_after();
                    // The row's maximum over both halves; the second one is read again for its
                    // weights, so that registers hold half a row besides what is in flight.
                    const bool partly = j0 + kKeys - 1 > wp0 || (p.window > 0 && j0 <= wp1 - p.window && j0 + kKeys > p.sinks);
                    const int hi = pos - j0, lo = p.window > 0 && pos >= 0 ? pos - p.window - j0 : -1, sinks = p.sinks - j0;
                    auto mask = [&](uint32_t (&s)[64], int c0) {  // of columns c0 .., those the row does not see
#pragma unroll
                        for (int c = 0; c < 64; c += 32) {
                            const int d = c0 + c;
                            const uint32_t seen = bits_below(hi + 1 - d) & (~bits_below(lo + 1 - d) | bits_below(sinks - d));
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(seen >> e & 1)) s[c + e] = 0xff800000u;
                        }
                    };
                    // four chains: two warps a scheduler hide little of an instruction's latency
                    float tops[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
                    auto maxima = [&](const uint32_t (&s)[64]) {
#pragma unroll
                        for (int c = 0; c < 64; c += 8)
#pragma unroll
                            for (int e = 0; e < 4; ++e) tops[e] = max3(tops[e], __uint_as_float(s[c + 2 * e]), __uint_as_float(s[c + 2 * e + 1]));
                    };
                    uint32_t s[64];
                    {
                        uint32_t s2[64];
                        tmem_ld<64>(tS + 64, s2);
                        tmem_wait_ld();
                        tmem_ld<64>(tS, s);
                        if (partly) {
                            mask(s2, 64);
#pragma unroll
                            for (int c = 0; c < 64; c += 16) tmem_st16(tS + 64 + c, s2 + c);  // for the second reading
                        }
                        maxima(s2);
                    }
                    tmem_wait_ld();
                    if (partly) {
                        mask(s, 0);
                        tmem_wait_st();
                    }
                    maxima(s);
                    const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]) * scale;
                    const bool moves = top > m + kRefStep;  // also from -inf
                    if (__any_sync(0xffffffffu, moves)) {
                        const float alpha = moves && m > kNegInf ? ex2_approx(m - top) : 1.f;
                        if (moves) m = ref = top;
#pragma unroll
                        for (int e = 0; e < 2; ++e) l[e] = make_float2(l[e].x * alpha, l[e].y * alpha);
                        if (done > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                            if (kWide) {  // S was ready before the last tile's products
                                wait(&sm.o_full[0], ns & 1);
                                tc_fence_after();
                            }
                            for (int c = 0; c < p.D; c += 16) {
                                uint32_t o[16];
                                tmem_ld16(tO + c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st16(tO + c, o);
                            }
                        }
                    }
                    const float2 nref = make_float2(-ref, -ref);
                    auto weights = [&](const uint32_t *s, uint32_t at) {  // of 32 columns, into tensor memory
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float2 y = ffma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), scale2, nref);
                            y.x = ex2_approx(y.x);
                            y.y = ex2_approx(y.y);
                            l[e / 2 & 1] = fadd2(l[e / 2 & 1], y);
                            w[e / 2] = pack_bf16x2(y.x, y.y);
                        }
                        tmem_st16(at, w);
                    };
                    auto let_go = [&](int part) {  // of a half's weights, to the products
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.p_full[kWide ? (ns - 1) & 1 : a][part]);
                    };
                    uint32_t s2[64];
                    weights(s, tS);
                    tmem_ld<64>(tS + 64, s2);
                    weights(s + 32, tS + 16);
                    let_go(0);
                    tmem_wait_ld();
                    weights(s2, tS + 32);
                    weights(s2 + 32, tS + 48);
                    // wide: the next S may be there before this tile's products are, and a barrier's
                    // parity tells a phase only where the one before is known to be over
                    if (kWide && ns > 1) wait(&sm.o_full[0], ns & 1);
                    let_go(1);
                    ++done;
                }
                if (todo > 0) {
                    wait(&sm.o_full[a], (ns - 1) & 1);
                    tc_fence_after();
                }
                if (dead) break;
                const float sum = (l[0].x + l[0].y) + (l[1].x + l[1].y);
                const int64_t row = (int64_t)(x.row0 + token) * p.Hq + x.h * p.group + head_r;
                const bool whole = p.parts == 1;
                const float inv = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
                const int64_t slot = (int64_t)x.part * p.n_q * p.Hq + row;  // of a part's result
                uint16_t *dst = (uint16_t *)p.out + row * p.D;
                float *part_o = whole ? nullptr : p.part_o + slot * p.D;
                float odd4[4] = {0.f, 0.f, 0.f, 0.f};  // stay 0 while everything is finite
#pragma unroll 1
                for (int c0 = 0; c0 < p.D; c0 += 64) {
                    if (!whole && todo == 0) break;
                    uint32_t o[64];
                    if (todo > 0) {
                        tmem_ld<64>(tO + c0, o);  // columns past D are not used
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int c = 0; c < 64; c += 16) {
                        if (c0 + c >= p.D) break;
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float f = todo > 0 ? __uint_as_float(o[c + e]) * inv : 0.f, g = todo > 0 ? __uint_as_float(o[c + e + 1]) * inv : 0.f;
                            odd4[e & 2] = fmaf(f, 0.f, odd4[e & 2]);
                            odd4[(e & 2) + 1] = fmaf(g, 0.f, odd4[(e & 2) + 1]);
                            w[e / 2] = pack_bf16x2(f, g);
                        }
                        if (!mine) continue;
                        if (!whole) {
                            store_v8(part_o + c0 + c, o + c);
                            store_v8(part_o + c0 + c + 8, o + c + 8);
                        } else if (wide) {
                            store_v8(dst + c0 + c, w);
                        } else {
                            *(uint4 *)(dst + c0 + c) = make_uint4(w[0], w[1], w[2], w[3]);
                            *(uint4 *)(dst + c0 + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                }
                const float odd = (odd4[0] + odd4[1]) + (odd4[2] + odd4[3]);
                if (mine && !whole) {
                    p.part_ml[slot] = make_float2(ref, sum);
                    if (x.part == 0)  // the places that this request has no part for
                        for (int k = x.parts; k < p.parts; ++k) p.part_ml[(int64_t)k * p.n_q * p.Hq + row] = make_float2(kNegInf, 0.f);
                }
                if (mine && whole && p.lse) p.lse[row] = sum == 0.f ? kNegInf : (ref + log2f(sum)) * 0.6931471805599453f;
                tc_fence_before();
                if (__builtin_expect(__any_sync(0xffffffffu, odd != 0.f && mine && todo > 0), 0)) {
                    if (lane == 0 && round == 0) {
                        const uint32_t at = (uint32_t)(told - 1) % kMarks;
                        atomicOr(&sm.redo[at / 32], 1u << (at % 32));
                        (volatile uint32_t &)sm.redo_any = 1;
                    }
                    __syncwarp();
                }
            }
        } while (another_round() && round < 2);
        if (round == 2) {
            Item x;
            while (take(x)) {
                if (a >= subs) continue;
                const int first = x.tok0 + a * tokens, token = first + tok_r;
                const int pos = tok_r < min(tokens, x.n - first) ? x.off + token : -1;
                const int64_t row = (int64_t)(x.row0 + token) * p.Hq + x.h * p.group + head_r;
                const Tiles::Sub sub = a == 0 ? x.t.sub[0] : x.t.sub[1];
                put_back(p, x, tokens, sub, pos, lane, row);
            }
            another_round();
        }
    }
    if (warp == kMmaWarp) tmem_free(tm, 512);
    if (sm.watch.failed)
        for (int b = tid; b < p.B; b += kThreads) p.status[b] = SPEC_STATUS_INTERNAL;
}

// ------------------------------------------------------------------ parts of long items
// A row's parts joined, in order: a warp a row, 4 columns a lane.  Bound by reading them.
constexpr int kJoinThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) prompt_join_kernel(const PromptParams p) {
    const Prompt r = load_prompt(p, blockIdx.y);
    const int lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)r.n * p.Hq, all = (int64_t)p.n_q * p.Hq, step = (int64_t)gridDim.x * (kJoinThreads / 32);
    for (int64_t i = (int64_t)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5); i < rows; i += step) {
        const int64_t row = (int64_t)r.row0 * p.Hq + i;
        const float2 ml = lane < p.parts ? p.part_ml[lane * all + row] : make_float2(kNegInf, 0.f);
        const bool some = ml.y != 0.f;  // the part saw something (also NaN); without, it wrote no sums
        const uint32_t parts = __ballot_sync(0xffffffffu, some);
        const float top = warp_max_nan(some ? ml.x : kNegInf), ref = top == kNegInf ? 0.f : top;
        const float weight = some ? ex2_approx(ml.x - ref) : 0.f, sum = warp_sum(some ? weight * ml.y : 0.f);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        for (int c0 = 0; c0 < p.D; c0 += 128) {
            const int c = c0 + lane * 4;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            const float *src = p.part_o + row * p.D + c;
            for (int k0 = 0; k0 < p.parts; k0 += 4) {  // four loads at a time
                float4 y[4];
                const bool in = c < p.D;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (in && (parts >> (k0 + k) & 1)) y[k] = __ldcs((const float4 *)(src + (k0 + k) * all * p.D));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float w = __shfl_sync(0xffffffffu, weight, k0 + k);
                    if (in && (parts >> (k0 + k) & 1))
                        o = make_float4(fmaf(w, y[k].x, o.x), fmaf(w, y[k].y, o.y), fmaf(w, y[k].z, o.z), fmaf(w, y[k].w, o.w));
                }
            }
            if (c >= p.D) continue;
            T *dst = (T *)p.out + row * p.D + c;
            if (sizeof(T) == 2) *(uint2 *)dst = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
            else *(float4 *)dst = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        }
        if (p.lse && lane == 0) p.lse[row] = sum == 0.f ? kNegInf : (ref + log2f(sum)) * 0.6931471805599453f;
    }
}

// ------------------------------------------------------------------ host
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
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

bool encode(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return enc && enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box, one,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NP>
int launch(const PromptParams &p, const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap, int tokens, int subs,
           int ctas, int dev, cudaStream_t st) {
    constexpr int bytes = (int)sizeof(PromptShared<NP>);
    static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
    static std::atomic<bool> set[64];
    if (!set[dev].load()) {
        const cudaError_t e = cudaFuncSetAttribute(prompt_tc_kernel<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) {
            note_cuda_error((int)e);
            return SPEC_ECUDA;
        }
        set[dev].store(true);
    }
    prompt_tc_kernel<NP><<<ctas, kThreads, bytes, st>>>(p, qmap, kmap, vmap, tokens, subs);
    const int rc = launch_status();
    return rc || p.parts == 1 ? rc : launch_prompt_join(p, true, st);
}

}  // namespace

int launch_prompt_join(const PromptParams &p, bool bf16, cudaStream_t st) {
    const int64_t blocks = ((int64_t)p.max_query * p.Hq + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
    const dim3 grid((unsigned)(blocks < 1 ? 1 : blocks < 16384 ? blocks : 16384), p.B);
    if (bf16) prompt_join_kernel<uint16_t><<<grid, kJoinThreads, 0, st>>>(p);
    else prompt_join_kernel<float><<<grid, kJoinThreads, 0, st>>>(p);
    return launch_status();
}

int launch_prompt_tc(const PromptParams &p, int dev, int sms, cudaStream_t st) {
    if (p.D > 256 || p.group > kRows || p.n_q == 0 || p.n_k == 0) return SPEC_EUNSUPPORTED;
    const int tokens = kRows / p.group;
    const cuuint64_t head = (cuuint64_t)p.D * 2;
    const bool wide = p.D > 128;
    alignas(64) CUtensorMap qmap, kmap, vmap;
    {
        const cuuint64_t dims[4] = {(cuuint64_t)p.D, (cuuint64_t)p.group, (cuuint64_t)p.H, (cuuint64_t)p.n_q};
        const cuuint64_t strides[3] = {head, head * p.group, (cuuint64_t)p.ld_q * 2};
        const cuuint32_t box[4] = {64, (cuuint32_t)p.group, 1, (cuuint32_t)tokens};
        if (!encode(&qmap, p.q, 4, dims, strides, box)) return SPEC_EUNSUPPORTED;
    }
    for (int v = 0; v < 2; ++v) {
        const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.H, (cuuint64_t)p.n_k};
        const cuuint64_t strides[2] = {head, (cuuint64_t)(v ? p.ld_v : p.ld_k) * 2};
        const cuuint32_t box[3] = {64, 1, (cuuint32_t)(wide ? PromptShared<4>::kRingKeys : PromptShared<2>::kRingKeys)};
        if (!encode(v ? &vmap : &kmap, v ? p.v : p.k, 3, dims, strides, box)) return SPEC_EUNSUPPORTED;
    }
    const PromptPlan plan = prompt_plan(p.n_q, p.n_k, p.B, p.group, p.H, p.D, p.window, p.sinks);
    const int64_t items = plan.items * plan.parts;  // at most
    const int ctas = (int)(items < sms ? items : sms), subs = plan.subs;
    if (p.D <= 64) return launch<1>(p, qmap, kmap, vmap, tokens, subs, ctas, dev, st);
    if (p.D <= 128) return launch<2>(p, qmap, kmap, vmap, tokens, subs, ctas, dev, st);
    if (p.D <= 192) return launch<3>(p, qmap, kmap, vmap, tokens, subs, ctas, dev, st);
    return launch<4>(p, qmap, kmap, vmap, tokens, subs, ctas, dev, st);
}

}  // namespace specv
