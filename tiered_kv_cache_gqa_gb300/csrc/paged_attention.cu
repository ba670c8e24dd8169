// Attention of a step's queries over a paged cache held in 4 bits, in 8 or in 16: tkv_paged_attention.  The mathematics of a
// tile is in paged_tile.cuh; here is how the work is split and the cache brought in.
//
// Work split.  The positions of every item (sequence, KV head, tile of rows) are cut into tiles of 32 (16 with 16-bit
// pages, and with 8-bit pages of d 128: about 4 KB each).  The tiles of all items, in that order, are dealt out in equal contiguous shares to the CTAs that fit on the
// device at once, and within a CTA to its seven computing warps, whatever the lengths are.  Every CTA computes the
// deal itself, from lengths and cu_tokens.  An eighth warp, four lanes for each of the seven, walks over the pieces of
// items in their shares, looks up the pages and copies the tiles into a ring of each warp's, as far ahead as the ring has
// room, across the pieces' ends: a 4-bit or 8-bit record by one cp.async.bulk, 16-bit rows by cp.async in 16-byte pieces (a bulk
// copy a row, 256 bytes, took 110 us for 134 MB where these take 30).  A warp
// computes alone and writes an item that ends within its share as soon as it is done.  Only the last piece of every warp
// waits for the others: the CTA joins them in shared memory, and what is cut at a CTA's end goes to the
// workspace, two records a CTA, which a second kernel, started early, joins in order.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <type_traits>

#include "paged_tile.cuh"

using namespace tkv;

namespace {

constexpr int kWarps = 7, kThreads = (kWarps + 1) * 32;   // warps that compute, and one that copies
constexpr int kCombineWarps = 8;
constexpr int kMinTiles = kWarps;       // of a CTA's share: one a warp; below, joining costs more than it brings
// Up to these numbers of positions in sight a CTA takes whole items, and nothing is left to join: always; where the items
// may be as many as the SMs and the pages are of 4 bits.  One launch instead of two, but uneven shares.  Whole and cut, us, 8 KV
// heads, groups of 4:
//   4 bits, d 128: batch 1, 256 positions 6.9 and 8.1, 512 positions 8.7 and 8.3; batch 8, 512 positions 10.5 and 9.9; batch 64,
//     256 positions 11.8 and 13.7, 512 positions 16.7 and 19.7, 1,024 positions 25.2 and 26.5
//   4 bits, d 64: batch 1, 256 positions 6.2 and 7.1; batch 64, 512 positions 11.7 and 13.5, 1,024 positions 18.1 and 18.9; but
//     batch 67 of mixed lengths with a window of 700 positions 20.3 and 16.2, so not beyond 512
//   8 bits, 24/4 heads of 128, the cut ones with kItemTiles: batch 8, 256 positions 7.9 and 8.6; batch 160, 256 positions 13.0 and 14.7, 512
//     positions 22.1 and 23.4; of mixed lengths up to 256 12.3 and 11.8, up to 512 16.2 and 13.0, with two drafted tokens 26.5 and 18.6; of
//     64: 6.7 and 7.9; 9.3 and 12.2, 13.7 and 15.0; 9.8 and 10.8, 12.3 and 11.5, 19.7 and 14.5; so not beyond 256, as lengths mostly differ
//   bf16, d 128: batch 1, 64 positions 5.5 and 9.0, 256 positions 7.6 and 7.6; batch 64, 256 positions 20.0 and 20.4, 512 positions
//     33.1 and 32.3; d 64: batch 64, 256 positions 15.8 and 16.0, 512 positions 24.6 and 23.7
constexpr int kWholeShort = 256, kWholeMany = 512;
// 8 bits: what an item costs beside its tiles, in tiles: q's rows, 0.7 us, its output and the next one's begin.  The deal counts them behind an
// item's own tiles, or the short sequences of a batch would be one warp's: 16 sequences of 0 to 24,268 positions, 25/5 heads of 64, 28.8
// us with none and 21.7 with 3; 19 mixed ones of 24/8 heads, drafted tokens and a window 16.4 and 12.1; 110 of up to 575 27.3 and 18.4;
// with 1 or 6 up to 10 % more; of one length the same.
constexpr int kItemTiles = 3;
constexpr int kSpinLimit = 1 << 18;     // tries of a wait; 1.5 us each where nothing comes, so 0.4 s
constexpr double kLog2E = 1.4426950408889634;

struct PagedAttnArgs {
    tkv_paged c;
    const void* q;
    void* out;
    float* lse;
    const int32_t* cu;
    float4* part;                        // records (below): [grid][2], then [grid][kWarps]
    int32_t* status;
    int64_t rows, q_row, q_head, out_row, out_head;
    int hq, group, window, page_shift, grid, whole_items, q_fp16;
    int pad;                             // tiles that an item counts for beyond its own: what its begin and end cost
    uint32_t group_mul;                  // floor((2^32 - 1) / group)
    int give_up;                         // this computing warp of the grid behaves as if its first wait had run out; -1: none
    float scale_log2;
};

// ------------------------------------------------------------------ copies
__device__ __forceinline__ void mbar_init(uint32_t bar, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect(uint32_t bar, int bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Whether the phase of that parity has ended (the hardware may wait for it a while).
__device__ __forceinline__ bool mbar_try(uint32_t bar, int parity) {
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done;
}
// Whether it has ended by now.
__device__ __forceinline__ bool mbar_test(uint32_t bar, int parity) {
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done;
}
// Bounded: false if the phase did not end.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, int parity) {
    for (int i = 0; i < kSpinLimit; ++i)
        if (mbar_try(bar, parity)) return true;
    return false;
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, int bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives when the lane's cp.async so far are done.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// ------------------------------------------------------------------ the deal
// What sequence b brings: its queries n (-1: cu_tokens makes no sense there), the positions that exist (len) and that its last query counts from (full), where
// its tiles begin, how many an item has, and the tiles of rows.
struct Seq {
    int first_row, n, len, full, lo, units, tiles;
};

// The first position that a query at `position` sees.  In 64 bits: the position may be negative (more queries than positions)
// and the window as large as an int.
__device__ __forceinline__ int window_begin(const PagedAttnArgs& a, int position) {
    return a.window > 0 ? (int)max((int64_t)0, (int64_t)position - a.window + 1) : 0;
}

// The joining kernel calls this before its own wait.  What precedes the main kernel in the stream is done by then, as the main
// kernel lets the joining one start behind its own wait, on every SM.  Ordinary loads: the lines are there from the main
// kernel's reads (8 x 4,096 positions in bf16 30.2 us; with reads from L2 31.1).
template <int R, int TP>
__device__ __forceinline__ Seq sequence_of(const PagedAttnArgs& a, int c0, int c1, int length) {
    Seq s;
    s.full = max(0, length);
    s.first_row = c0;
    s.n = (c0 < 0 || c1 < c0 || c1 > a.rows) ? -1 : c1 - c0;
    s.len = min(s.full, a.c.max_pages << a.page_shift);
    s.lo = 0;
    if (a.window > 0) s.lo = min(s.len, window_begin(a, s.full - s.n)) & ~31;
    s.units = max(1, (s.len - s.lo + TP - 1) / TP) + a.pad;   // a row that sees nothing is written too
    s.tiles = s.n > 0 ? (int)(((int64_t)s.n * a.group + R - 1) / R) : 0;
    return s;
}

template <int R, int TP>
__device__ __forceinline__ Seq sequence(const PagedAttnArgs& a, int b) {
    return sequence_of<R, TP>(a, a.cu[b], a.cu[b + 1], a.c.lengths[b]);
}

// Tiles of a sequence.  The host has made sure that the batch's tiles are fewer than 2^31.
__device__ __forceinline__ int weight(const PagedAttnArgs& a, const Seq& s) { return s.tiles * a.c.num_kv_heads * s.units; }

// Tiles are counted in 32 bits: the host refuses a step of more than kMostTiles, and if cu_tokens counts rows more than
// once all the same, sums stay at kTooMany.  A share more than that is still below 2^31.
constexpr int kMostTiles = 2000000000, kTooMany = 2050000000;
__device__ __forceinline__ int add_up_to(int a, int b) { return (int)min((uint32_t)a + (uint32_t)b, (uint32_t)kTooMany); }

// All tiles of the batch (kTooMany: or more); *before, *own: those of the sequences before this thread's and of its own (blocks of
// ceil(batch / threads) sequences a thread).  `sums`: an int of shared memory a warp;
// `status`: raised where cu_tokens descends or leaves the rows, or null.
template <int R, int TP, int WARPS>
__device__ __forceinline__ int scan_batch(const PagedAttnArgs& a, int* sums, int* before, int* own, int32_t* status) {
    constexpr int threads = WARPS * 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.c.batch + threads - 1) / threads;
    int mine = 0;
#pragma unroll 1
    for (int b = tid * per; b < min(a.c.batch, (tid + 1) * per); ++b) {
        const Seq s = sequence<R, TP>(a, b);
        mine = add_up_to(mine, weight(a, s));
        if (s.n < 0) raise_status(status, TKV_EINVAL);
    }
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum = add_up_to(sum, x);
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    uint32_t base = 0;
    int total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        const int x = sums[w];
        base += w < warp ? (uint32_t)x : 0u;
        total = add_up_to(total, x);
    }
    *before = (int)(base + (uint32_t)(sum - mine));
    *own = mine;
    return total;
}

// Where tile u of the deal lies: its sequence, and the tiles of that sequence before it.  All threads call it with the
// same targets u0, u0 + step, .. (COUNT of them; those not below the total are left out); a barrier follows before
// `where` is read.
struct Where {
    int b, in_seq;
};

template <int R, int TP, int WARPS, int COUNT>
__device__ __forceinline__ void locate(const PagedAttnArgs& a, int u0, int step, int before, int own, Where* where) {
    const int per = (a.c.batch + WARPS * 32 - 1) / (WARPS * 32);
#pragma unroll 1
    for (int k = 0; k < COUNT; ++k) {
        const int left0 = u0 + k * step - before;
        if (left0 < 0 || left0 >= own) continue;
        int left = left0, b = threadIdx.x * per;
#pragma unroll 1
        for (; per > 1; ++b) {
            const int w = weight(a, sequence<R, TP>(a, b));
            if (left < w) break;
            left -= w;
        }
        where[k] = Where{b, left};
    }
}

__device__ __forceinline__ int share_of(const PagedAttnArgs& a, int total) {
    const int even = (int)(((uint32_t)total + a.grid - 1) / (uint32_t)a.grid);
    return max(even, a.whole_items ? 1 : kMinTiles);
}

// ------------------------------------------------------------------ shapes
// Stages of a warp's ring: two CTAs, or one, share the SM's 227 KB and 64 K registers (launch bounds below).
template <int D, int NT, int KIND>
struct Config {
    static constexpr int R = 8 * NT;
    static constexpr int ctas = (in_records(KIND) && NT == 1) ? 2 : 1;
    static constexpr int stages = KIND == kE4m3 || (KIND == kInt4 && D == 128) ? (NT == 1 ? 3 : NT == 2 ? 6 : 5)
                                  : KIND == kInt4                             ? (NT == 1 ? 5 : 10)
                                                                              : (D == 128 ? 3 : 6);
    static constexpr int queue = stages <= 6 ? 8 : 16;   // pieces: the one computed, one a stage, one not yet copied
    static constexpr int warp_ring = stages * TileOf<D, KIND>::bytes;
    static constexpr int at_once = NT == 4 ? 1 : TileOf<D, KIND>::groups;   // groups of positions, by the registers
};

// A warp's part of an item.
struct Piece {
    Rows rows;
    int begin, tiles, flags;
};
// begins within the item; reaches its end; exists; there was an earlier, cut one; a wait ran out
enum { kContinues = 1, kEnds = 2, kValid = 4, kHead = 8, kFailed = 16 };

template <int D, int NT, int KIND>
struct Shared {
    using C = Config<D, NT, KIND>;
    union {
        uint8_t ring[kWarps][C::warp_ring];
        float4 merge[kWarps][NT * (D / 16) * 32];
    };
    uint64_t full[kWarps][C::stages], empty[kWarps][C::stages], known[kWarps][C::queue];   // a tile is there, is used; a piece is known
    Piece queue[kWarps][C::queue];
    float4 ml[kWarps][C::R / 2];        // references and sums of a warp's rows, two rows each
    int sums[kWarps + 1];
    Where where[kWarps], ends[2];
    int flags[kWarps], last[kWarps];    // of each warp's last piece, and its place in the queue
    int stopped[kWarps], issued[kWarps];   // the warp takes no more tiles; tiles that were brought for it
    uint8_t bad[kWarps][C::stages][2];  // records of a stage that have no page
    uint2 q[kWarps][Query<D, NT>::words];
    // 8 bits: what a warp's last piece counts in its item's sums, two rows each; what the record of the item's end counts, and the sums
    static constexpr int weights = KIND == kE4m3 ? kWarps : 1;
    float2 weight[weights][C::R / 2], tail_weight[weights][C::R / 2];
    float4 total[weights][C::R / 2];
};

// ------------------------------------------------------------------ out
// A record of a cut item: the accumulators as the lanes hold them, float4 j of row tile nt and lane at [(nt D/16 + j) 32 +
// lane] (rows 8 nt + 2 cq and + 1, each in two channels), then m and l of two rows each, [4 nt + cq].  Everything that
// joins pieces adds float4s in this order, so that little code stands behind the tiles: it comes cold into the
// instruction cache at the very end, and with the memory busy 80 instructions took 3 us there.
template <int D, int NT>
struct Rec4 {
    static constexpr int sums = NT * (D / 16) * 32, size = sums + NT * 4;   // float4s
};

// The channels of component c of float4 j: row 2 cq + (c & 1).
template <int D, int KIND>
__device__ __forceinline__ int channel_of(int r, int j, int c) {
    return KIND == kE4m3   ? 8 * (r + 8 * (j >> 2)) + 2 * (j & 3) + (c >> 1)
           : KIND == kInt4 ? (D / 8) * r + 2 * j + (c >> 1)
                           : 16 * j + r + 8 * (c >> 1);
}

__device__ __forceinline__ uint32_t pack16(float a, float b, bool fp16) {
    return fp16 ? half2_bits(__floats2half2_rn(a, b)) : bf162_bits(__floats2bfloat162_rn(a, b));
}

// Where a row's out (and lse) lies; null: no such row.
__device__ __forceinline__ uint16_t* out_row(const PagedAttnArgs& a, const Rows& rows, int row, float** lse) {
    if (rows.row0 + row >= rows.seq_rows) return nullptr;
    const int t = query_of(rows.row0 + row, a.group, a.group_mul), head = rows.h * a.group + rows.row0 + row - t * a.group;
    if (lse) *lse = a.lse ? a.lse + (int64_t)(rows.first_row + t) * a.hq + head : nullptr;
    return reinterpret_cast<uint16_t*>(a.out) + (rows.first_row + t) * a.out_row + head * a.out_head;
}

__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718056f; }
__device__ __forceinline__ float inverse(float l, float gain) { return l == 0.0f ? 0.0f : gain / l; }   // a row that saw nothing is 0
// The same for 8-bit pages, in a few instructions: 2^-22 of l and of its logarithm, far below the 2^-11 of p.
__device__ __forceinline__ float inverse8(float l) { return l == 0.0f ? 0.0f : __fdividef(1.0f, l); }
__device__ __forceinline__ float lse8_of(float m, float l) { return l == 0.0f ? -INFINITY : (m + __log2f(l)) * 0.69314718056f; }

// float4 j of row tile nt, of rows with these m and l, to out (lse with j = 0, lane row 0).
template <int D, int KIND>
__device__ __forceinline__ void emit4(const PagedAttnArgs& a, const Rows& rows, int nt, int j, int lane, float4 x, float4 ml, float gain, bool fp16) {
    const int r = lane >> 2, row = 8 * nt + 2 * (lane & 3);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float* lse;
        uint16_t* to = out_row(a, rows, row + e, &lse);
        if (!to) continue;
        const float m = e ? ml.z : ml.x, l = e ? ml.w : ml.y, inv = inverse(l, gain);
        const uint32_t w = pack16((e ? x.y : x.x) * inv, (e ? x.w : x.z) * inv, fp16);
        if (in_records(KIND)) {
            *reinterpret_cast<uint32_t*>(to + channel_of<D, KIND>(r, j, 0)) = w;
        } else {
            to[channel_of<D, KIND>(r, j, 0)] = (uint16_t)w;
            to[channel_of<D, KIND>(r, j, 2)] = (uint16_t)(w >> 16);
        }
        if (lse && j == 0 && r == 0) *lse = lse_of(m, l);
    }
}

// (ml, x) += (ml2, x2): sums of two rows at their references.
__device__ __forceinline__ void join(float4& ml, float4& x, float4 ml2, float4 x2) {
    const float m0 = fmaxf(ml.x, ml2.x), m1 = fmaxf(ml.z, ml2.z);
    const float f0 = exp2_approx(ml.x - m0), g0 = exp2_approx(ml2.x - m0), f1 = exp2_approx(ml.z - m1), g1 = exp2_approx(ml2.z - m1);
    ml = make_float4(m0, ml.y * f0 + ml2.y * g0, m1, ml.w * f1 + ml2.w * g1);
    x = make_float4(x.x * f0 + x2.x * g0, x.y * f1 + x2.y * g1, x.z * f0 + x2.z * g0, x.w * f1 + x2.w * g1);
}

// The sums of a lane's two rows over the lanes that share them: (m, l, m, l).
template <int D, int NT>
__device__ __forceinline__ float4 reduce_sums(const Sums<D, NT>& s, int nt) {
    float l[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        l[e] = s.l[nt][e];
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
    }
    return make_float4(s.m[nt][0], l[0], s.m[nt][1], l[1]);
}

// ------------------------------------------------------------------ copying
// The eighth warp: lanes 4 w .. 4 w + 3 bring the tiles of warp w, `left` of them from `from` on.
template <int D, int NT, int KIND>
__device__ __forceinline__ void copy_tiles(const PagedAttnArgs& a, Shared<D, NT, KIND>& sh, int lane, int w, const Where& from, int left) {
    using C = Config<D, NT, KIND>;
    using T = TileOf<D, KIND>;
    constexpr int R = C::R, S = C::stages, TP = T::positions;
    const int k = lane & 3;
    const int64_t head_bytes = in_records(KIND) ? (int64_t)(a.c.page_size >> 4) * T::record : (int64_t)a.c.page_size * (4 * D);
    const int64_t page_bytes = head_bytes * a.c.num_kv_heads;
    const int in_page = a.c.page_size - 1;
    const uint32_t full0 = smem_u32(sh.full[w]), empty0 = smem_u32(sh.empty[w]), ring = smem_u32(sh.ring[w]);
    // the next piece's place
    int b = left ? from.b : 0, h = 0, row_tile = 0, unit = 0;
    Seq s{};
    // 8 bits: the next sequence is read while this one is copied, its pages once for all its heads (below)
    int next_c0 = 0, next_c1 = 0, next_length = 0;
    auto read_next = [&]() {
        if (b + 1 < a.c.batch) {
            next_c1 = a.cu[b + 2];
            next_length = a.c.lengths[b + 1];
        }
    };
    if (left) {
        const int c1 = a.cu[b + 1];
        s = sequence_of<R, TP>(a, a.cu[b], c1, a.c.lengths[b]);
        next_c0 = c1;
        if (KIND == kE4m3) read_next();
        const int item = from.in_seq / s.units;
        unit = from.in_seq - item * s.units;
        h = item / s.tiles;
        row_tile = item - h * s.tiles;
    }
    // the piece that is copied: tiles, the next one's position, where its rows see nothing, its page table, page 0 of its head
    int tiles = 0, pos = 0, end = 0, pieces = 0, page = -2;
    const int32_t* table = nullptr;
    const uint8_t* pages = nullptr;
    int st = 0, parity = 0, spins = 0, issued = 0;
    bool first = true;   // the ring's first round: nothing to wait for
    // 8 bits: the four lanes look up the pages of 64 positions at once, and those of the next 64 while these are copied: the copying
    // warp as a whole waits for what any of its lanes needs next.  Those at the beginning of a sequence serve all its items.
    constexpr bool kAhead = KIND == kE4m3;
    constexpr int kBatch = 4 / T::groups;   // tiles
    int now = -2, ahead = -2, in_batch = 0, first_now = -2, first_ahead = -2, first_of = -1;
    auto page_of = [&](int p) {
        p += k * 16;
        return p < s.len ? table[p >> a.page_shift] : -2;
    };
    auto look_up = [&]() {   // a tile may have two records, which may lie in two pages
        const int p = pos + (T::groups == 2 ? (k & 1) * 16 : 0);
        page = p < end ? table[p >> a.page_shift] : -2;
    };
    while (__any_sync(0xffffffffu, left + tiles > 0 && spins < kSpinLimit)) {
        bool moved = false;
        uint32_t tile_to = 0, tile_bar = 0;
        int tile_rows = 0;
        uint64_t tile_src = 0;
        if (kAhead) page = __shfl_sync(0xffffffffu, now, (lane & ~3) + in_batch * T::groups + (k & (T::groups - 1)));
        if (left + tiles > 0 && spins < kSpinLimit) {
            if (tiles == 0) {
                while (h >= a.c.num_kv_heads || s.tiles == 0) {   // the deal leaves tiles, so there is a next item
                    ++b;
                    if (kAhead) {
                        s = sequence_of<R, TP>(a, next_c0, next_c1, next_length);
                        next_c0 = next_c1;
                        read_next();
                    } else {
                        s = sequence<R, TP>(a, b);
                    }
                    h = 0;
                }
                Piece p;
                p.rows.h = h;
                p.rows.row0 = row_tile * R;
                p.rows.first_row = s.first_row;
                p.rows.n = s.n;
                p.rows.seq_rows = s.n * a.group;
                p.rows.len = s.len;
                p.rows.last0 = s.full - s.n;
                const int t_lo = query_of(p.rows.row0, a.group, a.group_mul);
                const int t_hi = query_of(min(p.rows.seq_rows, p.rows.row0 + R) - 1, a.group, a.group_mul);
                p.rows.all_until = min(s.len, p.rows.last0 + t_lo + 1);
                p.rows.any_until = min(s.len, p.rows.last0 + t_hi + 1);
                p.rows.all_from = window_begin(a, p.rows.last0 + t_hi);
                p.rows.any_from = window_begin(a, p.rows.last0 + t_lo);
                p.begin = s.lo + unit * TP;
                p.tiles = min(s.units - unit, left);
                p.flags = kValid | (unit ? kContinues : 0) | (unit + p.tiles == s.units ? kEnds : 0);
                if (k == 0) {
                    sh.queue[w][pieces & (C::queue - 1)] = p;
                    mbar_arrive(smem_u32(&sh.known[w][pieces & (C::queue - 1)]));
                    if (s.full > s.len) raise_status(a.status, TKV_ECAPACITY);
                }
                ++pieces;
                tiles = p.tiles;
                left -= tiles;
                pos = p.begin;
                end = p.rows.any_until;
                table = a.c.page_table + (int64_t)b * a.c.max_pages;
                pages = reinterpret_cast<const uint8_t*>(a.c.pages) + head_bytes * h;
                if (kAhead) {
                    if (pos != s.lo) {
                        now = page_of(pos);
                        ahead = page_of(pos + 64);
                    } else {
                        if (first_of != b) {
                            first_of = b;
                            first_now = page_of(pos);
                            first_ahead = page_of(pos + 64);
                        }
                        now = first_now;
                        ahead = first_ahead;
                    }
                    page = now;
                    in_batch = 0;
                } else {
                    look_up();
                }
                unit += tiles;
                if (unit == s.units) {
                    unit = 0;
                    if (++row_tile == s.tiles) {
                        row_tile = 0;
                        ++h;
                    }
                }
            }
            if (first || mbar_test(empty0 + 8 * st, parity)) {
                moved = true;
                ++issued;
                if (kAhead && pos + (T::groups == 2 ? (k & 1) * 16 : 0) >= end) page = -2;   // nothing of the sequence that a row sees
                const bool ok = page >= 0 && page < a.c.num_pages;
                const uint32_t bar = full0 + 8 * st, to = ring + st * T::bytes;
                if (!ok && page != -2) raise_status(a.status, TKV_ECAPACITY);
                if (in_records(KIND)) {
                    if (k < T::groups) {
                        sh.bad[w][st][k] = !ok;
                        if (ok) {
                            mbar_arrive_expect(bar, T::record);
                            bulk_copy(to + k * T::record, pages + page * page_bytes + (((pos + k * 16) & in_page) >> 4) * T::record, T::record, bar);
                        } else {
                            mbar_arrive(bar);
                        }
                    }
                } else {
                    if (k == 0) {
                        sh.bad[w][st][0] = !ok;
                        mbar_arrive(bar);   // with this word: the arrivals behind the copies order nothing but the copies
                    }
                    tile_to = to;
                    tile_bar = bar;
                    tile_rows = ok ? min(16, end - pos) : 0;      // those behind the end are not needed
                    tile_src = reinterpret_cast<uint64_t>(pages + (ok ? page * page_bytes : 0) + (pos & in_page) * (2 * D));
                }
                if (++st == S) {
                    st = 0;
                    if (!first) parity ^= 1;
                    first = false;
                }
                pos += TP;
                --tiles;
                if (kAhead) {
                    if (++in_batch == kBatch && tiles > 0) {
                        now = ahead;
                        ahead = page_of(pos + 64);
                        in_batch = 0;
                    }
                } else if (tiles > 0) {
                    look_up();
                }
            }
            spins = moved ? 0 : spins + 1;
            if (!moved && *(volatile int*)&sh.stopped[w]) left = tiles = 0;
        }
        uint32_t groups = __ballot_sync(0xffffffffu, moved);
        if (groups == 0) __nanosleep(32);
        if (!in_records(KIND)) {
            // the whole warp copies the tile of each of its lane groups in turn
            constexpr int CH = D / 8;   // 16-byte pieces of a row
            for (groups &= 0x11111111u; groups; groups &= groups - 1) {
                const int from_lane = __ffs(groups) - 1;
                const uint32_t to = __shfl_sync(0xffffffffu, tile_to, from_lane), bar = __shfl_sync(0xffffffffu, tile_bar, from_lane);
                const int rows = __shfl_sync(0xffffffffu, tile_rows, from_lane);
                const uint8_t* src = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, tile_src, from_lane));
                const int64_t v_off = (int64_t)a.c.page_size * (2 * D);
#pragma unroll
                for (int i = 0; i < 16 * CH / 32; ++i) {
                    const int row = (i * 32 + lane) / CH, piece = lane % CH;
                    if (row < rows) {
                        cp_async16(to + row * T::row + piece * 16, src + row * (2 * D) + piece * 16);
                        cp_async16(to + (16 + row) * T::row + piece * 16, src + v_off + row * (2 * D) + piece * 16);
                    }
                }
                cp_async_arrive(bar);
            }
        }
    }
    if (spins >= kSpinLimit) raise_status(a.status, TKV_ETIMEOUT);
    issued = max(issued, __shfl_xor_sync(0xffffffffu, issued, 1));   // of both lanes that bring records
    if (k == 0 && lane >> 2 < kWarps) sh.issued[w] = issued;
}

// ------------------------------------------------------------------ joining in a CTA, 8 bits
// The warps' last pieces lie in sh.merge and sh.ml: `leads` are those that begin an item here.  The weights of all pieces come first, a
// thread a piece's two rows: then a sum is products alone, with no exponentials between one piece and the next, and a thread
// has 8 channels of a row to write at once.  Sequences of 2,000 positions and one of 70, windows of 1,000, 9 rows a KV head of 128:
// 3.8 us for the CTA that joins seven items and 1.7 for one that joins three, where one piece after the other took 10 and 2.5.
template <int D, int NT>
__device__ __forceinline__ void join_pieces(const PagedAttnArgs& a, Shared<D, NT, kE4m3>& sh, uint32_t valid, uint32_t continues, uint32_t ends,
                                            uint32_t heads, uint32_t leads) {
    constexpr int TWOS = 4 * NT, SUMS = Rec4<D, NT>::sums, SIZE = Rec4<D, NT>::size;
    const int tid = threadIdx.x, lane = tid & 31;
    auto last_of = [&](int g) { return __ffs((leads | heads | ~valid) & (~1u << g)) - 2; };   // the last piece that follows
    auto tail_of = [&](int w1) { return (heads >> (w1 + 1)) & 1 && !((ends >> w1) & 1) ? w1 + 1 : -1; };
    auto tail_record = [&](int tail) { return a.part + ((int64_t)a.grid * 2 + (int64_t)blockIdx.x * kWarps + tail) * SIZE; };
    const float4 nothing = make_float4(kLowest, 0.0f, kLowest, 0.0f);
    if (tid < kWarps * TWOS) {
        const int g = tid / TWOS, two = tid - g * TWOS;
        if (leads >> g & 1) {
            const int w1 = last_of(g), tail = tail_of(w1);
            const float4 t = tail >= 0 ? tail_record(tail)[SUMS + two] : nothing;
            float m0 = t.x, m1 = t.z;
            for (int w = g; w <= w1; ++w) {
                m0 = fmaxf(m0, sh.ml[w][two].x);
                m1 = fmaxf(m1, sh.ml[w][two].z);
            }
            float f0 = exp2_approx(t.x - m0), f1 = exp2_approx(t.z - m1), l0 = t.y * f0, l1 = t.w * f1;
            sh.tail_weight[g][two] = make_float2(f0, f1);
            for (int w = g; w <= w1; ++w) {
                const float4 ml = sh.ml[w][two];
                f0 = exp2_approx(ml.x - m0);
                f1 = exp2_approx(ml.z - m1);
                l0 = fmaf(ml.y, f0, l0);
                l1 = fmaf(ml.w, f1, l1);
                sh.weight[w][two] = make_float2(f0, f1);
            }
            sh.total[g][two] = make_float4(m0, l0, m1, l1);
        }
    }
    __syncthreads();
    constexpr int H = D / 64, UNITS = NT * H * 32;   // of an item: 8 channels of two rows
    const int all = __popc(leads) * UNITS;
#pragma unroll 1
    for (int i = tid; i < all; i += kThreads) {
        const int q = i / UNITS, nt = (i - q * UNITS) / (H * 32), h = i / 32 % H, two = 4 * nt + (lane & 3), at = (nt * (D / 16) + 4 * h) * 32 + lane;
        const int g = (int)__fns(leads, 0, q + 1), w1 = last_of(g), tail = tail_of(w1);
        const bool begins = !((continues >> g) & 1);
        float4 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = make_float4(0, 0, 0, 0);
        auto add = [&](const float4* from, float2 f) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 y = from[at + 32 * j];
                x[j] = make_float4(fmaf(y.x, f.x, x[j].x), fmaf(y.y, f.y, x[j].y), fmaf(y.z, f.x, x[j].z), fmaf(y.w, f.y, x[j].w));
            }
        };
        if (tail >= 0) add(tail_record(tail), sh.tail_weight[g][two]);
#pragma unroll 2
        for (int w = g; w <= w1; ++w) add(sh.merge[w], sh.weight[w][two]);
        const float4 ml = sh.total[g][two];
        if (begins && (((ends >> w1) & 1) || tail >= 0)) {
            const Rows& rows = sh.queue[g][sh.last[g]].rows;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float* lse;
                uint16_t* to = out_row(a, rows, 8 * nt + 2 * (lane & 3) + e, &lse);
                if (!to) continue;
                const float l = e ? ml.w : ml.y, inv = inverse8(l);
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = pack16((e ? x[j].y : x[j].x) * inv, (e ? x[j].w : x[j].z) * inv, a.q_fp16);
                *reinterpret_cast<uint4*>(to + channel_of<D, kE4m3>(lane >> 2, 4 * h, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
                if (lse && h == 0 && lane < 4) *lse = lse8_of(e ? ml.z : ml.x, l);
            }
        } else {
            float4* record = a.part + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * SIZE;
#pragma unroll
            for (int j = 0; j < 4; ++j) record[at + 32 * j] = x[j];
            if (h == 0 && lane < 4) record[SUMS + two] = ml;
        }
    }
}

// ------------------------------------------------------------------ a wait that ran out
// Every row that this CTA (tiles u0 .. u1 of the deal) has a part in becomes NaN: items that lie in it whole at once, those cut
// at its begin or end through its two records, which the joining kernel reads whatever happened here.  Not inlined: the code
// around the tiles then stays as it is without it (32 mixed sequences to 65,536: 147.3 us, and 148.9 with it in place).
template <int D, int NT, int KIND>
__device__ __noinline__ void fail_rows(const PagedAttnArgs& a, const Where& from, int u0, int u1) {
    constexpr int R = 8 * NT, TP = TileOf<D, KIND>::positions;
    const int tid = threadIdx.x;
    if (tid < 8 * NT)
        a.part[((int64_t)blockIdx.x * 2 + tid / (4 * NT)) * Rec4<D, NT>::size + Rec4<D, NT>::sums + tid % (4 * NT)] = make_float4(kLowest, NAN, kLowest, NAN);
    int b = from.b, in_seq = from.in_seq;
    Seq s = sequence<R, TP>(a, b);
#pragma unroll 1
    for (int u = u0; u < u1;) {
        const int item = in_seq / s.units, c = in_seq - item * s.units, rest = s.units - c;
        if (c == 0 && u + rest <= u1) {
            Rows rows{};
            rows.h = item / s.tiles;
            rows.row0 = (item - rows.h * s.tiles) * R;
            rows.first_row = s.first_row;
            rows.seq_rows = s.n * a.group;
#pragma unroll 1
            for (int i = tid; i < R * (D / 8); i += kThreads) {
                float* lse;
                uint16_t* to = out_row(a, rows, i / (D / 8), &lse);
                if (!to) continue;
                reinterpret_cast<uint4*>(to)[i % (D / 8)] = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);   // in both types
                if (lse) *lse = NAN;
            }
        }
        u += rest;
        in_seq += rest;
        if (in_seq == weight(a, s)) {
            in_seq = 0;
            while (u < u1 && (s = sequence<R, TP>(a, ++b)).tiles == 0) {}   // below u1 there is a next one
        }
    }
}

// ------------------------------------------------------------------ the kernel
template <int D, int NT, int KIND>
__global__ void __launch_bounds__(kThreads, Config<D, NT, KIND>::ctas) paged_attention_kernel(const __grid_constant__ PagedAttnArgs a) {
    using C = Config<D, NT, KIND>;
    using T = TileOf<D, KIND>;
    constexpr int R = C::R, S = C::stages, TP = T::positions, TB = T::bytes;
    extern __shared__ __align__(128) uint8_t smem[];
    Shared<D, NT, KIND>& sh = *reinterpret_cast<Shared<D, NT, KIND>*>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (warp == kWarps && lane < kWarps) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&sh.full[lane][s]), in_records(KIND) ? T::groups : 33);   // the lanes that bring a tile; 16 bits: and the one that says if there is a page
            mbar_init(smem_u32(&sh.empty[lane][s]), 1);
        }
        for (int s = 0; s < C::queue; ++s) mbar_init(smem_u32(&sh.known[lane][s]), 1);
        sh.stopped[lane] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }

    wait_for_previous();
    let_next_start();   // not earlier than here: the joining kernel reads lengths and cu_tokens before its own wait

    // -------------------------------------------------------- this CTA's tiles of the deal, and each warp's
    int before, own;
    const int total = scan_batch<R, TP, kWarps + 1>(a, sh.sums, &before, &own, blockIdx.x == 0 ? a.status : nullptr);
    if (total == kTooMany) {
        if (tid == 0) raise_status(a.status, TKV_EINVAL);
        return;
    }
    const int share = share_of(a, total);
    int u0 = (int)min((int64_t)total, (int64_t)blockIdx.x * share), u1 = min(total, u0 + share);
    if (a.whole_items) {
        // both ends move up to the next item's begin
        locate<R, TP, kWarps + 1, 2>(a, u0, share, before, own, sh.ends);
        __syncthreads();
        auto up = [&](int u, const Where& w) {
            if (u >= total) return total;
            const int units = sequence<R, TP>(a, w.b).units, c = w.in_seq % units;
            return c ? u + units - c : u;
        };
        const int v0 = up(u0, sh.ends[0]);
        u1 = up(u0 + share, sh.ends[1]);
        u0 = v0;
    }
    if (u0 >= u1) return;
    const int per_warp = (u1 - u0 + kWarps - 1) / kWarps;
    locate<R, TP, kWarps + 1, kWarps>(a, u0, per_warp, before, own, sh.where);
    __syncthreads();
    auto tiles_of = [&](int w) { return max(0, min(per_warp, u1 - u0 - w * per_warp)); };

    int taken = 0;                       // pieces of this warp
    Sums<D, NT> sums;
    const bool fp16 = KIND == kFp16 || (in_records(KIND) && a.q_fp16);
    auto gain_of = [&](int h) { return KIND == kInt4 ? 16.0f * (a.c.v_gain ? a.c.v_gain[h] : 1.0f) : 1.0f; };
    if (warp == kWarps) {
        const int w = min(lane >> 2, kWarps - 1);
        copy_tiles<D, NT, KIND>(a, sh, lane, w, sh.where[w], lane >> 2 < kWarps ? tiles_of(w) : 0);
    } else {
        // ---------------------------------------------------- compute
        const uint32_t full0 = smem_u32(sh.full[warp]), empty0 = smem_u32(sh.empty[warp]);
        int left = tiles_of(warp), stage = 0, parity = 0, flags = 0;
        bool failed = left > 0 && (int)blockIdx.x * kWarps + warp == a.give_up;
#pragma unroll 1
        while (left > 0 && !failed) {
            const int place = taken & (C::queue - 1);
            failed = __any_sync(0xffffffffu, !mbar_wait(smem_u32(&sh.known[warp][place]), (taken / C::queue) & 1));
            if (failed) break;
            const Piece& piece = sh.queue[warp][place];   // stays where it is: its place is taken again much later
            ++taken;
            const int all_from = piece.rows.all_from, all_until = piece.rows.all_until, any_until = piece.rows.any_until, tiles = piece.tiles;
            Query<D, NT> q;
            q.s = sh.q[warp] + lane;
            load_query<D, NT, KIND>(reinterpret_cast<const uint16_t*>(a.q), a.q_row, a.q_head, a.q_fp16, a.group, a.group_mul, a.scale_log2,
                                    KIND == kInt4 && a.c.k_gain ? a.c.k_gain[piece.rows.h] : 1.0f, lane, piece.rows, q);
            sums.clear();
            failed = __any_sync(0xffffffffu, !mbar_wait(full0 + 8 * stage, parity));
            if (failed) break;
            int p0 = piece.begin;
#pragma unroll 1
            for (int t = 1;; ++t, p0 += TP) {
                const uint8_t* at = sh.ring[warp] + stage * TB;
                const uint32_t at_s = smem_u32(at);
                const uint32_t bad = sh.bad[warp][stage][0] | (T::groups == 2 ? sh.bad[warp][stage][1] << 1 : 0);
                if (KIND == kE4m3 && p0 >= any_until) {
                    // a tile that only counts
                } else if (!bad && p0 + TP <= all_until && p0 >= all_from) {
#pragma unroll 1
                    for (int g = 0; g < T::groups; g += C::at_once)
                        attend_tile<D, NT, KIND, C::at_once, true>(at + g * T::record, at_s, lane, p0 + 16 * g, false, piece.rows, a.group,
                                                                   a.group_mul, a.window, q, sums);
                } else {
#pragma unroll 1
                    for (int g = 0; g < T::groups; ++g)
                        attend_tile<D, NT, KIND, 1, false>(at + g * T::record, at_s, lane, p0 + 16 * g, (bad >> g) & 1, piece.rows, a.group,
                                                           a.group_mul, a.window, q, sums);
                }
                __syncwarp();   // every lane has read the slot
                if (t == tiles) break;
                if (lane == 0) mbar_arrive(empty0 + 8 * stage);
                if (++stage == S) stage = 0, parity ^= 1;
                failed = __any_sync(0xffffffffu, !mbar_wait(full0 + 8 * stage, parity));
                if (failed) break;
            }
            if (failed) break;
            left -= tiles;
            const bool cut = piece.flags & kContinues;
            if (left == 0) {
                if (cut || !(piece.flags & kEnds)) {   // the last piece, of an item that others hold parts of
                    flags |= piece.flags;
                    break;
                }
            } else {
                if (lane == 0) mbar_arrive(empty0 + 8 * stage);
                if (++stage == S) stage = 0, parity ^= 1;
            }
            // The item ends here.  If it began before this warp's share, to a record: the CTA's first for the first warp (it
            // joins the CTA before), else the warp's own.
            float4* record = a.part + (warp ? (int64_t)a.grid * 2 + (int64_t)blockIdx.x * kWarps + warp : (int64_t)blockIdx.x * 2) * Rec4<D, NT>::size;
            if (cut) flags = kHead;
            const float gain = gain_of(piece.rows.h);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float4 ml = reduce_sums<D, NT>(sums, nt);
                if (cut) {
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
                        record[(nt * (D / 16) + j) * 32 + lane] = make_float4(sums.o[nt][j][0], sums.o[nt][j][1], sums.o[nt][j][2], sums.o[nt][j][3]);
                    if (lane < 4) record[Rec4<D, NT>::sums + 4 * nt + lane] = ml;
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = lane >> 2;
                        float* lse;
                        uint16_t* to = out_row(a, piece.rows, 8 * nt + 2 * (lane & 3) + e, &lse);
                        if (!to) continue;
                        const float l = e ? ml.w : ml.y, inv = KIND == kE4m3 ? inverse8(l) : inverse(l, gain);
                        uint32_t w[D / 16];
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) w[j] = pack16(sums.o[nt][j][e] * inv, sums.o[nt][j][e + 2] * inv, fp16);
                        if (in_records(KIND)) {   // 4 bits: D / 8 channels next to one another; 8 bits: 8 in every 64
#pragma unroll
                            for (int j = 0; j < D / 16; j += 4)
                                *reinterpret_cast<uint4*>(to + channel_of<D, KIND>(r, j, 0)) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
                        } else {
#pragma unroll
                            for (int j = 0; j < D / 16; ++j) {
                                to[channel_of<D, KIND>(r, j, 0)] = (uint16_t)w[j];
                                to[channel_of<D, KIND>(r, j, 2)] = (uint16_t)(w[j] >> 16);
                            }
                        }
                        if (lse && r == 0) *lse = KIND == kE4m3 ? lse8_of(e ? ml.z : ml.x, l) : lse_of(e ? ml.z : ml.x, l);
                    }
                }
            }
        }
        if (failed) {   // a copy did not come in time
            flags = kFailed;
            if (lane == 0) {
                *(volatile int*)&sh.stopped[warp] = 1;
                raise_status(a.status, TKV_ETIMEOUT);
            }
        }
        if (lane == 0) {
            sh.flags[warp] = flags;
            sh.last[warp] = (taken - 1) & (C::queue - 1);
        }
    }

    // -------------------------------------------------------- join the warps' last pieces
    __syncthreads();   // every warp is done with its ring
    const int f = lane < kWarps ? sh.flags[lane] : 0;
    if (__any_sync(0xffffffffu, f & kFailed)) {
        // no copy may be under way when the CTA ends; the ring's last round, of which each warp's tiles have come or will
        if (warp < kWarps)
            for (int i = max(0, sh.issued[warp] - S); i < sh.issued[warp]; ++i) mbar_wait(smem_u32(&sh.full[warp][i % S]), (i / S) & 1);
        __syncthreads();
        fail_rows<D, NT, KIND>(a, sh.where[0], u0, u1);
        return;
    }
    if (taken) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float4 ml = reduce_sums<D, NT>(sums, nt);
            if (lane < 4) sh.ml[warp][4 * nt + lane] = ml;
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                sh.merge[warp][(nt * (D / 16) + j) * 32 + lane] = make_float4(sums.o[nt][j][0], sums.o[nt][j][1], sums.o[nt][j][2], sums.o[nt][j][3]);
        }
    }
    __syncthreads();
    // A warp's piece that is the first of its item here leads; the warps behind it that hold nothing else follow, and the
    // record of the one in which the item ended.
    const uint32_t valid = __ballot_sync(0xffffffffu, f & kValid), continues = __ballot_sync(0xffffffffu, f & kContinues);
    const uint32_t ends = __ballot_sync(0xffffffffu, f & kEnds), heads = __ballot_sync(0xffffffffu, f & kHead);
    const uint32_t leads = valid & ~(continues & ~1u);
    if constexpr (KIND == kE4m3) {
        join_pieces<D, NT>(a, sh, valid, continues, ends, heads, leads);
        return;
    }
    // all groups at once, each with its share of the CTA's warps
    const int groups = __popc(leads), team = groups <= 1 ? 8 : groups == 2 ? 4 : groups <= 4 ? 2 : 1;
    if (warp / team < groups) {
        const int g = (int)__fns(leads, 0, warp / team + 1);
        const int w1 = __ffs((leads | heads | ~valid) & (~1u << g)) - 2;   // the last that follows
        const int tail = (heads >> (w1 + 1)) & 1 && !((ends >> w1) & 1) ? w1 + 1 : -1;
        const bool begins = !((continues >> g) & 1), complete = begins && (((ends >> w1) & 1) || tail >= 0);
        const Rows& rows = sh.queue[g][sh.last[g]].rows;
        float4* record = a.part + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * Rec4<D, NT>::size;
        const float4* tail_record = a.part + ((int64_t)a.grid * 2 + (int64_t)blockIdx.x * kWarps + tail) * Rec4<D, NT>::size;
        const float gain = gain_of(rows.h);
#pragma unroll 1
        for (int i = warp % team * 32 + lane; i < Rec4<D, NT>::sums; i += team * 32) {
            const int two = i / (D / 16 * 32) * 4 + (i & 3);   // its two rows
            float4 ml = make_float4(kLowest, 0.0f, kLowest, 0.0f), x = make_float4(0, 0, 0, 0);
#pragma unroll 1
            for (int w = g; w <= w1 + (tail >= 0); ++w)
                join(ml, x, w <= w1 ? sh.ml[w][two] : tail_record[Rec4<D, NT>::sums + two], w <= w1 ? sh.merge[w][i] : tail_record[i]);
            if (complete) {
                emit4<D, KIND>(a, rows, i / (D / 16 * 32), i / 32 % (D / 16), lane, x, ml, gain, fp16);
            } else {
                record[i] = x;
                if (i % (D / 16 * 32) < 4) record[Rec4<D, NT>::sums + two] = ml;
            }
        }
    }
}

// ------------------------------------------------------------------ joining cut items
// CTA i takes the item that is cut at the end of share i, if it began in share i: its pieces are record 1 of CTA i and
// record 0 of the CTAs after it.  The pieces' references and sums are turned into weights first, a piece a lane and two
// rows a warp at a time; the sums of O then have no order to wait for but their own.
//
// 8 bits: where an item has more than kFewPieces, the CTAs that are cut within it share its sums: an eighth each, 32 at least, and in a CTA
// groups of threads take every so manieth piece.  The call for one sequence of 36,171 positions, 16/2 heads of 128, which is two items
// of 152 pieces: 20.5 us with one CTA an item, 12.8 like this; of 100,000, 8/1 heads, 32.7 and 16.3; of 2,512, 28/4 heads, 9.4 and 8.6.
constexpr int kFewPieces = 8, kBatchPieces = 128;
template <int D, int NT>
struct Slice {
    static constexpr int slots = Rec4<D, NT>::sums / 8 > 32 ? Rec4<D, NT>::sums / 8 : 32, count = Rec4<D, NT>::sums / slots;
    static_assert(count <= kFewPieces, "a CTA that is cut within the item for each");
};

template <int D, int NT>
__device__ __forceinline__ void join_many(const PagedAttnArgs& a, const Rows& rows, const float4* first, int pieces, int slice, bool fp16) {
    constexpr int SLOTS = Rec4<D, NT>::sums, SIZE = Rec4<D, NT>::size, WIDE = Slice<D, NT>::slots, G = kCombineWarps * 32 / WIDE, IN_FLIGHT = 8;
    static_assert(WIDE % 32 == 0 && WIDE <= 4 * D / 2 * NT && G >= 2, "whole warps, in one tile of 8 rows or several");
    constexpr int TWOS = 4 * NT;
    __shared__ float2 weight_of[kBatchPieces][TWOS];
    __shared__ float4 scale_ml[TWOS], total_ml[TWOS];
    __shared__ float4 part[kCombineWarps * 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = tid / WIDE, slot = slice * WIDE + tid % WIDE;
    auto record = [&](int i) { return first + (i ? 2 * (int64_t)i * SIZE : SIZE); };
    const int my_two = slot / (D / 16 * 32) * 4 + (tid & 3);
    float4 x = make_float4(0, 0, 0, 0);
    float4 ml_of[(TWOS + kCombineWarps - 1) / kCombineWarps];
#pragma unroll
    for (int k = 0; k < (TWOS + kCombineWarps - 1) / kCombineWarps; ++k) ml_of[k] = make_float4(kLowest, 0.0f, kLowest, 0.0f);
#pragma unroll 1
    for (int i0 = 0; i0 < pieces; i0 += kBatchPieces) {
        const int n = min(kBatchPieces, pieces - i0);
        float4 y[IN_FLIGHT];
        auto read = [&](int p) {   // pieces p + g, p + g + G, ..
#pragma unroll
            for (int q = 0; q < IN_FLIGHT; ++q) y[q] = record(i0 + min(p + q * G + g, n - 1))[slot];
        };
        read(0);
#pragma unroll
        for (int k = 0; k < (TWOS + kCombineWarps - 1) / kCombineWarps; ++k) {
            const int two = warp + k * kCombineWarps;
            if (two >= TWOS) break;
            float4 v[kBatchPieces / 32];
            float m0 = ml_of[k].x, m1 = ml_of[k].z;
#pragma unroll
            for (int q = 0; q < kBatchPieces / 32; ++q) {
                const int i = q * 32 + lane;
                v[q] = i < n ? record(i0 + i)[SLOTS + two] : make_float4(kLowest, 0.0f, kLowest, 0.0f);
            }
#pragma unroll
            for (int q = 0; q < kBatchPieces / 32; ++q) {
                m0 = fmaxf(m0, v[q].x);
                m1 = fmaxf(m1, v[q].z);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
                m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
            }
            float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
            for (int q = 0; q < kBatchPieces / 32; ++q) {
                const float w0 = exp2_approx(v[q].x - m0), w1 = exp2_approx(v[q].z - m1);
                l0 = fmaf(v[q].y, w0, l0);
                l1 = fmaf(v[q].w, w1, l1);
                weight_of[q * 32 + lane][two] = q * 32 + lane < n ? make_float2(w0, w1) : make_float2(0.0f, 0.0f);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                l0 += __shfl_xor_sync(0xffffffffu, l0, o);
                l1 += __shfl_xor_sync(0xffffffffu, l1, o);
            }
            const float f0 = exp2_approx(ml_of[k].x - m0), f1 = exp2_approx(ml_of[k].z - m1);
            ml_of[k] = make_float4(m0, ml_of[k].y * f0 + l0, m1, ml_of[k].w * f1 + l1);
            if (lane == 0) {
                scale_ml[two] = make_float4(f0, f1, 0.0f, 0.0f);
                total_ml[two] = ml_of[k];
            }
        }
        __syncthreads();
        const float4 f = scale_ml[my_two];
        x = make_float4(x.x * f.x, x.y * f.y, x.z * f.x, x.w * f.y);
#pragma unroll 1
        for (int p = 0; p < n; p += IN_FLIGHT * G) {
            if (p) read(p);
#pragma unroll
            for (int q = 0; q < IN_FLIGHT; ++q) {
                const int i = p + q * G + g;
                const float2 w = i < n ? weight_of[i][my_two] : make_float2(0.0f, 0.0f);
                x = make_float4(fmaf(y[q].x, w.x, x.x), fmaf(y[q].y, w.y, x.y), fmaf(y[q].z, w.x, x.z), fmaf(y[q].w, w.y, x.w));
            }
        }
        __syncthreads();
    }
    part[tid] = x;
    __syncthreads();
    if (g) return;
#pragma unroll
    for (int k = 1; k < G; ++k) {
        const float4 y = part[tid + k * WIDE];
        x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
    }
    emit4<D, kE4m3>(a, rows, slot / (D / 16 * 32), slot / 32 % (D / 16), lane, x, total_ml[my_two], 1.0f, fp16);
}

template <int D, int NT, int KIND>
__global__ void __launch_bounds__(kCombineWarps * 32) paged_combine_kernel(const __grid_constant__ PagedAttnArgs a, bool fp16) {
    constexpr int R = 8 * NT, TP = TileOf<D, KIND>::positions, SLOTS = Rec4<D, NT>::sums, SIZE = Rec4<D, NT>::size;
    constexpr int PER = SLOTS / (kCombineWarps * 32) > 0 ? SLOTS / (kCombineWarps * 32) : 1;   // float4s a thread
    __shared__ float2 weight_of[32][4 * NT];   // of a piece, for two rows
    __shared__ float4 scale_ml[4 * NT];        // two rows: what the sums so far are scaled by; in the end m and l
    __shared__ float4 total_ml[4 * NT];
    __shared__ int sums[kCombineWarps];
    __shared__ Where at;
    int before, own;
    const int total = scan_batch<R, TP, kCombineWarps>(a, sums, &before, &own, nullptr);
    const int share = share_of(a, total);
    const int cut = total == kTooMany ? total : (int)min((int64_t)total, (int64_t)(blockIdx.x + 1) * share);
    locate<R, TP, kCombineWarps, 1>(a, cut, 0, before, own, &at);
    __syncthreads();
    int pieces = 0, slice = 0;
    Rows rows{};
    if (cut < total) {
        const Seq s = sequence<R, TP>(a, at.b);
        const int item = at.in_seq / s.units, c = at.in_seq - item * s.units;
        const int begin = (cut - c) / share;   // the CTA in whose share it began
        if (KIND == kE4m3 && c > 0) slice = (int)blockIdx.x - begin;
        if (c > 0 && (c <= share || KIND == kE4m3)) {   // something is cut here, and it began in this share
            pieces = (cut - c + s.units - 1) / share - begin + 1;
            rows.h = item / s.tiles;
            rows.row0 = (item - rows.h * s.tiles) * R;
            rows.first_row = s.first_row;
            rows.seq_rows = s.n * a.group;
        }
    }
    // what the main kernel wrote is read after this; every CTA waits, so that the grid ends after it.  Only lengths and
    // cu_tokens were read before.
    wait_for_previous();
    if (pieces == 0) return;
    if constexpr (KIND == kE4m3) {
        if (pieces > kFewPieces) {
            if (slice < Slice<D, NT>::count) join_many<D, NT>(a, rows, a.part + (int64_t)2 * ((int)blockIdx.x - slice) * SIZE, pieces, slice, fp16);
            return;
        }
        if (slice) return;
    }
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float gain = KIND == kInt4 ? 16.0f * (a.c.v_gain ? a.c.v_gain[rows.h] : 1.0f) : 1.0f;
    const float4* first = a.part + (int64_t)2 * blockIdx.x * SIZE;
    auto record = [&](int i) { return first + (i ? 2 * i * SIZE : SIZE); };
    float4 x[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) x[k] = make_float4(0, 0, 0, 0);
    constexpr int TWOS = (4 * NT + kCombineWarps - 1) / kCombineWarps;   // a warp takes two rows, or twice two
    float4 ml_of[TWOS];
#pragma unroll
    for (int k = 0; k < TWOS; ++k) ml_of[k] = make_float4(kLowest, 0.0f, kLowest, 0.0f);
    for (int i0 = 0; i0 < pieces; i0 += 32) {
        const int n = min(32, pieces - i0);
        float4 y[PER][8];   // eight loads in flight, the first of them while the weights are worked out
        auto read = [&](int p) {
#pragma unroll
            for (int k = 0; k < PER; ++k)
#pragma unroll
                for (int q = 0; q < 8; ++q) y[k][q] = record(i0 + min(p + q, n - 1))[min(tid + k * kCombineWarps * 32, SLOTS - 1)];
        };
        read(0);
#pragma unroll
        for (int k = 0; k < TWOS; ++k) {
            const int two = warp + k * kCombineWarps;
            if (two >= 4 * NT) break;
            float4& ml = ml_of[k];
            float4 v = make_float4(kLowest, 0.0f, kLowest, 0.0f);
            if (lane < n) v = record(i0 + lane)[SLOTS + two];
            float m0 = v.x, m1 = v.z;
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
                m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
            }
            m0 = fmaxf(m0, ml.x);
            m1 = fmaxf(m1, ml.z);
            const float w0 = exp2_approx(v.x - m0), w1 = exp2_approx(v.z - m1), f0 = exp2_approx(ml.x - m0), f1 = exp2_approx(ml.z - m1);
            float l0 = v.y * w0, l1 = v.w * w1;
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                l0 += __shfl_xor_sync(0xffffffffu, l0, o);
                l1 += __shfl_xor_sync(0xffffffffu, l1, o);
            }
            ml = make_float4(m0, ml.y * f0 + l0, m1, ml.w * f1 + l1);
            weight_of[lane][two] = make_float2(w0, w1);
            if (lane == 0) {
                scale_ml[two] = make_float4(f0, f1, 0.0f, 0.0f);
                total_ml[two] = ml;
            }
        }
        __syncthreads();
#pragma unroll 1
        for (int p = 0; p < n; p += 8) {
            if (p) read(p);
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int two = min(tid + k * kCombineWarps * 32, SLOTS - 1) / (D / 16 * 32) * 4 + (tid & 3);
                if (p == 0) {
                    const float4 f = scale_ml[two];
                    x[k] = make_float4(x[k].x * f.x, x[k].y * f.y, x[k].z * f.x, x[k].w * f.y);
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) {   // behind the last piece its weight is 0
                    const float2 w = p + q < n ? weight_of[p + q][two] : make_float2(0.0f, 0.0f);
                    x[k] = make_float4(x[k].x + y[k][q].x * w.x, x[k].y + y[k][q].y * w.y, x[k].z + y[k][q].z * w.x, x[k].w + y[k][q].w * w.y);
                }
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int i = tid + k * kCombineWarps * 32;
        if (i >= SLOTS) break;
        emit4<D, KIND>(a, rows, i / (D / 16 * 32), i / 32 % (D / 16), lane, x[k], total_ml[i / (D / 16 * 32) * 4 + (i & 3)], gain, fp16);
    }
}

// ------------------------------------------------------------------ launch
// Row tiles are 8 rows, or 16 where a step brings more than 8 rows a KV head: the cache is then read and expanded once for
// twice the rows.
int row_tiles(int group, int max_new) { return (int64_t)group * max_new > 8 ? 2 : 1; }

// Tiles of 32 rows of 4-bit and 8-bit pages do that once more, but the code is long and the joining heavy: worth it from so many tiles a
// computing warp on, by the host's estimate.  30 rows a KV head, 8 x 8 heads of 64: 36.3 us with 16 rows and 37.3 with 32 at
// 8,192 positions (15 tiles a warp), 65.7 and 58.4 at 16,384, 244 and 170 at 65,536; of 128: 90.0 and 93.1 at 16,384 (31
// tiles), 163.5 and 156.2 at 32,768, 307 and 276 at 65,536.  8 bits, 24 or 32 rows, heads of 64: 22.1 and 22.7 at 4,096 (7.7), 35.2
// and 30.2 at 8,192, 117 and 75 at 32,768; of 128: 29.8 and 31.7 at 4,096, 49.5 and 46.3 at 8,192 (15), 174 and 124 at 32,768.  Measured on sequences of one length; the rule takes every
// sequence to have max_new queries, so a ragged step may get the longer code for less than it is worth.
bool rows_of_32(const PagedAttnArgs& a, int max_new, int64_t sight, int sms) {
    const int64_t rows = (int64_t)a.group * max_new;
    if (!has_records(a.c.kv_type) || rows <= 16) return false;
    const double tiles = (double)a.c.batch * a.c.num_kv_heads * ((rows + 31) / 32) * ((sight + 31) / 32);
    return tiles >= (a.c.kv_type == TKV_E4M3 ? 10.0 : a.c.head_dim == 64 ? 18.0 : 45.0) * kWarps * sms;
}

// TKV_FAULT_INJECT=wait:N: computing warp N of every attention's grid gives up at its first wait, as if a copy had not come.
// A process that starts without the variable never looks at it again.
int warp_that_gives_up() {
    static const bool injects = std::getenv("TKV_FAULT_INJECT") != nullptr;
    const char* what = injects ? std::getenv("TKV_FAULT_INJECT") : nullptr;
    return what && !std::strncmp(what, "wait:", 5) ? std::atoi(what + 5) : -1;
}

cudaError_t device_sms(int* sms, int* dev) {
    const cudaError_t e = cudaGetDevice(dev);
    return e == cudaSuccess ? cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev) : e;
}

int64_t workspace_bytes_of(const tkv_paged* c, int32_t hq, int32_t max_new, int sms) {   // the most that any variant uses: two CTAs an SM, or one with twice the rows
    return (int64_t)2 * sms * (2 + kWarps) * 8 * row_tiles(hq / c->num_kv_heads, max_new) * (c->head_dim + 4) * 4;
}

template <int D, int NT, int KIND>
cudaError_t launch(PagedAttnArgs& a, int sms, int dev, cudaStream_t st) {
    using C = Config<D, NT, KIND>;
    constexpr int smem = sizeof(Shared<D, NT, KIND>);
    static_assert(C::ctas * (smem + 1024) <= 228 * 1024, "the CTAs of an SM share its memory");
    cudaError_t e = cudaSuccess;
    a.grid = C::ctas * sms;
    // the kernel's shared-memory limit, once a device
    static std::atomic<uint64_t> ready{0};
    if (!(dev < 64 && (ready.load(std::memory_order_acquire) >> dev & 1))) {
        e = cudaFuncSetAttribute(paged_attention_kernel<D, NT, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess && dev < 64) ready.fetch_or((uint64_t)1 << dev, std::memory_order_release);
    }
    if (e != cudaSuccess) return e;
    if ((e = launch_behind(paged_attention_kernel<D, NT, KIND>, dim3(a.grid), kThreads, smem, st, a)) != cudaSuccess || a.whole_items) return e;
    const bool fp16 = KIND == kFp16 || (in_records(KIND) && a.q_fp16);
    return launch_behind(paged_combine_kernel<D, NT, KIND>, dim3(a.grid), kCombineWarps * 32, 0, st, a, fp16);
}

template <int D, int NT>
cudaError_t launch_kind(PagedAttnArgs& a, int sms, int dev, cudaStream_t st) {
    return a.c.kv_type == TKV_INT4   ? launch<D, NT, kInt4>(a, sms, dev, st)
           : a.c.kv_type == TKV_E4M3 ? launch<D, NT, kE4m3>(a, sms, dev, st)
           : a.c.kv_type == TKV_BF16 ? launch<D, NT, kBf16>(a, sms, dev, st)
                                     : launch<D, NT, kFp16>(a, sms, dev, st);
}

template <int D>
cudaError_t launch_rows(PagedAttnArgs& a, int nt, int sms, int dev, cudaStream_t st) {
    return nt == 1                      ? launch_kind<D, 1>(a, sms, dev, st)
           : nt == 2                    ? launch_kind<D, 2>(a, sms, dev, st)
           : a.c.kv_type == TKV_E4M3    ? launch<D, 4, kE4m3>(a, sms, dev, st)
                                        : launch<D, 4, kInt4>(a, sms, dev, st);
}

bool attention_shape_ok(const tkv_paged* c, int32_t hq, int32_t max_new) {
    return check_paged(c) == TKV_OK && hq >= 1 && hq % c->num_kv_heads == 0 && max_new >= 1;
}

}  // namespace

extern "C" int64_t tkv_paged_attention_workspace(const tkv_paged* cache, int32_t num_q_heads, int32_t max_new) {
    if (!attention_shape_ok(cache, num_q_heads, max_new)) return 0;
    int sms = 0, dev = 0;
    if (device_sms(&sms, &dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    return workspace_bytes_of(cache, num_q_heads, max_new, sms);
}

extern "C" tkv_status tkv_paged_attention(const tkv_paged* cache, const void* q, void* out, float* lse, int32_t dtype,
                                          int64_t rows, int32_t num_q_heads, int64_t q_row_stride, int64_t q_head_stride,
                                          int64_t out_row_stride, int64_t out_head_stride, const int32_t* cu_tokens,
                                          int32_t max_new, int32_t max_len, int32_t window, float scale, void* workspace,
                                          int64_t workspace_bytes, int32_t* status, void* stream) {
    if (!attention_shape_ok(cache, num_q_heads, max_new) || max_len < 1 || window < 0 || !std::isfinite((float)((double)scale * kLog2E))) return TKV_EINVAL;
    if (dtype != TKV_BF16 && dtype != TKV_FP16) return TKV_EINVAL;
    if (!has_records(cache->kv_type) && cache->kv_type != dtype) return TKV_EINVAL;
    if (rows < 0 || rows > 0x7FFFFFFF || !cu_tokens) return TKV_EINVAL;
    if (rows == 0) return TKV_OK;
    // row indices within a sequence (queries x heads of a group) are 32-bit
    if (!q || !out || q == out || rows * (num_q_heads / cache->num_kv_heads) > 0x7FFF0000) return TKV_EINVAL;
    if (!aligned4(lse) || !aligned4(cu_tokens) || !aligned4(status)) return TKV_EINVAL;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || q_row_stride < 0 || q_head_stride < 0 || q_row_stride % 8 ||
        q_head_stride % 8 || out_row_stride % 8 || out_head_stride % 8)
        return TKV_EINVAL;
    if (!strides_apart(rows, out_row_stride, num_q_heads, out_head_stride, cache->head_dim)) return TKV_EINVAL;
    int sms = 0, dev = 0;
    cudaError_t e = device_sms(&sms, &dev);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return TKV_ECUDA;
    }
    if (!workspace || workspace_bytes < workspace_bytes_of(cache, num_q_heads, max_new, sms)) return TKV_ECAPACITY;
    PagedAttnArgs a{};
    a.c = *cache;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.cu = cu_tokens;
    a.part = reinterpret_cast<float4*>(workspace);
    a.status = status;
    a.rows = rows;
    a.q_row = q_row_stride;
    a.q_head = q_head_stride;
    a.out_row = out_row_stride;
    a.out_head = out_head_stride;
    a.hq = num_q_heads;
    a.group = num_q_heads / cache->num_kv_heads;
    a.group_mul = 0xFFFFFFFFu / (uint32_t)a.group;
    a.give_up = warp_that_gives_up();
    a.window = window;
    a.page_shift = __builtin_ctz((unsigned)cache->page_size);
    const int64_t sight = window > 0 ? std::min<int64_t>(max_len, (int64_t)window + max_new) : max_len;
    a.q_fp16 = dtype == TKV_FP16;
    a.scale_log2 = (float)((double)scale * kLog2E);
    cudaStream_t st = (cudaStream_t)stream;
    const int nt = rows_of_32(a, max_new, sight, sms) ? 4 : row_tiles(a.group, max_new);
    const double items = ((double)rows * a.group / (8 * nt) + cache->batch) * cache->num_kv_heads;   // at most
    a.whole_items = sight <= kWholeShort || (sight <= kWholeMany && items >= sms && cache->kv_type == TKV_INT4);
    const bool two_groups = cache->kv_type == TKV_INT4 || (cache->kv_type == TKV_E4M3 && cache->head_dim == 64);   // 32 positions a tile
    const int tile = two_groups ? 32 : 16;
    const double item_tiles = (double)(((int64_t)cache->max_pages * cache->page_size + tile - 1) / tile);
    if (items * item_tiles > kMostTiles) return TKV_EINVAL;
    // what an item counts beyond its tiles refuses no step
    a.pad = cache->kv_type == TKV_E4M3 && !a.whole_items && items * (item_tiles + kItemTiles) <= kMostTiles ? kItemTiles : 0;
    e = cache->head_dim == 128 ? launch_rows<128>(a, nt, sms, dev, st) : launch_rows<64>(a, nt, sms, dev, st);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return TKV_ECUDA;
    }
    return TKV_OK;
}
