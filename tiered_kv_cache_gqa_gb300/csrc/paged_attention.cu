// Attention of a step's queries over a paged cache held in 4 bits or in 16: tkv_paged_attention.
//
// Mathematics.  For a KV head, the rows of a step (query t of a sequence, query head g of the group: row
// t G + g) are columns of two small matrix products a tile of positions:
//   S^T = K q^T     (positions x rows; K from the cache, q in registers)
//   O^T += V^T P^T  (channels x rows; P = 2^(z - m), z = S scale log2 e)
// with one pass over the positions: every warp keeps, for each row, a reference m, the sum of its p and
// O in fp32.  m is not the running maximum but a number that the maximum has not passed by more than kTop
// (in powers of two): p stays within fp16's range, the common tile needs no exchange between lanes,
// and O is rescaled only where that room is used up.
// Transposed like this, a group of 8 heads fills the 8 columns of mma.m16n8k16 with nothing wasted; the
// operation is bound by memory (at G = 8 and 4 bits, 28 operations a byte), so mma.sync is enough.
//
// 4 bits to fp16, exactly.  (w & 0x000F000F) | 0x64006400 is the pair (1024 + n, 1024 + n') of two codes
// n = q + 8, and (w & 0x00F000F0) | 0x54005400 the pair (64 + n, 64 + n'); one fused multiply-add with
// s = scale / 16 gives (1024 + n) s - 1032 s = q s (and (64 + n) s - 72 s).  Every operand and result is
// exact in fp16: scale has 4 bits, 129 * 15 < 2^11, and 1032 * 448 / 16 is below its largest number.
// So K and V enter the products as stored; what is rounded is p (to fp16, 2^-11) and, for rows in
// bf16 of a wide range, what lies 2^-29 below a row's largest channel (q is scaled by a power of two).
// The channels that a lane holds of a position are those of its own bytes: K's products sum over all
// channels, so q is laid out to match; for V the lanes' channels are rows of O^T.
//
// Work split.  The positions of every (sequence, KV head, tile of rows) are cut into units of 128; the
// units of all of them, in that order, are dealt out in equal contiguous shares to the CTAs that fit on
// the device at once, whatever the lengths are.  Every CTA computes the deal from lengths and cu_tokens
// itself.  A CTA's piece of an item goes to `out` if it is the whole item, to the workspace (two
// records a CTA) if not; a second kernel, started early, joins the pieces of each cut item in order.
// Within a CTA, warp w takes tiles w, w + 8, ...; its copies run kStages tiles ahead in a ring of its own.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "paged.cuh"
#include "tkv_internal.cuh"

using namespace tkv;

namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kUnit = 128;              // positions that work is dealt in
constexpr int kMinUnits = 2;            // of a share: below, joining costs more than it brings
constexpr int kWholeItems = 512;        // up to this length a CTA takes whole items, and nothing is joined
constexpr float kTop = 15.0f;           // p = 2^(z - m) <= 2^15; in fp16 the smallest is 2^-24
constexpr float kLift = 5.0f;           // a new reference lies this far below the maximum: 10 are left to grow
constexpr float kLowest = -3.402823466e38f;   // a reference before anything is seen: 2^(-inf - it) = 0, no NaN
constexpr int kSpinLimit = 1 << 16;     // tries of a wait, each of which the hardware suspends for a while

enum PageKind { kInt4, kBf16, kFp16 };

struct PagedAttnArgs {
    tkv_paged c;
    const void* q;
    void* out;
    float* lse;
    const int32_t* cu;
    float* part;                         // [grid][2][R][D + 4]: O (unnormalised, its reference m), m, l
    int32_t* status;
    int64_t rows, q_row, q_head, out_row, out_head;
    int hq, group, window, page_shift, grid, whole_items, q_fp16;
    float scale_log2;
};

// ------------------------------------------------------------------ small pieces of PTX
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 x 8 16-bit matrix, one row's pair a lane -> its transpose
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (x & mask) | bits in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(mask), "r"(bits));
    return y;
}
__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_half2(uint32_t w) { return *reinterpret_cast<__half2*>(&w); }
__device__ __forceinline__ void mbar_init(uint32_t bar, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect(uint32_t bar, int bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Bounded: false if the phase did not end.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, int parity) {
    for (int i = 0; i < kSpinLimit; ++i) {
        uint32_t done;
        asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                     : "=r"(done) : "r"(bar), "r"(parity) : "memory");
        if (done) return true;
    }
    return false;
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, int bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {   // bytes: 16, or 0 for zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// ------------------------------------------------------------------ the deal
// What sequence b brings: its queries n, its visible end `len`, the first unit's position `lo`, the units
// of one item, and the items (KV head x tile of rows).
struct Seq {
    int first_row, n, len, lo, units, tiles;
};

template <int R>
__device__ __forceinline__ Seq sequence(const PagedAttnArgs& a, int b) {
    Seq s;
    const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1), len = max(0, __ldg(a.c.lengths + b));
    s.first_row = c0;
    s.n = (c0 < 0 || c1 <= c0 || c1 > a.rows) ? 0 : c1 - c0;
    const int cap = a.c.max_pages << a.page_shift;
    s.len = min(len, cap);
    s.lo = 0;
    if (a.window > 0) s.lo = max(0, min(s.len, len - s.n - a.window + 1)) & ~(kUnit - 1);
    s.units = s.n ? max(1, (s.len - s.lo + kUnit - 1) / kUnit) : 0;
    s.tiles = (int)(((int64_t)s.n * a.group + R - 1) / R);
    return s;
}

// Totals over the batch, and the place of unit `u` in it.  All threads of the CTA call it; `scratch`:
// kWarps + 1 int64 and one int4 of shared memory.
template <int R>
__device__ __forceinline__ int64_t weight(const PagedAttnArgs& a, const Seq& s) {   // units, or items, of a sequence
    return (int64_t)s.tiles * a.c.num_kv_heads * (a.whole_items ? (s.n ? 1 : 0) : s.units);
}

template <int R>
__device__ __forceinline__ int64_t scan_batch(const PagedAttnArgs& a, int64_t* scratch, int64_t* before, int64_t* own, int threads) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.c.batch + threads - 1) / threads;
    int64_t mine = 0;
    for (int b = tid * per; b < min(a.c.batch, (tid + 1) * per); ++b) mine += weight<R>(a, sequence<R>(a, b));
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
    }
    if (lane == 31) scratch[warp] = sum;
    __syncthreads();
    int64_t base = 0, total = 0;
    for (int w = 0; w < threads / 32; ++w) {
        if (w < warp) base += scratch[w];
        total += scratch[w];
    }
    *before = base + sum - mine;
    *own = mine;
    return total;
}

// The sequence that unit `u` (< total) lies in and what lies before it in that sequence, into where[0..1].
template <int R>
__device__ __forceinline__ void locate(const PagedAttnArgs& a, int64_t u, int64_t before, int64_t own, int64_t* where, int threads) {
    const int per = (a.c.batch + threads - 1) / threads;
    if (u >= before && u < before + own) {
        int64_t left = u - before;
        int b = threadIdx.x * per;
        for (;; ++b) {
            const int64_t w = weight<R>(a, sequence<R>(a, b));
            if (left < w) break;
            left -= w;
        }
        where[0] = b;
        where[1] = left;
    }
    __syncthreads();
}

__device__ __forceinline__ int64_t share_of(const PagedAttnArgs& a, int64_t total) {
    const int64_t even = (total + a.grid - 1) / a.grid;
    return a.whole_items ? even : (even > kMinUnits ? even : kMinUnits);
}

// ------------------------------------------------------------------ tiles of positions
template <int D, int KIND>
struct Tile {
    static constexpr int positions = KIND == kInt4 ? 32 : 16;
    static constexpr int bytes = KIND == kInt4 ? 2 * Record<D>::bytes : 2 * 16 * D * 2;
};

// Stages of a warp's ring.  One CTA or two share the SM's 227 KB (launch_bounds below).
template <int D, int NT, int KIND>
struct Config {
    static constexpr int R = 8 * NT;
    static constexpr int ctas = (KIND == kInt4 && NT == 1) ? 2 : 1;
    static constexpr int stages = KIND == kInt4 ? (D == 128 ? (NT == 1 ? 3 : 6) : (NT == 1 ? 5 : 10)) : (D == 128 ? 3 : 6);
    static constexpr int warp_ring = stages * Tile<D, KIND>::bytes;
    static constexpr int row_stride = D + 4;   // floats of a row in the merge: the lanes' 16-byte stores spread over the banks
    static constexpr int merge_bytes = kWarps * R * row_stride * 4;
    static constexpr int ring_bytes = kWarps * warp_ring > merge_bytes ? kWarps * warp_ring : merge_bytes;
    static constexpr int off_bars = ring_bytes;
    static constexpr int off_ml = off_bars + kWarps * stages * 8;
    static constexpr int off_scan = off_ml + kWarps * R * 8;
    static constexpr int smem = off_scan + (kWarps + 4) * 8;
};

// What a CTA works on.
struct Segment {
    int b, h, tile;          // sequence, KV head, tile of rows
    int begin, end;          // positions; empty if end <= begin
    int last0, n;            // the last position that query 0 sees; queries
    int first_row, row0, rows_of_seq;
    bool whole;
    int slot;                // of its partial record
};

template <int D, int NT, int KIND>
__global__ void __launch_bounds__(kThreads, Config<D, NT, KIND>::ctas) paged_attention_kernel(const __grid_constant__ PagedAttnArgs a) {
    using C = Config<D, NT, KIND>;
    using Rec = Record<D>;
    constexpr int R = C::R, S = C::stages, TP = Tile<D, KIND>::positions, TB = Tile<D, KIND>::bytes;
    constexpr int KM = D / 16;   // matrix steps over the channels, and 16-channel blocks of O^T
    extern __shared__ __align__(128) uint8_t smem[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, cq = lane & 3;   // a lane's row and quad column in the matrix fragments
    float2* ml = reinterpret_cast<float2*>(smem + C::off_ml);           // [warp][R]: reference, sum
    int64_t* scan = reinterpret_cast<int64_t*>(smem + C::off_scan);
    const uint32_t bar0 = smem_u32(smem + C::off_bars) + warp * S * 8;
    uint8_t* ring = smem + warp * C::warp_ring;
    const uint32_t ring_s = smem_u32(ring);
    if (KIND == kInt4 && lane == 0) {
        for (int s = 0; s < S; ++s) mbar_init(bar0 + 8 * s, 2);   // lanes 0 and 1 bring one record each
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    int64_t before, own;
    const int64_t total = scan_batch<R>(a, scan, &before, &own, kThreads);
    const int64_t share = share_of(a, total);
    int64_t u = (int64_t)blockIdx.x * share;
    const int64_t u1 = min(total, u + share);
    if (u >= u1) return;
    locate<R>(a, u, before, own, scan + kWarps, kThreads);
    int b = (int)scan[kWarps];
    int64_t in_seq = scan[kWarps + 1];
    Seq s = sequence<R>(a, b);
    // the ring, over all segments: the stage of the next tile, and the parity that its barrier ends with
    int stage = 0, parity = 0;
    auto after = [](int st, int k) { return st + k >= S ? st + k - S : st + k; };
    const int64_t page_bytes = (int64_t)a.c.num_kv_heads * (KIND == kInt4 ? (a.c.page_size >> 4) * Rec::bytes : a.c.page_size * 4 * D);
    const int in_page = a.c.page_size - 1;
    const uint32_t pages = (uint32_t)min(a.c.num_pages, (int64_t)0x7FFFFFFF);
    bool failed = false;

    while (u < u1) {
        // -------------------------------------------------------- the next segment
        while (in_seq >= weight<R>(a, s)) {
            in_seq -= weight<R>(a, s);
            s = sequence<R>(a, ++b);
        }
        const int per_item = a.whole_items ? 1 : s.units;
        const int item = (int)(in_seq / per_item), c0 = (int)(in_seq - (int64_t)item * per_item);
        const int c1 = (int)min((int64_t)per_item, c0 + (u1 - u));
        u += c1 - c0;
        in_seq += c1 - c0;
        const int h = item / s.tiles, tile = item - h * s.tiles;
        const bool whole = a.whole_items || (c0 == 0 && c1 == per_item);
        const int len = max(0, __ldg(a.c.lengths + b));  // not cut to the table: positions count from it
        const int last0 = len - s.n;                     // query t sees positions <= last0 + t
        const int seq_rows = s.n * a.group;
        const int row0 = tile * R, row_end = min(seq_rows, row0 + R);
        const int t_lo = row0 / a.group, t_hi = (row_end - 1) / a.group;
        const int seen_end = min(s.len, last0 + t_hi + 1);
        const int begin = a.whole_items ? s.lo : s.lo + c0 * kUnit;
        const int end = min(seen_end, a.whole_items ? s.len : s.lo + c1 * kUnit);
        const int all_until = min(s.len - 1, last0 + t_lo);                            // seen by every row up to here,
        const int all_from = a.window > 0 ? last0 + t_hi - a.window + 1 : 0;           // and from here;
        const int any_from = a.window > 0 ? last0 + t_lo - a.window + 1 : 0;           // seen by any row from here
        const bool several = t_hi > t_lo;                                              // queries: rows see different positions
        if (len > s.len && tid == 0) raise_status(a.status, TKV_ECAPACITY);
        const int tiles_here = end > begin && !failed ? (end - begin + TP - 1) / TP : 0;

        // -------------------------------------------------------- copies
        const int32_t* table = a.c.page_table + (int64_t)b * a.c.max_pages;
        uint32_t bad_bits = 0;          // int4: by stage, whether this lane's record is missing
        int page_next = 0;
        // the page of the record (int4: lanes 0, 1) or tile (16 bits) that is copied next; looked up one
        // tile ahead of its copy
        auto look_up = [&](int t) {
            const int p = begin + t * TP + (KIND == kInt4 ? (lane & 1) * 16 : 0);
            page_next = (t < tiles_here && p < end) ? __ldg(table + (p >> a.page_shift)) : -2;
        };
        const uint8_t* head_pages = reinterpret_cast<const uint8_t*>(a.c.pages) + page_bytes / a.c.num_kv_heads * h;
        auto issue = [&](int t, int st) {
            if (KIND == kInt4) {
                if (t < tiles_here && lane < 2) {
                    const int p = begin + t * TP + lane * 16;
                    if ((uint32_t)page_next < pages) {
                        mbar_arrive_expect(bar0 + 8 * st, Rec::bytes);
                        bulk_copy(ring_s + st * TB + lane * Rec::bytes,
                                  head_pages + page_next * page_bytes + ((p & in_page) >> 4) * Rec::bytes, Rec::bytes, bar0 + 8 * st);
                        bad_bits &= ~(1u << st);
                    } else {
                        mbar_arrive(bar0 + 8 * st);
                        bad_bits |= 1u << st;
                        if (page_next != -2) raise_status(a.status, TKV_ECAPACITY);
                    }
                }
            } else {
                if (t < tiles_here) {
                    const int p = begin + t * TP;
                    const bool ok = (uint32_t)page_next < pages;
                    if (!ok && lane == 0) raise_status(a.status, TKV_ECAPACITY);
                    if (ok) bad_bits &= ~(1u << st); else bad_bits |= 1u << st;
                    constexpr int CH = D / 8;            // 16-byte pieces of a row, stored at piece ^ (row & 7)
                    const uint8_t* src = head_pages + (ok ? page_next * page_bytes : 0) + (p & in_page) * (2 * D);
                    const int64_t v_off = (int64_t)a.c.page_size * (2 * D);
#pragma unroll
                    for (int i = 0; i < 16 * CH / 32; ++i) {
                        const int row = (i * 32 + lane) / CH, piece = lane % CH;
                        const int n = ok && p + row < end ? 16 : 0;      // absent rows are zeros
                        const uint32_t dst = ring_s + st * TB + row * (2 * D) + ((piece ^ (row & 7)) << 4);
                        cp_async16(dst, src + row * (2 * D) + piece * 16, n);
                        cp_async16(dst + 16 * D * 2, src + v_off + row * (2 * D) + piece * 16, n);
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
        };
        look_up(warp);
#pragma unroll 1
        for (int k = 0; k < S - 1; ++k) {
            issue(warp + k * kWarps, after(stage, k));
            look_up(warp + (k + 1) * kWarps);
        }

        // -------------------------------------------------------- q
        // fragments of q^T: column r of row tile nt; int4: channels in the order of the codes' pairs
        uint32_t qf[NT][KM][2];
        float zs0[NT], zs1[NT];                              // columns 2 cq, 2 cq + 1: S -> z
        const float gain_k = KIND == kInt4 && a.c.k_gain ? __ldg(a.c.k_gain + h) : 1.0f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = row0 + nt * 8 + r;
            const bool is_row = row < seq_rows;
            const int t = is_row ? row / a.group : 0, g = is_row ? row - t * a.group : 0;
            const uint16_t* q = reinterpret_cast<const uint16_t*>(a.q) + (s.first_row + t) * a.q_row + (h * a.group + g) * a.q_head;
            if (KIND == kInt4) {
                constexpr int W = D / 32;                    // words of codes, 8 channels each
                float x[8 * W];
                float top = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (is_row) v = __ldg(reinterpret_cast<const uint4*>(q + (D / 4) * cq + 8 * w));
                    const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = a.q_fp16 ? __half22float2(bits_half2(e[i])) : bf16x2_to_float2(e[i]);
                        x[8 * w + 2 * i] = f.x;
                        x[8 * w + 2 * i + 1] = f.y;
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // the largest channel into [2^14, 2^15): a power of two, undone in zs
                const int ex = min(254, max(1, 268 - (int)(__float_as_uint(top) >> 23)));
                const float up = __uint_as_float((uint32_t)ex << 23);
#pragma unroll
                for (int i = 0; i < KM; ++i) {
                    const int w = i >> 1, p = (i & 1) * 2;
                    qf[nt][i][0] = half2_bits(__floats2half2_rn(x[8 * w + p] * up, x[8 * w + p + 4] * up));
                    qf[nt][i][1] = half2_bits(__floats2half2_rn(x[8 * w + p + 1] * up, x[8 * w + p + 5] * up));
                }
                const float z = a.scale_log2 * gain_k * 16.0f / up;
                zs0[nt] = __shfl_sync(0xffffffffu, z, 8 * cq);
                zs1[nt] = __shfl_sync(0xffffffffu, z, 8 * cq + 4);
            } else {
#pragma unroll
                for (int i = 0; i < KM; ++i) {
                    qf[nt][i][0] = is_row ? __ldg(reinterpret_cast<const uint32_t*>(q + 16 * i + 2 * cq)) : 0u;
                    qf[nt][i][1] = is_row ? __ldg(reinterpret_cast<const uint32_t*>(q + 16 * i + 2 * cq + 8)) : 0u;
                }
                zs0[nt] = zs1[nt] = a.scale_log2;
            }
        }
        // the last position that the lane's columns see (rows behind the last: whatever)
        int last[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) last[nt][e] = last0 + (row0 + nt * 8 + 2 * cq + e) / a.group;

        // -------------------------------------------------------- the tiles of this warp
        float o[NT][KM][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = kLowest;
            l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
            for (int j = 0; j < KM; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.0f;
        }
#pragma unroll 1
        for (int t = warp; t < tiles_here; t += kWarps) {
            const int st = stage;
            // the slot that the last tile left is filled before this one is waited for
            issue(t + (S - 1) * kWarps, after(st, S - 1));
            look_up(t + S * kWarps);
            uint32_t bad;
            if (KIND == kInt4) {
                if (!failed && !mbar_wait(bar0 + 8 * st, parity)) {
                    failed = true;
                    if (lane == 0) raise_status(a.status, TKV_ETIMEOUT);
                }
                failed = __any_sync(0xffffffffu, failed);
                if (failed) break;
                bad = __ballot_sync(0xffffffffu, (bad_bits >> st) & 1) & 3;
            } else {
                asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
                __syncwarp();
                bad = (bad_bits >> st) & 1 ? 3 : 0;
            }
            const int p0 = begin + t * TP;
            const bool plain = !bad && p0 + TP - 1 <= all_until && p0 >= all_from;   // every row sees every position
            const uint8_t* tile_at = ring + st * TB;
            const uint32_t tile_s = ring_s + st * TB;
            constexpr int NG = TP / 16;
            auto tile = [&](auto whole_tile) {
            constexpr bool kPlain = decltype(whole_tile)::value;
            // The lane's four V positions of a group (the columns of its fragments): bit i set if position i lies in [from, to).
            constexpr bool kPermuted = KIND == kInt4;
            const int v0 = kPermuted ? (2 * cq) ^ (cq & 1) : 2 * cq, v1 = kPermuted ? (2 * cq + 1) ^ (cq & 1) : 2 * cq + 1;
            auto v_bits = [&](int base, int from, int to) -> uint32_t {
                uint32_t bits = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int p = base + (i & 1 ? v1 : v0) + (i >> 1) * 8;
                    bits |= p >= from && p < to ? 1u << i : 0u;
                }
                return bits;
            };
            // acc += V^T P^T of group g, V taken as 0 where `keep` has no bit (a plain tile has them all); with `look`
            // nothing is added: whether the lane's part of V, so masked, holds an infinity or a NaN.
            auto v_step = [&](int g, uint32_t keep, const uint32_t (&ph)[NT][2], const uint32_t (&plo)[NT][2],
                              float (&acc)[NT][KM][4], bool look) -> bool {
                const uint32_t m0 = (keep & 1 ? 0xFFFFu : 0u) | (keep & 2 ? 0xFFFF0000u : 0u);
                const uint32_t m1 = (keep & 4 ? 0xFFFFu : 0u) | (keep & 8 ? 0xFFFF0000u : 0u);
                bool odd = false;
                if (KIND == kInt4) {
                    const uint8_t* rec = tile_at + g * Rec::bytes;
                    // scales of the two position pairs, in the order of the slots
                    const uint8_t* vs = rec + Rec::v_scales + (D == 128 ? r : r >> 1) * 16 + 2 * cq;
                    const uint32_t swap = cq & 1 ? 0x1032u : 0x3210u;
                    __half2 s_lo[2], n_lo[2], n_hi[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t x = half2_bits(__half2(__nv_cvt_fp8x2_to_halfraw2(*reinterpret_cast<const uint16_t*>(vs + 8 * i), __NV_E4M3)));
                        x = __byte_perm(x, 0, swap);
                        if (!kPlain) x &= i ? m1 : m0;
                        odd |= (x & 0x7C00u) == 0x7C00u || (x & 0x7C000000u) == 0x7C000000u;
                        s_lo[i] = __hmul2(bits_half2(x), __half2half2(__float2half(0.0625f)));
                        n_lo[i] = __hmul2(s_lo[i], __half2half2(__float2half(-1032.0f)));
                        n_hi[i] = __hmul2(s_lo[i], __half2half2(__float2half(-72.0f)));
                    }
                    if (look) return odd;
                    const uint8_t* vc = rec + Rec::v_codes + r * (D / 16);
                    constexpr int W = D / 64;                     // words of 8 channels a position
                    uint32_t w[4][W];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint8_t* at = vc + ((i & 1 ? v1 : v0) + (i >> 1) * 8) * (D / 2);
                        if (D == 128) {
                            const uint2 x = *reinterpret_cast<const uint2*>(at);
                            w[i][0] = x.x;
                            w[i][W - 1] = x.y;
                        } else {
                            w[i][0] = *reinterpret_cast<const uint32_t*>(at);
                        }
                    }
                    // a word of the positions' low (high) halves: four channels of the pair
#pragma unroll
                    for (int wi = 0; wi < W; ++wi)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            uint32_t x = __byte_perm(w[0][wi], w[1][wi], half ? 0x7632 : 0x5410);
                            uint32_t y = __byte_perm(w[2][wi], w[3][wi], half ? 0x7632 : 0x5410);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t f0 = half2_bits(__hfma2(bits_half2(and_or(x, 0x000F000Fu, 0x64006400u)), s_lo[0], n_lo[0]));
                                const uint32_t f1 = half2_bits(__hfma2(bits_half2(and_or(x, 0x00F000F0u, 0x54005400u)), s_lo[0], n_hi[0]));
                                const uint32_t f2 = half2_bits(__hfma2(bits_half2(and_or(y, 0x000F000Fu, 0x64006400u)), s_lo[1], n_lo[1]));
                                const uint32_t f3 = half2_bits(__hfma2(bits_half2(and_or(y, 0x00F000F0u, 0x54005400u)), s_lo[1], n_hi[1]));
                                const int j = 4 * wi + 2 * half + i;   // rows r and r + 8: channels (D / 8) r + 2 j and + 1
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt][j], f0, f1, f2, f3, ph[nt][0], ph[nt][1]);
                                x >>= 8;
                                y >>= 8;
                            }
                        }
                } else {
#pragma unroll
                    for (int j = 0; j < KM; ++j) {
                        uint32_t f[4];
                        const int row = (lane & 7) + ((lane >> 4) << 3), piece = 2 * j + ((lane >> 3) & 1);
                        ldmatrix4_trans(f, tile_s + 16 * D * 2 + row * (2 * D) + ((piece ^ (row & 7)) << 4));
                        if (!kPlain) {
                            f[0] &= m0; f[1] &= m0; f[2] &= m1; f[3] &= m1;
                        }
                        if (look) {
                            constexpr uint32_t ex = KIND == kBf16 ? 0x7F80u : 0x7C00u;
#pragma unroll
                            for (int i = 0; i < 4; ++i) odd |= (f[i] & ex) == ex || (f[i] & (ex << 16)) == (ex << 16);
                            continue;
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (KIND == kBf16) {
                                mma_bf16(acc[nt][j], f[0], f[1], f[2], f[3], ph[nt][0], ph[nt][1]);
                                mma_bf16(acc[nt][j], f[0], f[1], f[2], f[3], plo[nt][0], plo[nt][1]);
                            } else {
                                mma_f16(acc[nt][j], f[0], f[1], f[2], f[3], ph[nt][0], ph[nt][1]);
                            }
                        }
                    }
                }
                return odd;
            };
            // ---- S^T, z
            float z[NG][NT][4];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) z[g][nt][0] = z[g][nt][1] = z[g][nt][2] = z[g][nt][3] = 0.0f;
                if (KIND == kInt4) {
                    // rows of the fragment: positions 0 1 3 2 4 5 7 6, so that the lanes of a quarter warp
                    // (K) and of a half warp (V) read from different banks
                    const int pr = r ^ ((r >> 1) & 1);
                    const uint8_t* rec = tile_at + g * Rec::bytes;
                    constexpr int W = D / 32;
                    uint32_t wa[W], wb[W];
                    __half2 sa[W / 2], sb[W / 2];   // scale / 16 of the lane's blocks, twice each; d = 64: one block
                    if (D == 128) {
                        const uint4 x = *reinterpret_cast<const uint4*>(rec + pr * 64 + cq * 16);
                        const uint4 y = *reinterpret_cast<const uint4*>(rec + (pr + 8) * 64 + cq * 16);
                        wa[0] = x.x; wa[1] = x.y; wa[W - 2] = x.z; wa[W - 1] = x.w;
                        wb[0] = y.x; wb[1] = y.y; wb[W - 2] = y.z; wb[W - 1] = y.w;
                        const uint16_t s8a = *reinterpret_cast<const uint16_t*>(rec + Rec::k_scales + pr * 8 + cq * 2);
                        const uint16_t s8b = *reinterpret_cast<const uint16_t*>(rec + Rec::k_scales + (pr + 8) * 8 + cq * 2);
                        const __half2 fa = __hmul2(__half2(__nv_cvt_fp8x2_to_halfraw2(s8a, __NV_E4M3)), __half2half2(__float2half(0.0625f)));
                        const __half2 fb = __hmul2(__half2(__nv_cvt_fp8x2_to_halfraw2(s8b, __NV_E4M3)), __half2half2(__float2half(0.0625f)));
                        sa[0] = __low2half2(fa); sa[W / 2 - 1] = __high2half2(fa);
                        sb[0] = __low2half2(fb); sb[W / 2 - 1] = __high2half2(fb);
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2*>(rec + pr * 32 + cq * 8);
                        const uint2 y = *reinterpret_cast<const uint2*>(rec + (pr + 8) * 32 + cq * 8);
                        wa[0] = x.x; wa[1] = x.y;
                        wb[0] = y.x; wb[1] = y.y;
                        const __half_raw ha = __nv_cvt_fp8_to_halfraw(rec[Rec::k_scales + pr * 4 + cq], __NV_E4M3);
                        const __half_raw hb = __nv_cvt_fp8_to_halfraw(rec[Rec::k_scales + (pr + 8) * 4 + cq], __NV_E4M3);
                        sa[0] = __hmul2(__half2half2(__half(ha)), __half2half2(__float2half(0.0625f)));
                        sb[0] = __hmul2(__half2half2(__half(hb)), __half2half2(__float2half(0.0625f)));
                    }
#pragma unroll
                    for (int k = 0; k < W / 2; ++k) {
                        const __half2 a_lo = sa[k], b_lo = sb[k];
                        const __half2 a_lo0 = __hmul2(a_lo, __half2half2(__float2half(-1032.0f))), a_hi0 = __hmul2(a_lo, __half2half2(__float2half(-72.0f)));
                        const __half2 b_lo0 = __hmul2(b_lo, __half2half2(__float2half(-1032.0f))), b_hi0 = __hmul2(b_lo, __half2half2(__float2half(-72.0f)));
#pragma unroll
                        for (int w2 = 0; w2 < 2; ++w2) {
                            uint32_t x = wa[2 * k + w2], y = wb[2 * k + w2];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t f0 = half2_bits(__hfma2(bits_half2(and_or(x, 0x000F000Fu, 0x64006400u)), a_lo, a_lo0));
                                const uint32_t f2 = half2_bits(__hfma2(bits_half2(and_or(x, 0x00F000F0u, 0x54005400u)), a_lo, a_hi0));
                                const uint32_t f1 = half2_bits(__hfma2(bits_half2(and_or(y, 0x000F000Fu, 0x64006400u)), b_lo, b_lo0));
                                const uint32_t f3 = half2_bits(__hfma2(bits_half2(and_or(y, 0x00F000F0u, 0x54005400u)), b_lo, b_hi0));
                                const int step_k = 2 * (2 * k + w2) + i;
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) mma_f16(z[g][nt], f0, f1, f2, f3, qf[nt][step_k][0], qf[nt][step_k][1]);
                                x >>= 8;
                                y >>= 8;
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < KM; ++i) {
                        uint32_t f[4];
                        const int row = (lane & 7) + (lane & 8), piece = 2 * i + (lane >> 4);
                        ldmatrix4(f, tile_s + row * (2 * D) + ((piece ^ (row & 7)) << 4));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (KIND == kBf16) mma_bf16(z[g][nt], f[0], f[1], f[2], f[3], qf[nt][i][0], qf[nt][i][1]);
                            else mma_f16(z[g][nt], f[0], f[1], f[2], f[3], qf[nt][i][0], qf[nt][i][1]);
                        }
                    }
                }
            }
            // position of the lane's rows r and r + 8 in group g
            const int pr0 = KIND == kInt4 ? r ^ ((r >> 1) & 1) : r;
            uint32_t keep[NG];   // which of the lane's four V positions of a group any row sees
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                keep[g] = 15;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    z[g][nt][0] *= zs0[nt];
                    z[g][nt][1] *= zs1[nt];
                    z[g][nt][2] *= zs0[nt];
                    z[g][nt][3] *= zs1[nt];
                }
                if (!kPlain) {
                    const bool here = !((bad >> g) & 1);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int p = p0 + 16 * g + pr0 + (e >> 1) * 8, to = last[nt][e & 1];
                            if (!here || p >= s.len || p > to || (a.window > 0 && p <= to - a.window)) z[g][nt][e] = -INFINITY;
                        }
                    // the others may hold anything: their V is taken as 0
                    keep[g] = here ? v_bits(p0 + 16 * g, any_from, seen_end) : 0u;
                }
            }
            // ---- softmax
            bool over = false;
            float top[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(z[0][nt][e], z[0][nt][e + 2]);
                    if (NG == 2) x = fmaxf(x, fmaxf(z[NG - 1][nt][e], z[NG - 1][nt][e + 2]));
                    top[nt][e] = x;
                    over |= x - m[nt][e] > kTop;
                }
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = top[nt][e];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        const float mn = fmaxf(m[nt][e], x - kLift);
                        const float f = exp2_approx(m[nt][e] - mn);
                        m[nt][e] = mn;
                        l[nt][e] *= f;
#pragma unroll
                        for (int j = 0; j < KM; ++j) {
                            o[nt][j][e] *= f;
                            o[nt][j][e + 2] *= f;
                        }
                    }
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint32_t ph[NT][2], plo[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float p00 = exp2_approx(z[g][nt][0] - m[nt][0]), p01 = exp2_approx(z[g][nt][1] - m[nt][1]);
                    const float p10 = exp2_approx(z[g][nt][2] - m[nt][0]), p11 = exp2_approx(z[g][nt][3] - m[nt][1]);
                    l[nt][0] += p00 + p10;
                    l[nt][1] += p01 + p11;
                    if (KIND == kBf16) {
                        // bf16 keeps 8 bits: p as a sum of two, which the products add up in fp32
                        const __nv_bfloat162 h0 = __floats2bfloat162_rn(p00, p01), h1 = __floats2bfloat162_rn(p10, p11);
                        const float2 f0 = __bfloat1622float2(h0), f1 = __bfloat1622float2(h1);
                        const __nv_bfloat162 g0 = __floats2bfloat162_rn(p00 - f0.x, p01 - f0.y), g1 = __floats2bfloat162_rn(p10 - f1.x, p11 - f1.y);
                        ph[nt][0] = transpose8(*reinterpret_cast<const uint32_t*>(&h0));
                        ph[nt][1] = transpose8(*reinterpret_cast<const uint32_t*>(&h1));
                        plo[nt][0] = transpose8(*reinterpret_cast<const uint32_t*>(&g0));
                        plo[nt][1] = transpose8(*reinterpret_cast<const uint32_t*>(&g1));
                    } else {
                        ph[nt][0] = transpose8(half2_bits(__floats2half2_rn(p00, p01)));
                        ph[nt][1] = transpose8(half2_bits(__floats2half2_rn(p10, p11)));
                    }
                }
                // ---- O^T += V^T P^T
                const bool odd = !kPlain && several && __any_sync(0xffffffffu, v_step(g, keep[g], ph, plo, o, true));
                if (!odd) {
                    v_step(g, keep[g], ph, plo, o, false);
                } else {
                    // An infinity or a NaN in V where some rows look and others do not: 0 times it is no 0, so each
                    // row gets products of its own, without the positions that it does not see.
#pragma unroll 1
                    for (int n = 0; n < R; ++n) {
                        const int to = last0 + (row0 + n) / a.group;
                        float x[NT][KM][4];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < KM; ++j) x[nt][j][0] = x[nt][j][1] = x[nt][j][2] = x[nt][j][3] = 0.0f;
                        v_step(g, keep[g] & v_bits(p0 + 16 * g, a.window > 0 ? to - a.window + 1 : 0, to + 1), ph, plo, x, false);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (nt * 8 + 2 * cq + e == n) {
#pragma unroll
                                    for (int j = 0; j < KM; ++j) {
                                        o[nt][j][e] += x[nt][j][e];
                                        o[nt][j][e + 2] += x[nt][j][e + 2];
                                    }
                                }
                    }
                }
            }
            };
            if (plain) tile(std::true_type{});
            else tile(std::false_type{});
            stage = after(st, 1);
            parity ^= stage == 0;
            __syncwarp();   // every lane has read the slot before the next turn fills it again
        }
        if (KIND != kInt4) asm volatile("cp.async.wait_all;" ::: "memory");
        if (failed) {
            // a copy did not come in time: the status says so, the rows are NaN, nothing more is issued, and
            // what may still be in flight is given as long again
            for (int k = 0; k < S; ++k) mbar_wait(bar0 + 8 * after(stage, k), parity ^ (stage + k >= S));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = 0.0f, l[nt][0] = l[nt][1] = NAN;
        }

        // -------------------------------------------------------- join the warps
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[nt][e];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (r == 0) ml[warp * R + nt * 8 + 2 * cq + e] = make_float2(m[nt][e], x);
            }
        __syncthreads();   // every warp is done with its ring
        float* merge = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float* to = merge + (warp * R + nt * 8 + 2 * cq + e) * C::row_stride;
                if (KIND == kInt4) {
#pragma unroll
                    for (int j = 0; j < KM; j += 2)
                        *reinterpret_cast<float4*>(to + (D / 8) * r + 2 * j) =
                            make_float4(o[nt][j][e], o[nt][j][e + 2], o[nt][j + 1][e], o[nt][j + 1][e + 2]);
                } else {
#pragma unroll
                    for (int j = 0; j < KM; ++j) {
                        to[16 * j + r] = o[nt][j][e];
                        to[16 * j + r + 8] = o[nt][j][e + 2];
                    }
                }
            }
        __syncthreads();
        const float gain_v = KIND == kInt4 ? 16.0f * (a.c.v_gain ? __ldg(a.c.v_gain + h) : 1.0f) : 1.0f;
        for (int i = tid; i < R * D / 4; i += kThreads) {
            const int row = i / (D / 4), d = (i % (D / 4)) * 4;
            if (row0 + row >= seq_rows) continue;
            float mm = kLowest;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ml[w * R + row].x);
            float sum = 0.0f;
            float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 v = ml[w * R + row];
                const float f = exp2_approx(v.x - mm);
                const float4 x = *reinterpret_cast<const float4*>(merge + (w * R + row) * C::row_stride + d);
                sum += v.y * f;
                acc.x += x.x * f;
                acc.y += x.y * f;
                acc.z += x.z * f;
                acc.w += x.w * f;
            }
            if (whole) {
                const int t = (row0 + row) / a.group, g = row0 + row - t * a.group;
                const int64_t out_row = s.first_row + t;
                const int head = h * a.group + g;
                const float inv = sum == 0.0f ? 0.0f : gain_v / sum;
                const float y[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
                uint16_t* to = reinterpret_cast<uint16_t*>(a.out) + out_row * a.out_row + head * a.out_head + d;
                uint2 w;
                if (KIND == kBf16 || (KIND == kInt4 && !a.q_fp16)) {
                    const __nv_bfloat162 y0 = __floats2bfloat162_rn(y[0], y[1]), y1 = __floats2bfloat162_rn(y[2], y[3]);
                    w = make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
                } else {
                    w = make_uint2(half2_bits(__floats2half2_rn(y[0], y[1])), half2_bits(__floats2half2_rn(y[2], y[3])));
                }
                *reinterpret_cast<uint2*>(to) = w;
                if (a.lse && d == 0)
                    a.lse[out_row * a.hq + head] = sum == 0.0f ? -INFINITY : (mm + log2f(sum)) * 0.69314718056f;
            } else {
                float* rec = a.part + ((int64_t)(blockIdx.x * 2 + (c0 > 0 ? 0 : 1)) * R + row) * (D + 4);
                *reinterpret_cast<float4*>(rec + d) = acc;
                if (d == 0) *reinterpret_cast<float2*>(rec + D) = make_float2(mm, sum);
            }
        }
        if (KIND == kInt4) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before copies land here again
        __syncthreads();
    }
}

// ------------------------------------------------------------------ joining cut items
// CTA i takes the item that is cut at the end of share i, if it began in share i: its pieces are record 1
// of CTA i and record 0 of the CTAs after it.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads) paged_combine_kernel(const __grid_constant__ PagedAttnArgs a, int out_fp16, float gain16) {
    constexpr int R = 8 * NT, LANES = D / 4;   // threads of a row, four channels each
    __shared__ int64_t scan[kWarps + 4];
    int64_t before, own;
    const int64_t total = scan_batch<R>(a, scan, &before, &own, kThreads);
    const int64_t share = share_of(a, total);
    const int64_t cut = (int64_t)(blockIdx.x + 1) * share;
    // what the main kernel wrote is read after this; every CTA waits, so that the grid ends after it
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (cut >= total) return;
    locate<R>(a, cut, before, own, scan + kWarps, kThreads);
    const int b = (int)scan[kWarps];
    const int64_t in_seq = scan[kWarps + 1];
    const Seq s = sequence<R>(a, b);
    const int item = (int)(in_seq / s.units), c = (int)(in_seq - (int64_t)item * s.units);
    if (c == 0 || cut - c < cut - share) return;   // nothing is cut here, or it began before
    const int pieces = (int)((cut - c + s.units - 1) / share) - (int)blockIdx.x + 1;
    const int h = item / s.tiles, tile = item - h * s.tiles;
    const int row0 = tile * R, seq_rows = s.n * a.group;
    const float gain_v = gain16 * (a.c.kv_type == TKV_INT4 && a.c.v_gain ? __ldg(a.c.v_gain + h) : 1.0f);
    const int d = (threadIdx.x % LANES) * 4;
    for (int row = threadIdx.x / LANES; row < R; row += kThreads / LANES) {
        if (row0 + row >= seq_rows) continue;
        const float* rec0 = a.part + ((int64_t)(blockIdx.x * 2 + 1) * R + row) * (D + 4);
        const int64_t next = (int64_t)2 * R * (D + 4);
        const float* rec1 = rec0 + (int64_t)R * (D + 4);   // record 0 of the next CTA
        float mm = kLowest, sum = 0.0f;
        float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll 4
        for (int i = 0; i < pieces; ++i) {
            const float* rec = i == 0 ? rec0 : rec1 + (i - 1) * next;
            const float2 v = *reinterpret_cast<const float2*>(rec + D);
            const float4 x = *reinterpret_cast<const float4*>(rec + d);
            const float mn = fmaxf(mm, v.x);
            const float f = exp2_approx(mm - mn), g = exp2_approx(v.x - mn);
            mm = mn;
            sum = sum * f + v.y * g;
            acc.x = acc.x * f + x.x * g;
            acc.y = acc.y * f + x.y * g;
            acc.z = acc.z * f + x.z * g;
            acc.w = acc.w * f + x.w * g;
        }
        const int t = (row0 + row) / a.group, g = row0 + row - t * a.group;
        const int64_t out_row = s.first_row + t;
        const int head = h * a.group + g;
        const float inv = sum == 0.0f ? 0.0f : gain_v / sum;
        uint16_t* to = reinterpret_cast<uint16_t*>(a.out) + out_row * a.out_row + head * a.out_head + d;
        uint2 w;
        if (!out_fp16) {
            const __nv_bfloat162 y0 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), y1 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
            w = make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
        } else {
            w = make_uint2(half2_bits(__floats2half2_rn(acc.x * inv, acc.y * inv)), half2_bits(__floats2half2_rn(acc.z * inv, acc.w * inv)));
        }
        *reinterpret_cast<uint2*>(to) = w;
        if (a.lse && d == 0)
            a.lse[out_row * a.hq + head] = sum == 0.0f ? -INFINITY : (mm + log2f(sum)) * 0.69314718056f;
    }
}

// ------------------------------------------------------------------ launch
// Row tiles are 8 rows, or 16 where a step brings more than 8 rows a KV head: the cache is then read and
// expanded once for twice the rows.
int row_tiles(int group, int max_new) { return (int64_t)group * max_new > 8 ? 2 : 1; }

cudaError_t device_ctas(int ctas, int* grid) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    *grid = ctas * sms;
    return e;
}

template <int D, int NT, int KIND>
cudaError_t launch(PagedAttnArgs& a, cudaStream_t st) {
    using C = Config<D, NT, KIND>;
    cudaError_t e = device_ctas(C::ctas, &a.grid);
    // the kernel's shared-memory limit, once a device
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(dev < 64 && (ready.load(std::memory_order_acquire) >> dev & 1))) {
        e = cudaFuncSetAttribute(paged_attention_kernel<D, NT, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
        if (e == cudaSuccess && dev < 64) ready.fetch_or((uint64_t)1 << dev, std::memory_order_release);
    }
    if (e != cudaSuccess) return e;
    paged_attention_kernel<D, NT, KIND><<<a.grid, kThreads, C::smem, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess || a.whole_items) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int out_fp16 = KIND == kFp16 || (KIND == kInt4 && a.q_fp16);
    return cudaLaunchKernelEx(&cfg, paged_combine_kernel<D, NT>, (const PagedAttnArgs)a, out_fp16, KIND == kInt4 ? 16.0f : 1.0f);
}

template <int D, int NT>
cudaError_t launch_kind(PagedAttnArgs& a, cudaStream_t st) {
    return a.c.kv_type == TKV_INT4   ? launch<D, NT, kInt4>(a, st)
           : a.c.kv_type == TKV_BF16 ? launch<D, NT, kBf16>(a, st)
                                     : launch<D, NT, kFp16>(a, st);
}

bool attention_shape_ok(const tkv_paged* c, int32_t hq, int32_t max_new) {
    return check_paged(c) == TKV_OK && hq >= 1 && hq % c->num_kv_heads == 0 && max_new >= 1;
}

}  // namespace

extern "C" int64_t tkv_paged_attention_workspace(const tkv_paged* cache, int32_t num_q_heads, int32_t max_new) {
    if (!attention_shape_ok(cache, num_q_heads, max_new)) return 0;
    int grid = 0;
    if (device_ctas(2, &grid) != cudaSuccess) {   // the most that any variant uses
        (void)cudaGetLastError();
        return 0;
    }
    return (int64_t)grid * 2 * 8 * row_tiles(num_q_heads / cache->num_kv_heads, max_new) * (cache->head_dim + 4) * 4;
}

extern "C" tkv_status tkv_paged_attention(const tkv_paged* cache, const void* q, void* out, float* lse, int32_t dtype,
                                          int64_t rows, int32_t num_q_heads, int64_t q_row_stride, int64_t q_head_stride,
                                          int64_t out_row_stride, int64_t out_head_stride, const int32_t* cu_tokens,
                                          int32_t max_new, int32_t max_len, int32_t window, float scale, void* workspace,
                                          int64_t workspace_bytes, int32_t* status, void* stream) {
    if (!attention_shape_ok(cache, num_q_heads, max_new) || max_len < 1 || window < 0 || !std::isfinite(scale)) return TKV_EINVAL;
    if (dtype != TKV_BF16 && dtype != TKV_FP16) return TKV_EINVAL;
    if (cache->kv_type != TKV_INT4 && cache->kv_type != dtype) return TKV_EINVAL;
    if (rows < 0 || rows > 0x7FFFFFFF || !cu_tokens) return TKV_EINVAL;
    if (rows == 0) return TKV_OK;
    // row indices within a sequence (queries x heads of a group) are 32-bit
    if (!q || !out || rows * (num_q_heads / cache->num_kv_heads) > 0x7FFF0000) return TKV_EINVAL;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || q_row_stride < 0 || q_head_stride < 0 || q_row_stride % 8 ||
        q_head_stride % 8 || out_row_stride % 8 || out_head_stride % 8)
        return TKV_EINVAL;
    if (!strides_apart(rows, out_row_stride, num_q_heads, out_head_stride, cache->head_dim)) return TKV_EINVAL;
    const int64_t need = tkv_paged_attention_workspace(cache, num_q_heads, max_new);
    if (need == 0) return TKV_ECUDA;
    if (!workspace || workspace_bytes < need) return TKV_ECAPACITY;
    PagedAttnArgs a{};
    a.c = *cache;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.cu = cu_tokens;
    a.part = reinterpret_cast<float*>(workspace);
    a.status = status;
    a.rows = rows;
    a.q_row = q_row_stride;
    a.q_head = q_head_stride;
    a.out_row = out_row_stride;
    a.out_head = out_head_stride;
    a.hq = num_q_heads;
    a.group = num_q_heads / cache->num_kv_heads;
    a.window = window;
    a.page_shift = __builtin_ctz((unsigned)cache->page_size);
    a.whole_items = max_len <= kWholeItems;
    a.q_fp16 = dtype == TKV_FP16;
    a.scale_log2 = (float)((double)scale * 1.4426950408889634);
    cudaStream_t st = (cudaStream_t)stream;
    const int nt = row_tiles(a.group, max_new);
    const cudaError_t e = cache->head_dim == 128 ? (nt == 1 ? launch_kind<128, 1>(a, st) : launch_kind<128, 2>(a, st))
                                                 : (nt == 1 ? launch_kind<64, 1>(a, st) : launch_kind<64, 2>(a, st));
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return TKV_ECUDA;
    }
    return TKV_OK;
}
