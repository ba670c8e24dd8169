// Beam search: tkv_beam_select (the best continuations over beams and vocabulary) and tkv_paged_reorder (the paged caches of all
// layers follow the beams that were chosen).
//
// Selection.  total[b, w, v] = scores[b, w] + x[b, w, v] - lse[b, w],  lse = log sum_v exp x;  the `count` largest over (w, v), the
// lower w V + v first where totals are equal.  Within a row (a beam's logits) the order is that of x itself, so a row's best `count`
// by (x, v) are all that it can bring.  One pass over the logits: a CTA takes a chunk of a row, 16 KB at a time in registers, and
// keeps per thread a running maximum and sum of exponentials, per CTA the best `count` so far.  A second kernel, started
// early, joins a sequence's chunks.
//
// The best of a chunk.  While the logits stream past, a thread only notes the maximum of each of its cells (its 32 values of a tile, of
// as many tiles as make 16 cells of the chunk): choosing from every tile, with its barriers, took 12 us of 39 for 512 rows of 131,072.
// Behind the stream the count-th largest maximum of all cells is a bound: no more than `count` cells lie above it, and only those
// and the ones that are equal to it can hold any of the best.  They are read once more.
// Where too many maxima are equal (a mask, say) the chunk is looked over tile by tile instead.  There, and where the chunk is one
// tile, the bound is the count-th largest of the maxima of groups of threads, each with its place, so that no two are equal:
// `count` values at least reach it, and only the `count` groups whose maxima do can hold any, so a quarter of a tile at most
// comes into the list, whatever the values are.
//
// What bounds it is memory, then issue: a 16-bit value costs three and a half instructions (half of a maximum, one to unpack, half a
// fused multiply-add, an exponential, half a sum).
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "paged.cuh"

using namespace tkv;

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCount = 64, kMaxBeams = 64;
constexpr int kVectors = 4;                       // 16-byte pieces of a thread and tile
constexpr int kCtas = 4;                          // on an SM at once, by their registers
constexpr int kCells = 16;                        // of a thread
constexpr int kIndexBits = 12;                    // of a candidate's index in its rank, in the joining kernel
constexpr int kMostCandidates = 1 << kIndexBits;  // of a sequence
constexpr int kMostGroups = kThreads;
constexpr int kFew = 64;                          // candidates of a sequence that are sorted whole
constexpr float kLog2E = 1.44269504f;
constexpr float kFar = 3e38f;
constexpr float kFloor = -3.402823466e38f;        // a maximum before anything is seen

struct Candidate {
    float x;
    int v;        // -1: none
};
struct Stat {
    float m, sum;   // of a chunk: the reference, and the sum of exp(x - m)
};

struct SelectArgs {
    const void* logits;
    const float* scores;
    const uint8_t* finished;      // may be null
    float* out_scores;
    int32_t* out_beams;
    int32_t* out_tokens;
    Stat* stats;                  // [batch * beams][chunks]
    Candidate* best;              // [batch * beams][chunks][count]
    int64_t batch_stride, beam_stride;
    int batch, beams, vocab, eos, count, chunks, per_chunk;
};

__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);   // -0 is 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_ordered(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o); }

// Larger is better: the value first, the lower place next.  0 is none.
__device__ __forceinline__ uint64_t key_of(float x, int v) { return (uint64_t)ordered(x) << 32 | (uint32_t)~v; }
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A beam that brings nothing of its logits: finished, or with a score that is not finite.
__device__ __forceinline__ bool is_out(const SelectArgs& a, int row) {
    return !(fabsf(a.scores[row]) < INFINITY) || (a.finished && a.finished[row]);
}

// *bound = the k-th largest of the maxima of groups of 2^shift threads (their keys are different where they are not 0; at least k
// groups have one).  A barrier follows before `bound` is read; `maxima` may be written again behind another.
__device__ __forceinline__ void kth_largest(uint64_t mine, int k, int shift, uint64_t (&maxima)[kMostGroups], uint64_t* bound) {
    for (int o = 1; o < 1 << shift; o <<= 1) mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, o));
    const int groups = kThreads >> shift, tid = threadIdx.x;
    if ((tid & ((1 << shift) - 1)) == 0) maxima[tid >> shift] = mine;
    __syncthreads();
    if (tid >= groups) return;
    mine = maxima[tid];
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i < groups; i += 2) {
        const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(maxima + i);
        rank += (two.x > mine) + (two.y > mine);
    }
    if (mine && rank == k - 1) *bound = mine;
}
// Groups are as large as leaves four times as many of them as wanted, and at least 8: their k largest then reach little further down
// than single threads' would, and k of them have at most kGroupThreads threads.
constexpr int kGroupThreads = 64;
__device__ __forceinline__ int group_shift(int k) { return min(5, 31 - __clz(kGroupThreads / k)); }

// How many groups have a thread with `has`, to every thread.
__device__ __forceinline__ int groups_with(bool has, int shift) {
    const int lane = threadIdx.x & 31, in_group = lane & ~((1 << shift) - 1);
    const uint32_t with = __ballot_sync(0xffffffffu, has), group = (shift == 5 ? 0xffffffffu : (1u << (1 << shift)) - 1) << in_group;
    return __syncthreads_count((lane == in_group) && (with & group));
}

// The best `count` of keys[0 .. n) (all different) into list, in order.  Barriers around it are the caller's.
__device__ __forceinline__ void sort_best(const uint64_t* keys, int n, int count, uint64_t* list) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t k = keys[i];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) rank += keys[j] > k;
        if (rank < count) list[rank] = k;
    }
}

// 16 bytes from `shift` elements (not 0) into two pieces on.
template <typename T>
__device__ __forceinline__ uint4 shifted(uint4 u, uint4 v, int shift) {
    const int words = shift * (int)sizeof(T) / 4, bits = sizeof(T) == 4 ? 0 : (shift & 1) * 16;
    uint32_t x0, x1, x2, x3, x4;
    if (words == 0) x0 = u.x, x1 = u.y, x2 = u.z, x3 = u.w, x4 = v.x;
    else if (words == 1) x0 = u.y, x1 = u.z, x2 = u.w, x3 = v.x, x4 = v.y;
    else if (words == 2) x0 = u.z, x1 = u.w, x2 = v.x, x3 = v.y, x4 = v.z;
    else x0 = u.w, x1 = v.x, x2 = v.y, x3 = v.z, x4 = v.w;
    return make_uint4(__funnelshift_r(x0, x1, bits), __funnelshift_r(x1, x2, bits), __funnelshift_r(x2, x3, bits), __funnelshift_r(x3, x4, bits));
}

// The values of a piece, two at a time.
template <typename T>
__device__ __forceinline__ float2 two_of(uint4 u, int i) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    else return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

// 16-bit values are compared two at a time.
template <typename T> struct Two { using type = float; };
template <> struct Two<__half> { using type = __half2; };
template <> struct Two<__nv_bfloat16> { using type = __nv_bfloat162; };
__device__ __forceinline__ float max2(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ __half2 max2(__half2 a, __half2 b) { return __hmax2(a, b); }
__device__ __forceinline__ __nv_bfloat162 max2(__nv_bfloat162 a, __nv_bfloat162 b) { return __hmax2(a, b); }
__device__ __forceinline__ float larger_of(float x) { return x; }
__device__ __forceinline__ float larger_of(__half2 x) { return fmaxf(__low2float(x), __high2float(x)); }
__device__ __forceinline__ float larger_of(__nv_bfloat162 x) { return fmaxf(__low2float(x), __high2float(x)); }
// Both halves as large as the least value of their type that is not below x.
template <typename P> __device__ __forceinline__ P both_at_least(float x);
template <> __device__ __forceinline__ float both_at_least<float>(float x) { return x; }
template <> __device__ __forceinline__ __half2 both_at_least<__half2>(float x) { return __half2half2(__float2half_ru(x)); }
template <> __device__ __forceinline__ __nv_bfloat162 both_at_least<__nv_bfloat162>(float x) { return __bfloat162bfloat162(__float2bfloat16_ru(x)); }
__device__ __forceinline__ uint32_t reach(float x, float low) { return x >= low ? 0xFFFFFFFFu : 0u; }
__device__ __forceinline__ uint32_t reach(__half2 x, __half2 low) { return __hge2_mask(x, low); }
__device__ __forceinline__ uint32_t reach(__nv_bfloat162 x, __nv_bfloat162 low) { return __hge2_mask(x, low); }

// The largest of a piece (of each half of its words); NaN counts only where nothing else is.
template <typename P>
__device__ __forceinline__ P largest_of(uint4 u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    const P* x = reinterpret_cast<const P*>(w);
    return max2(max2(x[0], x[1]), max2(x[2], x[3]));
}

// Which values of a piece reach `low`: bit j for the low half of word j, bit 16 + j for the high one; bit j for word j of 32 bits.
template <typename P>
__device__ __forceinline__ uint32_t at_least(uint4 u, P low) {
    constexpr uint32_t kBit = sizeof(P) == 4 && std::is_same<P, float>::value ? 1u : 0x00010001u;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    const P* x = reinterpret_cast<const P*>(w);
    return (reach(x[0], low) & kBit) | (reach(x[1], low) & kBit << 1) | (reach(x[2], low) & kBit << 2) | (reach(x[3], low) & kBit << 3);
}

// A bit's value, and its place in the piece.
template <typename T>
__device__ __forceinline__ float value_at(uint4 u, int bit) {
    const uint32_t w = bit & 2 ? (bit & 1 ? u.w : u.z) : (bit & 1 ? u.y : u.x);
    if constexpr (sizeof(T) == 4) return __uint_as_float(w);
    const uint16_t h = (uint16_t)(bit & 16 ? w >> 16 : w);
    return to_float(*reinterpret_cast<const T*>(&h));
}
template <typename T>
__device__ __forceinline__ int place_of(int bit) { return sizeof(T) == 4 ? bit : 2 * (bit & 3) + (bit >> 4); }

// A warp's part of the block's reference and sum, and, behind a barrier, all of it, to every thread.
__device__ __forceinline__ void sum_warp(float m, float sum, Stat (&stats)[kWarps]) {
    const float top = of_ordered(__reduce_max_sync(0xffffffffu, ordered(m)));
    sum *= exp2_fast((m - top) * kLog2E);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) stats[threadIdx.x >> 5] = Stat{top, sum};
}
__device__ __forceinline__ Stat sum_block(const Stat (&stats)[kWarps]) {
    Stat t{kFloor, 0.0f};
#pragma unroll
    for (int i = 0; i < kWarps; ++i) t.m = fmaxf(t.m, stats[i].m);
#pragma unroll
    for (int i = 0; i < kWarps; ++i) t.sum += stats[i].sum * exp2_fast((stats[i].m - t.m) * kLog2E);
    return t;
}

constexpr int kMost = kGroupThreads * 32 + kMaxCount;   // values in a list: what one tile can bring, and the best so far

// The best so far: a list that the CTA adds to and sorts.
struct Best {
    __align__(16) uint64_t keys[kMost];
    __align__(16) uint64_t maxima[kMostGroups];
    uint64_t list[kMaxCount], bound;
    int found;
    // of cells: how many come into question, how many hold the best, and the least of those cells' maxima, ordered
    int asked, placed;
    uint32_t lowest;
};

// What a thread knows of it.
struct Bound {
    float lowest;     // values below it are none of the best
    uint64_t least;   // and keys below this
    int held;         // in the list, sorted
};

__device__ __forceinline__ void add_key(Best& best, uint64_t k) {
    const int slot = atomicAdd(&best.found, 1);
    if ((uint32_t)slot < (uint32_t)kMost) best.keys[slot] = k;
}

// Adds a piece's values that reach the bound; v0: the place of its first.
template <typename T>
__device__ __forceinline__ void add_piece(Best& best, uint4 u, int v0, const Bound& b) {
    using P = typename Two<T>::type;
    for (uint32_t bits = at_least(u, both_at_least<P>(b.lowest)); bits; bits &= bits - 1) {
        const int bit = __ffs(bits) - 1;
        const float x = value_at<T>(u, bit);
        const uint64_t k = key_of(x, v0 + place_of<T>(bit));
        if (k >= b.least && x > -INFINITY) add_key(best, k);
    }
}

// A tile's part of the best: pieces p + i kThreads + tid.  Tiles come in order; ONLY: there is one, and a barrier follows.
template <typename T, bool ONLY>
__device__ __forceinline__ void look_over(Best& best, const uint4 (&raw)[kVectors], int p, int count, Bound& b) {
    using P = typename Two<T>::type;
    constexpr int E = 16 / sizeof(T);
    const int tid = threadIdx.x;
    P tops[kVectors];
#pragma unroll
    for (int i = 0; i < kVectors; ++i) tops[i] = largest_of<P>(raw[i]);
    const float top = larger_of(max2(max2(tops[0], tops[1]), max2(tops[2], tops[3])));
    const bool has = top > -INFINITY && top >= b.lowest;
    const int shift = group_shift(count), above = ONLY ? count + 1 : groups_with(has, shift);
    if (above == 0) return;
    if (above > count) {   // otherwise all of theirs come into the list
        int at = 0;                                        // the lowest place of the largest
#pragma unroll
        for (int i = kVectors - 1; i >= 0; --i) {
            const uint32_t bits = at_least(raw[i], both_at_least<P>(top));
            const int low = place_of<T>(__ffs(bits) - 1), high = sizeof(T) == 2 && bits >> 16 ? place_of<T>(__ffs(bits >> 16) + 15) : E;
            if (bits) at = (p + i * kThreads + tid) * E + min(sizeof(T) == 2 && !(bits & 0xFFFFu) ? E : low, high);
        }
        kth_largest(has ? key_of(top, at) : 0, count, shift, best.maxima, &best.bound);
        __syncthreads();
        if (best.bound > b.least) {
            b.least = best.bound;
            b.lowest = of_ordered((uint32_t)(b.least >> 32));
        }
    }
    if (top >= b.lowest && top > -INFINITY) {
#pragma unroll
        for (int i = 0; i < kVectors; ++i)
            if (larger_of(tops[i]) >= b.lowest) add_piece<T>(best, raw[i], (p + i * kThreads + tid) * E, b);
    }
    __syncthreads();
    const int n = best.found;
    sort_best(best.keys, n, count, best.list);
    b.held = min(n, count);
    if (ONLY) return;
    __syncthreads();
    if (b.held == count) {
        b.least = best.list[count - 1] + 1;
        b.lowest = of_ordered((uint32_t)(best.list[count - 1] >> 32) + 1);   // the next number: what is equal comes too late
    }
    if (tid < b.held) best.keys[tid] = best.list[tid];
    if (tid == 0) best.found = b.held;
    __syncthreads();
}

// blockIdx.x: chunk, blockIdx.y (and z, behind 65,535 rows): row.
template <typename T>
__global__ void __launch_bounds__(kThreads, kCtas) select_rows_kernel(const __grid_constant__ SelectArgs a) {
    using P = typename Two<T>::type;
    constexpr int E = 16 / sizeof(T);                           // values of a piece
    constexpr int kTile = kVectors * kThreads;                  // pieces
    __shared__ Best best;
    __shared__ float cells[kCells][kThreads];
    __shared__ Stat stats[kWarps];
    wait_for_previous();
    let_next_start();   // not earlier: the joining kernel reads scores and finished before its own wait
    const int row = blockIdx.y + blockIdx.z * 65535, tid = threadIdx.x;
    if (row >= a.batch * a.beams) return;
    const int seq = row / a.beams, w = row - seq * a.beams;
    const T* x0 = reinterpret_cast<const T*>(a.logits) + seq * a.batch_stride + w * a.beam_stride;
    // Piece p is values p E .. p E + E - 1 of the row wherever the row begins, so that equal rows have equal sums: of a row that does not
    // begin on 16 bytes it is put together from two of memory's pieces.
    const int shift = (int)((reinterpret_cast<uintptr_t>(x0) & 15) / sizeof(T));
    const uint4* memory = reinterpret_cast<const uint4*>(x0 - shift);
    const int first = blockIdx.x * a.per_chunk, end = min(first + a.per_chunk, (a.vocab + E - 1) / E);
    const int whole = shift ? (a.vocab + shift) / E - 1 : a.vocab / E;   // pieces before it (and behind 0, if shifted) are read whole
    constexpr uint32_t kNone = sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;   // -infinity
    auto load = [&](int p) {
        uint4 u = make_uint4(kNone, kNone, kNone, kNone);
        if (p >= end) return u;
        if (p < whole && (p > 0 || !shift)) return shift ? shifted<T>(memory[p], memory[p + 1], shift) : memory[p];
        Vec16<T> part;
        part.u = u;
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (p * E + i < a.vocab) part.e[i] = x0[p * E + i];
        return part.u;
    };
    // The thread's maximum m and sum of 2^(x log2 e - c), c = m log2 e rounded: one fused multiply-add a pair.  Beyond 3e38 c stays there
    // and the sum is 0 or infinite: the row is then added up again below.
    float m = kFloor, c = -kFar, sum = 0.0f;
    uint4 raw[kVectors], next[kVectors];
#pragma unroll
    for (int i = 0; i < kVectors; ++i) next[i] = load(first + i * kThreads + tid);
    bool apart = false;   // next holds memory's pieces, of a row that does not begin on 16 bytes: put together when they are there
    if (is_out(a, row)) return;
    if (tid == 0) {
        best.found = best.asked = best.placed = 0;
        best.lowest = 0xFFFFFFFFu;
        best.bound = 0;
    }
    const int tiles = (end - first + kTile - 1) / kTile, span = (tiles + kCells - 1) / kCells;   // tiles of a cell
    float cell = -INFINITY;
    int in_cell = 0, cell_at = tid;
#pragma unroll 1
    for (int p = first; p < end; p += kTile) {
#pragma unroll
        for (int i = 0; i < kVectors; ++i) raw[i] = next[i];
        if (apart) {
#pragma unroll
            for (int i = 0; i < kVectors; ++i) {
                uint4 v = make_uint4(__shfl_down_sync(0xffffffffu, raw[i].x, 1), __shfl_down_sync(0xffffffffu, raw[i].y, 1),
                                     __shfl_down_sync(0xffffffffu, raw[i].z, 1), __shfl_down_sync(0xffffffffu, raw[i].w, 1));
                if ((tid & 31) == 31) v = memory[p + i * kThreads + tid + 1];
                raw[i] = shifted<T>(raw[i], v, shift);
            }
        }
        apart = shift && p + 2 * kTile <= min(end, whole);
        if (p + 2 * kTile <= min(end, whole)) {
#pragma unroll
            for (int i = 0; i < kVectors; ++i) next[i] = memory[p + kTile + i * kThreads + tid];
        } else {
#pragma unroll
            for (int i = 0; i < kVectors; ++i) next[i] = load(p + kTile + i * kThreads + tid);
        }
        P tops = largest_of<P>(raw[0]);
#pragma unroll
        for (int i = 1; i < kVectors; ++i) tops = max2(tops, largest_of<P>(raw[i]));
        const float top = larger_of(tops);
        cell = fmaxf(cell, top);
        if (++in_cell == span) {
            (&cells[0][0])[cell_at] = cell;
            cell_at += kThreads;
            in_cell = 0;
            cell = -INFINITY;
        }
        if (top > m) {
            const float z = fminf(fmaxf(top * kLog2E, -kFar), kFar);
            sum *= exp2_fast(c - z);
            m = top;
            c = z;
        }
        F2 s[2] = {f2(0.0f, 0.0f), f2(0.0f, 0.0f)};
        const F2 minus = f2(-c, -c), log2e = f2(kLog2E, kLog2E);
#pragma unroll
        for (int i = 0; i < kVectors; ++i)
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                const float2 x = two_of<T>(raw[i], j), y = parts(fma2(f2(x.x, x.y), log2e, minus));
                s[j & 1] = add2(s[j & 1], f2(exp2_fast(y.x), exp2_fast(y.y)));
            }
        const float2 both = parts(add2(s[0], s[1]));
        sum += both.x + both.y;
    }
    if (in_cell) (&cells[0][0])[cell_at] = cell;
    // ---- the chunk's reference and sum
    if (fabsf(c) < kFar) sum *= exp2_fast(-fmaf(m, kLog2E, -c));   // from c to m
    sum_warp(m, sum, stats);
    // ---- the best
    Bound b{-INFINITY, 0, 0};
    bool by_tiles = false;
    if (tiles == 1) {
        look_over<T, true>(best, raw, first, a.count, b);
    } else {
        // A bound from below: `count` groups of threads have a value that reaches it.  Then the cells that do.
        const int used = (tiles + span - 1) / span;
        kth_largest(m > kFloor ? (uint64_t)ordered(m) << 32 | (uint32_t)~tid : 0, a.count, group_shift(a.count), best.maxima, &best.bound);
        __syncthreads();
        const float low = best.bound ? of_ordered((uint32_t)(best.bound >> 32)) : -INFINITY;   // 0: fewer groups have any
        uint32_t* asked = reinterpret_cast<uint32_t*>(best.keys);   // maxima of cells, ordered, and
        uint32_t* cell_of = asked + kMost;                          // the cells
        if (m >= low)
            for (int i = 0; i < used; ++i) {
                const float x = cells[i][tid];
                if (x >= low && x > -INFINITY) {
                    const int slot = atomicAdd(&best.asked, 1);
                    if (slot < kMost) {
                        asked[slot] = ordered(x);
                        cell_of[slot] = i * kThreads + tid;
                    }
                }
            }
        __syncthreads();
        const int n = best.asked;
        by_tiles = n > kMost;
        if (!by_tiles) {
            // Those that fewer than `count` others exceed hold the best.
            int* places = reinterpret_cast<int*>(best.maxima);
            constexpr int kPlaces = sizeof(best.maxima) / sizeof(int);
            for (int i = tid; i < n; i += kThreads) {
                const uint32_t x = asked[i];
                int above = 0, j = 0;
#pragma unroll 4
                for (; j + 4 <= n; j += 4) {
                    const uint4 u = *reinterpret_cast<const uint4*>(asked + j);
                    above += (u.x > x) + (u.y > x) + (u.z > x) + (u.w > x);
                }
                for (; j < n; ++j) above += asked[j] > x;
                if (above < a.count) {
                    const int slot = atomicAdd(&best.placed, 1);
                    if (slot < kPlaces) places[slot] = (int)cell_of[i];
                    atomicMin(&best.lowest, x);
                }
            }
            __syncthreads();
            const int placed = best.placed;
            by_tiles = placed > kPlaces;
            if (!by_tiles) {
                if (n >= a.count) b.lowest = of_ordered(best.lowest);   // the count-th largest cell's
                for (int i = tid; i < placed * span * kVectors; i += kThreads) {
                    const int cell_at = places[i / (span * kVectors)], in = i % (span * kVectors);
                    const int q = first + (cell_at / kThreads * span + in / kVectors) * kTile + in % kVectors * kThreads + cell_at % kThreads;
                    add_piece<T>(best, load(q), q * E, b);
                }
                __syncthreads();
                const int found = best.found;
                by_tiles = found > kMost;
                if (!by_tiles) {
                    sort_best(best.keys, found, a.count, best.list);
                    b.held = min(found, a.count);
                }
            }
        }
        if (by_tiles) {
            __syncthreads();   // everyone has read it
            if (tid == 0) best.found = best.bound = 0;
            b = Bound{-INFINITY, 0, 0};
            __syncthreads();
            for (int p = first; p < end; p += kTile) {
#pragma unroll
                for (int i = 0; i < kVectors; ++i) raw[i] = load(p + i * kThreads + tid);
                look_over<T, false>(best, raw, p, a.count, b);
            }
        }
    }
    __syncthreads();
    const int64_t at = (int64_t)row * a.chunks + blockIdx.x;
    Stat t = sum_block(stats);
    if (b.held && !(t.sum > 0.0f && t.sum < INFINITY)) {   // the largest beyond 2e38 either way, or a NaN or an infinity: the slow way
        m = of_ordered((uint32_t)(best.list[0] >> 32));
        sum = 0.0f;
        for (int p = first + tid; p < end; p += kThreads) {
            const uint4 u = load(p);
            for (int j = 0; j < E / 2; ++j) {
                const float2 x = two_of<T>(u, j);
                sum += exp2_fast((x.x - m) * kLog2E) + exp2_fast((x.y - m) * kLog2E);
            }
        }
        __syncthreads();
        sum_warp(m, sum, stats);
        __syncthreads();
        t = sum_block(stats);
    }
    if (tid == 0) a.stats[at] = t;
    if (tid < a.count) {
        const uint64_t k = best.list[tid];
        a.best[at * a.count + tid] = tid < b.held ? Candidate{of_ordered((uint32_t)(k >> 32)), (int)~(uint32_t)k} : Candidate{0.0f, -1};
    }
}

// ------------------------------------------------------------------ joining
// A row's sum and its logarithm are sums of two fp32 numbers, good to 2^-46 or so: fp64 instructions are few and slow here (20 us for a
// kernel with them throughout).  sum_of is Knuth's exact sum of two numbers, plus the usual sum of two double-length
// numbers (after Dekker), and log_of splits ln 2 as Cody and Waite do.
struct Wide {
    float hi, lo;   // hi is the nearest to hi + lo
};
__device__ __forceinline__ Wide sum_of(float a, float b) {   // exactly
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return Wide{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Wide plus(Wide a, Wide b) {
    const Wide s = sum_of(a.hi, b.hi), t = sum_of(a.lo, b.lo);
    const float e = __fadd_rn(s.lo, t.hi), h = __fadd_rn(s.hi, e), l = __fadd_rn(__fsub_rn(e, __fsub_rn(h, s.hi)), t.lo);
    const float hi = __fadd_rn(h, l);
    return Wide{hi, __fsub_rn(l, __fsub_rn(hi, h))};
}
// log x, x > 0 and finite: its power of two apart, so that what logf rounds lies below 0.35.
__device__ __forceinline__ Wide log_of(float x) {
    const int e = ((int)(__float_as_uint(x) - 0x3F3504F3u) >> 23);                     // x = m 2^e, m in [sqrt 1/2, sqrt 2)
    const float m = __int_as_float(__float_as_int(x) - (e << 23)), k = (float)e;
    return plus(sum_of(__fmul_rn(k, 0.693145751953125f), __fmul_rn(k, 1.42860682030941723e-6f)), Wide{logf(m), 0.0f});   // ln 2 in 16 bits, and the rest
}

// A candidate's rank.  Its total is (x - reference) + offset, two roundings to 64 bits that never turn the order of a row's x round, so
// what is equal there is left to the logit itself: the larger total comes first, then the lower beam, the larger x, and the lower
// candidate, whose token is lower where x is equal too.  All zeros: none.
struct __align__(16) Rank {
    uint64_t total, rest;
};
__device__ __forceinline__ bool precedes(Rank a, Rank b) { return a.total > b.total || (a.total == b.total && a.rest > b.rest); }
__device__ __forceinline__ uint64_t ordered(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x);
    return u >> 63 ? ~u + (u << 1 == 0) : u | 1ull << 63;   // -0 is 0
}
__device__ __forceinline__ double of_ordered(uint64_t o) { return __longlong_as_double((long long)(o >> 63 ? o & ~(1ull << 63) : ~o)); }

constexpr int kMostRanks = 512;
static_assert(kMostRanks >= kMaxCount + kThreads, "the best so far and a candidate of each thread");

// *bound = the k-th largest of the maxima of groups of 2^shift threads, if so many are not 0.  A barrier follows before it is read.
__device__ __forceinline__ void kth_largest(uint32_t mine, int k, int shift, uint32_t (&maxima)[kMostGroups], uint32_t* bound) {
    for (int o = 1; o < 1 << shift; o <<= 1) mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, o));
    const int groups = kThreads >> shift, tid = threadIdx.x;
    if ((tid & ((1 << shift) - 1)) == 0) maxima[tid >> shift] = mine;
    __syncthreads();
    if (tid >= groups) return;
    mine = maxima[tid];
    int above = 0, equal = 0;
#pragma unroll 2
    for (int i = 0; i < groups; i += 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(maxima + i);
        above += (u.x > mine) + (u.y > mine) + (u.z > mine) + (u.w > mine);
        equal += (u.x == mine) + (u.y == mine) + (u.z == mine) + (u.w == mine);
    }
    if (mine && above < k && above + equal >= k) *bound = mine;   // all that are equal write the same
}

// One CTA a sequence.  Candidates are counted by beam, chunk and place in the chunk's list.  Which of them come into question is found in 32
// bits, with room for what these round; only those get a rank, as an SM does two operations of 64 bits a cycle (0.1 to 0.3 us of the call).
// The shared memory is kept below 16 KB: with 24 an SM that has run the main kernel is divided anew for this one, and the call for 64 x 8
// beams of 131,072, 16 chosen, took 36.1 us instead of 31.8, for 16 x 4 of 32,000, 8 chosen, 13.2 instead of 9.8.
__global__ void __launch_bounds__(kThreads) select_join_kernel(const __grid_constant__ SelectArgs a) {
    __shared__ float reference[kMaxBeams], score_of[kMaxBeams];
    __shared__ bool is_done[kMaxBeams];
    __shared__ Wide offset[kMaxBeams];                            // total = (x - reference) + offset; NaN: the beam offers none
    __shared__ double offset64[kMaxBeams], reference64[kMaxBeams];
    __shared__ __align__(16) uint32_t maxima[kMostGroups];
    __shared__ Rank ranks[kMostRanks];                            // at first x and the candidate's number
    __shared__ int tokens[kMostRanks];
    __shared__ uint32_t least;
    __shared__ int found, none;
    const int b = blockIdx.x, tid = threadIdx.x, per_row = a.chunks * a.count, n = a.beams * per_row;
    const Candidate* best = a.best + (int64_t)b * n;
    for (int w = tid; w < a.beams; w += kThreads) {               // what precedes the main kernel has been done before this one starts
        const int row = b * a.beams + w;
        score_of[w] = __ldcg(a.scores + row);
        is_done[w] = a.finished && __ldcg(a.finished + row);
    }
    __syncthreads();
    wait_for_previous();
    // the thread's first candidates, while the sums are on their way
    constexpr int kEarly = 2;
    Candidate early[kEarly];
#pragma unroll
    for (int k = 0; k < kEarly; ++k) early[k] = tid + k * kThreads < n ? best[tid + k * kThreads] : Candidate{0.0f, -1};
    const int lanes = a.chunks > 16 ? 32 : a.chunks > 8 ? 16 : a.chunks > 4 ? 8 : a.chunks > 2 ? 4 : a.chunks;   // of a beam
    const int mine_of = tid & (lanes - 1);
    for (int from = 0; from < a.beams; from += kThreads / lanes) {
        const int w = from + tid / lanes;
        const Stat* s = a.stats + ((int64_t)b * a.beams + min(w, a.beams - 1)) * a.chunks;   // of a beam that is out: anything
        float top = kFloor;
        for (int i = mine_of; i < a.chunks; i += lanes) top = fmaxf(top, s[i].m);
        for (int d = lanes / 2; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        Wide sum{0.0f, 0.0f};
        for (int i = mine_of; i < a.chunks; i += lanes) sum = plus(sum, Wide{s[i].sum * exp2_fast((s[i].m - top) * kLog2E), 0.0f});
        for (int d = lanes / 2; d; d >>= 1) sum = plus(sum, Wide{__shfl_xor_sync(0xffffffffu, sum.hi, d), __shfl_xor_sync(0xffffffffu, sum.lo, d)});
        if (w < a.beams && mine_of == 0) {
            const float score = score_of[w];
            Wide o{NAN, 0.0f};
            if (fabsf(score) < INFINITY) {
                if (is_done[w]) {
                    o = Wide{score, 0.0f};
                } else if (sum.hi > 0.0f && sum.hi < INFINITY) {   // not: a NaN or an infinity among the logits, or nothing above -infinity
                    const Wide l = plus(log_of(sum.hi), Wide{__fdividef(sum.lo, sum.hi), 0.0f});
                    o = plus(Wide{score, 0.0f}, Wide{-l.hi, -l.lo});
                }
            }
            reference[w] = top;
            offset[w] = o;
        }
    }
    if (tid == 0) {
        found = none = 0;
        least = ordered(-INFINITY);
    }
    __syncthreads();
    const uint32_t by_row = ((1u << 24) + per_row - 1) / per_row;   // i * by_row >> 24 = i / per_row, as i < 64 per_row and i per_row < 2^24
    // Candidate i of the sequence: whether it is one, and what its total is at least and at most.  Thread t takes t, t + 256, ..
    auto bounds_of = [&](int i, Candidate c, float* low, float* high) -> bool {
        const int w = (int)(i * by_row >> 24);
        const float o = offset[w].hi;
        const bool done = is_done[w];
        if (isnan(o) || (done ? i != w * per_row : c.v < 0)) return false;
        const float x = done ? 0.0f : c.x - reference[w], t = x + o;
        const float off = (fabsf(x) + fabsf(o)) * 0x1p-22f;   // x, t and the offset are rounded by 2^-24 of themselves, *low and *high too
        *low = t - off;
        *high = fabsf(t) < INFINITY ? t + off : INFINITY;
        return true;
    };
    uint32_t mine = 0;
    float top = -INFINITY;
    auto consider = [&](int i, Candidate c) {
        float low, high = NAN;
        if (!bounds_of(i, c, &low, &high)) return high;
        mine = max(mine, ordered(low));
        top = fmaxf(top, high);
        return high;
    };
    float early_high[kEarly];
#pragma unroll
    for (int k = 0; k < kEarly; ++k) early_high[k] = tid + k * kThreads < n ? consider(tid + k * kThreads, early[k]) : NAN;
#pragma unroll 1
    for (int i = tid + kEarly * kThreads; i < n; i += 4 * kThreads) {   // a few at once
        Candidate c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = i + k * kThreads < n ? best[i + k * kThreads] : Candidate{0.0f, -1};
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
            if (i + k * kThreads < n) consider(i + k * kThreads, c[0]);
            c[0] = c[1];
            c[1] = c[2];
            c[2] = c[3];
        }
    }
    // few candidates are sorted as they are
    if (n > kFew) kth_largest(mine, a.count, group_shift(a.count), maxima, &least);
    if (tid >= kThreads - a.beams) {   // the last warps, which have less to do there
        const int w = kThreads - 1 - tid;
        reference64[w] = reference[w];
        offset64[w] = (double)offset[w].hi + (double)offset[w].lo;
    }
    __syncthreads();
    auto take = [&](int i, Candidate c) {
        const int slot = atomicAdd(&found, 1);
        if (slot >= kMostRanks) return;
        ranks[slot] = Rank{__float_as_uint(c.x), (uint64_t)i};
        tokens[slot] = c.v;
    };
    const float reach = of_ordered(least);
    if (top >= reach) {
        auto add = [&](int i, Candidate c) {
            float low, high;
            if (bounds_of(i, c, &low, &high) && high >= reach) take(i, c);
        };
#pragma unroll
        for (int k = 0; k < kEarly; ++k)
            if (early_high[k] >= reach) take(tid + k * kThreads, early[k]);
        for (int i = tid + kEarly * kThreads; i < n; i += kThreads) add(i, best[i]);
    }
    __syncthreads();
    auto rank_of = [&](int i, Candidate c) -> Rank {
        const int w = (int)(i * by_row >> 24);
        const bool done = is_done[w];
        if (done ? i != w * per_row : c.v < 0) return Rank{0, 0};
        const float x = done ? 0.0f : c.x;
        const double o = offset64[w], t = done ? o : ((double)x - reference64[w]) + o;
        if (!(fabs(t) < 0x1.ffffffp+127)) return Rank{0, 0};   // none, or below the lowest number of 32 bits
        return Rank{ordered(t), (uint64_t)(kMaxBeams - 1 - w) << (32 + kIndexBits) | (uint64_t)ordered(x) << kIndexBits | (uint32_t)(kMostCandidates - 1 - i)};
    };
    int m = found;
    if (m <= kMostRanks) {
        for (int i = tid; i < m; i += kThreads) {
            const Rank r = ranks[i] = rank_of((int)ranks[i].rest, Candidate{__uint_as_float((uint32_t)ranks[i].total), tokens[i]});
            if (!r.total) atomicAdd(&none, 1);
        }
        __syncthreads();
    } else {   // as many that are equal or nearly: a candidate of each thread joins the best so far, and so on
        m = 0;
        for (int i = tid; i - tid < n; i += kThreads) {
            __syncthreads();
            if (tid == 0) found = m;
            __syncthreads();
            const Candidate c = i < n ? best[i] : Candidate{0.0f, -1};
            const Rank r = i < n ? rank_of(i, c) : Rank{0, 0};
            if (r.total && (m < a.count || precedes(r, ranks[a.count - 1]))) {
                const int slot = atomicAdd(&found, 1);
                ranks[slot] = r;
                tokens[slot] = c.v;
            }
            __syncthreads();
            const int all = found;
            Rank kept[2];
            int token[2], place[2] = {kMaxCount, kMaxCount};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int j = tid + k * kThreads;
                if (j >= all) continue;
                kept[k] = ranks[j];
                token[k] = tokens[j];
                place[k] = 0;
                for (int q = 0; q < all; ++q) place[k] += precedes(ranks[q], kept[k]);
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (place[k] < a.count) {
                    ranks[place[k]] = kept[k];
                    tokens[place[k]] = token[k];
                }
            m = min(all, a.count);
        }
        __syncthreads();
    }
    const int64_t out = (int64_t)b * a.count;
    const int each = m <= kThreads / 4 ? 4 : m <= kThreads / 2 ? 2 : 1;   // threads of a candidate
    for (int from = 0; from < m * each; from += kThreads) {
        const int i = (from + tid) / each;
        const Rank r = i < m ? ranks[i] : Rank{0, 0};
        int rank = 0;
        if (r.total) {
#pragma unroll 4
            for (int j = tid & (each - 1); j < m; j += each) rank += precedes(ranks[j], r);
        }
        for (int o = each / 2; o; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
        if (rank >= a.count || !r.total || (tid & (each - 1))) continue;
        const int w = kMaxBeams - 1 - (int)(r.rest >> (32 + kIndexBits));
        a.out_scores[out + rank] = (float)of_ordered(r.total);
        a.out_beams[out + rank] = w;
        a.out_tokens[out + rank] = is_done[w] ? a.eos : tokens[i];
    }
    for (int i = m - none + tid; i < a.count; i += kThreads) {
        a.out_scores[out + i] = -INFINITY;
        a.out_beams[out + i] = a.out_tokens[out + i] = -1;
    }
}

// How the rows are cut: as many CTAs as the device holds at once, chunks of 512 pieces at least, and no more candidates than the
// joining kernel takes.  With c chunks a row, a chunk's stream takes about 0.4 ns for each of its pieces / c pieces and joining 3 ns for
// each of beams count c candidates: the sum is least at c = sqrt(pieces / (8 beams count)).  Up to a candidate a thread joining costs the
// same, so with no more than two CTAs an SM there are as many chunks as that allows (4 beams of 32,000, 8 chosen: 7.5 us with 8 chunks, 8.2
// with the 4 of the root).  One sequence of 8 beams of 131,072, 16 of
// them chosen: 11.2 us with 4 chunks, 18.8 with the most, 32; 2 x 5 beams of 100,003 in fp32, 10 chosen: 12.7 and 15.9.
struct Split {
    int chunks, per_chunk;   // pieces of a chunk
};
Split split_rows(int64_t rows, int beams, int vocab, int count, int element, int sms) {
    const int pieces = (vocab + 16 / element - 1) / (16 / element);
    int64_t chunks = std::max<int64_t>(1, (int64_t)sms * kCtas / rows);
    chunks = std::min<int64_t>(chunks, (pieces + 2 * kThreads - 1) / (2 * kThreads));
    chunks = std::min<int64_t>(chunks, std::max(1, kMostCandidates / (beams * count)));
    const int64_t balanced = std::llrint(std::sqrt(pieces / (8.0 * beams * count)));
    const int64_t cheap = std::min<int64_t>(kThreads / (beams * count), 2 * sms / rows);
    chunks = std::min(chunks, std::max<int64_t>({1, balanced, cheap}));
    Split s;
    s.per_chunk = (int)((pieces + chunks - 1) / chunks);
    s.chunks = (pieces + s.per_chunk - 1) / s.per_chunk;
    return s;
}

int64_t select_bytes(int64_t rows, int chunks, int count) { return (rows * chunks * (int64_t)(sizeof(Stat) + count * sizeof(Candidate)) + 15) / 16 * 16; }

bool select_shape_ok(int dtype, int64_t batch, int beams, int vocab, int count) {
    return is_dtype(dtype) && batch >= 0 && batch <= 0x7FFFFFFF && beams >= 1 && beams <= kMaxBeams && vocab >= 1 && count >= 1 && count <= kMaxCount &&
           beams * count <= kMostCandidates && (int64_t)beams * vocab <= 0x7FFFFF00 && batch * beams <= 0x7FFFFFFF / 64;
}

cudaError_t device_sms(int* sms) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return e == cudaSuccess ? cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) : e;
}

// ------------------------------------------------------------------ reordering
// The beams of a sequence go on from one another's caches: columns of the page table before the current page are exchanged, and
// what the current, partly filled page holds is copied.  All beams of a thread's piece are read before any is written, so
// a permutation needs no second buffer.  Pages before the current one are only read from then on, so that beams may share them.
// The current page is the same in all caches, so a CTA serves one sequence of beams in all caches of a launch, which have one shape: it
// reads the sequence's parents, lengths and pages once (three trips to memory in a row) and walks over 16-byte pieces, those of one cache
// behind those of the last.  With CTAs of one cache each, 7 layers of 8 x 12 beams took 36.2 us instead of 15.8, and 32 layers of two
// positions in pages of 128 22 instead of 5.3.
constexpr int kMaxCaches = 128;   // of a launch: 2 KB of arguments

struct ReorderArgs {
    uint8_t* pages[kMaxCaches];
    int64_t num_pages[kMaxCaches];
    int32_t* table;
    const int32_t* lengths;
    const int32_t* parents;
    int32_t* status;
    int64_t groups, least_pages;   // sequences of beams; the least of num_pages
    int64_t head_bytes;            // of a page
    int num_caches, beams, max_pages, page_shift;
    int heads;
    int parts;                     // of a head's page that hold positions: 1 (records), or K and V
    int unit;                      // bytes of a part's `per` positions
    int per;
    int split, table_split;        // CTAs of a sequence; of its table (0: the table stays)
};

// CTAs of an SM, by the registers of a piece of W beams.
template <int W>
constexpr int reorder_ctas() { return W <= 4 ? 8 : W <= 8 ? 4 : W == 16 ? 2 : 1; }

template <int W>
__global__ void __launch_bounds__(kThreads, reorder_ctas<W>()) reorder_kernel(const __grid_constant__ ReorderArgs a) {
    __shared__ int page[W], length, last_page;
    __shared__ uint32_t children[W];   // beams that go on from this one, itself not among them
    let_next_start();
    wait_for_previous();
    const int tid = threadIdx.x;
    int64_t unit = blockIdx.x;
    const int64_t copies = a.groups * a.split;
    const bool is_table = unit >= copies;
    if (is_table) unit -= copies;
    const int parts_of = is_table ? a.table_split : a.split, part = (int)(unit % parts_of);
    const int64_t group = unit / parts_of;
    if (tid < 32) {   // a lane a beam
        const int64_t seq = group * a.beams + tid;
        const bool is_beam = tid < a.beams;
        int p = is_beam ? a.parents[seq] : -1;
        const int mine = is_beam ? a.lengths[seq] : 0, len = __shfl_sync(0xffffffffu, mine, 0);
        const int column = len >> a.page_shift, rest = len & ((1 << a.page_shift) - 1);
        const bool fits = len >= 0 && (column < a.max_pages || (column == a.max_pages && rest == 0));
        const bool same = __all_sync(0xffffffffu, !is_beam || mine == len), has_page = is_beam && fits && rest && !is_table;
        const int pg = has_page ? a.table[seq * a.max_pages + column] : -1;
        int report = !same ? TKV_EINVAL : !fits ? TKV_ECAPACITY : TKV_OK;
        if (p >= a.beams) {
            report = max(report, (int)TKV_EINVAL);
            p = -1;
        }
        if (p < 0) p = tid;   // none: it stays
        const int from = __shfl_sync(0xffffffffu, pg, p);
        const bool goes = is_beam && p != tid && same && fits && (is_table || (rest && from != pg));
        if (report != TKV_OK && part == 0) raise_status(a.status, report);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const uint32_t of = __ballot_sync(0xffffffffu, goes && p == i);
            if (tid == i) children[i] = of;
        }
        const uint32_t last = __reduce_max_sync(0xffffffffu, goes ? max((uint32_t)from, (uint32_t)pg) : 0u);
        if (tid < W) page[tid] = pg;
        if (tid == 0) {
            length = len;
            last_page = (int)last;
        }
    }
    __syncthreads();
    const int len = length, column = len >> a.page_shift, rest = len & ((1 << a.page_shift) - 1);
    uint32_t kids[W];
    bool any = false;
#pragma unroll
    for (int p = 0; p < W; ++p) {
        kids[p] = children[p];
        any |= kids[p] != 0;
    }
    if (!any) return;
    const uint32_t at = part * kThreads + tid, step = parts_of * kThreads;
    if (is_table) {
        int32_t* table = a.table + group * a.beams * a.max_pages;
        for (int i = at; i < column; i += step) {
            int v[W];
#pragma unroll
            for (int p = 0; p < W; ++p)
                if (kids[p]) v[p] = table[(int64_t)p * a.max_pages + i];
#pragma unroll
            for (int p = 0; p < W; ++p)
                for (uint32_t k = kids[p]; k; k &= k - 1) table[(int64_t)(__ffs(k) - 1) * a.max_pages + i] = v[p];
        }
        return;
    }
    const bool all_there = (uint32_t)last_page < (uint64_t)a.least_pages;
    if (!all_there && part == 0 && tid == 0) raise_status(a.status, TKV_ECAPACITY);
    const uint32_t pieces = (rest + a.per - 1) / a.per * (a.unit / 16);   // of a part
    const uint32_t total = pieces * a.parts * a.heads;                   // of a cache, below 2^31: i + step fits
    const int64_t part_bytes = a.head_bytes / a.parts, page_bytes = a.head_bytes * a.heads;
    uint32_t n = at / total, i = at - n * total;                         // cache, piece
#pragma unroll 1
    while (n < (uint32_t)a.num_caches) {
        uint32_t there = ~0u;   // beams whose page there is
        if (!all_there) {
            for (int b = 0; b < a.beams; ++b)
                if ((uint32_t)page[b] >= (uint64_t)a.num_pages[n]) there &= ~(1u << b);
        }
        const uint32_t q = i / pieces;                                   // head and part
        uint8_t* to = a.pages[n] + q * part_bytes + (int64_t)(i - q * pieces) * 16;
        uint4 v[W];
#pragma unroll
        for (int p = 0; p < W; ++p)
            if (kids[p] && there >> p & 1) v[p] = *reinterpret_cast<const uint4*>(to + page[p] * page_bytes);
#pragma unroll
        for (int p = 0; p < W; ++p)
            if (there >> p & 1)
                for (uint32_t k = kids[p] & there; k; k &= k - 1) *reinterpret_cast<uint4*>(to + page[__ffs(k) - 1] * page_bytes) = v[p];
        i += step;
        const uint32_t further = i / total;
        n += further;
        i -= further * total;
    }
}

// Caches whose pages are moved alike: bf16 and fp16 are.
bool same_shape(const tkv_paged& a, const tkv_paged& b) {
    return a.num_kv_heads == b.num_kv_heads && a.head_dim == b.head_dim && (a.kv_type == b.kv_type || !(has_records(a.kv_type) || has_records(b.kv_type)));
}

}  // namespace

extern "C" int64_t tkv_beam_select_workspace(int32_t dtype, int64_t batch, int32_t beams, int32_t vocab, int32_t count) {
    if (!select_shape_ok(dtype, batch, beams, vocab, count) || batch == 0) return 0;
    int sms = 0;
    if (device_sms(&sms) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    return select_bytes(batch * beams, split_rows(batch * beams, beams, vocab, count, dtype_size(dtype), sms).chunks, count);
}

extern "C" tkv_status tkv_beam_select(const void* logits, int32_t dtype, int64_t batch, int32_t beams, int32_t vocab, int64_t batch_stride,
                                      int64_t beam_stride, const float* scores, const uint8_t* finished, int32_t eos, int32_t count,
                                      float* out_scores, int32_t* out_beams, int32_t* out_tokens, void* workspace, int64_t workspace_bytes,
                                      void* stream) {
    if (!select_shape_ok(dtype, batch, beams, vocab, count) || batch_stride < 0 || beam_stride < 0) return TKV_EINVAL;
    if (finished && (eos < 0 || eos >= vocab)) return TKV_EINVAL;
    if (batch == 0) return TKV_OK;
    if (!logits || !scores || !out_scores || !out_beams || !out_tokens) return TKV_EINVAL;
    if ((reinterpret_cast<uintptr_t>(logits) & (dtype_size(dtype) - 1)) || !aligned4(scores) || !aligned4(out_scores) || !aligned4(out_beams) ||
        !aligned4(out_tokens) || !aligned16(workspace))
        return TKV_EINVAL;
    int sms = 0;
    cudaError_t e = device_sms(&sms);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return TKV_ECUDA;
    }
    const int64_t rows = batch * beams;
    const Split s = split_rows(rows, beams, vocab, count, dtype_size(dtype), sms);
    if (!workspace || workspace_bytes < select_bytes(rows, s.chunks, count)) return TKV_ECAPACITY;
    SelectArgs a{};
    a.logits = logits;
    a.scores = scores;
    a.finished = finished;
    a.out_scores = out_scores;
    a.out_beams = out_beams;
    a.out_tokens = out_tokens;
    a.stats = reinterpret_cast<Stat*>(workspace);
    a.best = reinterpret_cast<Candidate*>(a.stats + rows * s.chunks);
    a.batch_stride = batch_stride;
    a.beam_stride = beam_stride;
    a.batch = (int)batch;
    a.beams = beams;
    a.vocab = vocab;
    a.eos = eos;
    a.count = count;
    a.chunks = s.chunks;
    a.per_chunk = s.per_chunk;
    cudaStream_t st = (cudaStream_t)stream;
    const dim3 grid(s.chunks, (unsigned)std::min<int64_t>(rows, 65535), (unsigned)((rows + 65534) / 65535));
    e = launch_behind(dtype == TKV_BF16   ? select_rows_kernel<__nv_bfloat16>
                      : dtype == TKV_FP16 ? select_rows_kernel<__half>
                                          : select_rows_kernel<float>,
                      grid, kThreads, 0, st, a);
    if (e == cudaSuccess) e = launch_behind(select_join_kernel, dim3((unsigned)batch), kThreads, 0, st, a);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return TKV_ECUDA;
    }
    return TKV_OK;
}

extern "C" tkv_status tkv_paged_reorder(const tkv_paged* caches, int32_t num_caches, const int32_t* parents, int32_t beams, int32_t* status,
                                        void* stream) {
    if (!caches || num_caches < 1 || !parents || !aligned4(parents) || !aligned4(status) || beams < 1 || beams > 32) return TKV_EINVAL;
    for (int i = 0; i < num_caches; ++i) {
        const tkv_paged &c = caches[i], &f = caches[0];
        if (check_paged(&c) != TKV_OK || c.page_table != f.page_table || c.lengths != f.lengths || c.batch != f.batch || c.max_pages != f.max_pages ||
            c.page_size != f.page_size || (int64_t)c.page_size * c.num_kv_heads * 32 > 0x7FFFFFFF)   // pieces of a page are counted in 32 bits
            return TKV_EINVAL;
    }
    if (caches[0].batch % beams) return TKV_EINVAL;
    int sms = 0;
    cudaError_t e = device_sms(&sms);
    ReorderArgs a{};
    a.table = const_cast<int32_t*>(caches[0].page_table);
    a.lengths = caches[0].lengths;
    a.parents = parents;
    a.status = status;
    a.groups = caches[0].batch / beams;
    a.beams = beams;
    a.max_pages = caches[0].max_pages;
    a.page_shift = __builtin_ctz((unsigned)caches[0].page_size);
    // CTAs of an SM: several rounds, which even out what SMs get of the memory, but a round of CTAs without work costs 1.2 us.  80 layers of 8 x 8
    // beams of 1,000 positions: 78.2 us with 20, 91.5 with four; 64 x 4 beams 144 with 48, 173 with eight.  32 layers of 8 x 12 beams of two
    // positions in pages of 128: 5.3 us with four, 4.2 with two, 10.8 with sixteen; 80 layers of 4 x 16 beams 134.6 with four, 138.6 with two, 131.3
    // with eight.  Behind 16 beams, with one, two, four, eight: 80 layers of 2 x 32 158.8, 158.5, 160.8, 165.8 us; 32 layers of 4 x 32 of 16-bit pages
    // 20.5, 18.5, 18.8, 24.9; 28 of 1 x 32 6.4, 8.6, 8.6, 8.6; but 16 layers of 16 x 24, heads of 64, 115, 113, 95, 92.
    const int ctas = beams <= 4 ? 48 : beams <= 8 ? 20 : beams <= 16 ? 4 : 2;
    a.table_split = std::max(1, std::min((a.max_pages + kThreads - 1) / kThreads, 16));   // of the first launch
    for (int first = 0; first < num_caches && e == cudaSuccess; ++first) {   // the caches of one shape after those of another
        const tkv_paged& c = caches[first];
        int before = 0;
        while (before < first && !same_shape(caches[before], c)) ++before;
        if (before < first) continue;
        const bool records = has_records(c.kv_type);
        a.heads = c.num_kv_heads;
        a.parts = records ? 1 : 2;
        a.per = records ? 16 : 1;
        a.unit = c.kv_type == TKV_INT4 ? 18 * c.head_dim : records ? 32 * c.head_dim + 16 : 2 * c.head_dim;
        a.head_bytes = (int64_t)(c.page_size / a.per) * a.unit * a.parts;
        for (int at = first; at < num_caches && e == cudaSuccess;) {
            a.num_caches = 0;
            a.least_pages = LLONG_MAX;
            for (; at < num_caches && a.num_caches < kMaxCaches; ++at) {
                if (!same_shape(caches[at], c)) continue;
                a.pages[a.num_caches] = reinterpret_cast<uint8_t*>(caches[at].pages);
                a.num_pages[a.num_caches++] = caches[at].num_pages;
                a.least_pages = std::min<int64_t>(a.least_pages, caches[at].num_pages);
            }
            if (a.num_caches == 0) break;
            // none without a piece
            const int64_t most = a.head_bytes / 16 * a.heads * a.num_caches;
            a.split = (int)std::min(std::max<int64_t>(1, (int64_t)sms * ctas / a.groups), (most + kThreads - 1) / kThreads);
            const int64_t grid = a.groups * (a.split + a.table_split);
            if (grid > 0x7FFFFFFF) return TKV_EINVAL;
            cudaStream_t st = (cudaStream_t)stream;
            e = beams <= 4    ? launch_behind(reorder_kernel<4>, dim3((unsigned)grid), kThreads, 0, st, a)
                : beams <= 8  ? launch_behind(reorder_kernel<8>, dim3((unsigned)grid), kThreads, 0, st, a)
                : beams <= 16 ? launch_behind(reorder_kernel<16>, dim3((unsigned)grid), kThreads, 0, st, a)
                              : launch_behind(reorder_kernel<32>, dim3((unsigned)grid), kThreads, 0, st, a);
            a.table_split = 0;
        }
    }
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return TKV_ECUDA;
    }
    return TKV_OK;
}
