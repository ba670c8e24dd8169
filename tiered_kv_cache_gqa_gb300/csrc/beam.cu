// Beam search: tkv_beam_select (the best continuations over beams and vocabulary) and tkv_paged_reorder (the paged caches of all
// layers follow the beams that were chosen).
//
// Selection.  total[b, w, v] = scores[b, w] + x[b, w, v] - lse[b, w],  lse = log sum_v exp x;  the `count` largest over (w, v), the
// lower w V + v first where totals are equal.  Within a row (a beam's logits) the order is that of x itself, so a row's best `count`
// by (x, v) are all that it can bring.  One pass over the logits: a CTA takes a chunk of a row, 16 KB at a time in registers, and
// keeps per thread a running maximum and sum of exponentials, per CTA the best `count` so far.  A second kernel, started
// early, joins a sequence's chunks: totals in 64 bits (two beams' totals may lie as near as fp32's rounding), the best of them.
//
// The best of a tile.  The count-th largest of the 256 threads' maxima (each with its place, so no two are equal) is a bound:
// `count` values at least reach it, and only the `count` threads whose maxima do can hold any, so at most count * 32 are looked
// at, whatever the values are: no distribution and no number of ties makes the list overflow.  Once the list is
// full only values above its last one are looked at, which after the first tiles are few.
//
// What bounds it is memory, then issue: an element costs about seven instructions (unpack, maximum, difference, product,
// exponential, sum).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "paged.cuh"

using namespace tkv;

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCount = 64, kMaxBeams = 64;
constexpr int kVectors = 4;                       // 16-byte pieces of a thread and tile
constexpr int kCtas = 4;                          // on an SM at once, by their registers
constexpr int kMostCandidates = 8192;             // of a sequence, for the joining kernel
constexpr float kLog2E = 1.44269504f;
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

// Larger is better: the value first, the lower place next.
__device__ __forceinline__ uint64_t key_of(float x, int v) {
    const uint32_t u = __float_as_uint(x + 0.0f);   // -0 is 0
    const uint32_t ordered = u & 0x80000000u ? ~u : u | 0x80000000u;
    return (uint64_t)ordered << 32 | (uint32_t)~v;
}
__device__ __forceinline__ Candidate of_key(uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return Candidate{__uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o), (int)~(uint32_t)key};
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A beam that brings nothing of its logits: finished, or with a score that is not finite.
__device__ __forceinline__ bool is_out(const SelectArgs& a, int row) {
    const float s = a.scores[row];
    return !(fabsf(s) < INFINITY) || (a.finished && a.finished[row]);
}

// A value that is left out: an infinity below, like what lies behind the vocabulary.
template <typename T, int E>
__device__ __forceinline__ void unpack16(uint4 u, float (&x)[E]) {
    if (sizeof(T) == 4) {
        x[0] = __uint_as_float(u.x);
        x[1] = __uint_as_float(u.y);
        x[2 % E] = __uint_as_float(u.z);
        x[3 % E] = __uint_as_float(u.w);
    } else {
        Vec16<T> w;
        w.u = u;
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = to_float(w.e[i]);
    }
}

// blockIdx.x: chunk, blockIdx.y (and z, behind 65,535 rows): row.
template <typename T>
__global__ void __launch_bounds__(kThreads, kCtas) select_rows_kernel(const __grid_constant__ SelectArgs a) {
    constexpr int E = 16 / sizeof(T), N = kVectors * E;         // values of a piece, of a thread and tile
    constexpr int kMost = kMaxCount * N + kMaxCount;            // values that are looked at
    __shared__ uint64_t keys[kMost];                             // the list, then what a tile adds to it
    __shared__ uint64_t list[kMaxCount];
    __shared__ uint64_t maxima[kThreads];
    __shared__ uint64_t bound;
    __shared__ int found;
    __shared__ Stat stats[kWarps];
    let_next_start();
    wait_for_previous();
    const int row = blockIdx.y + blockIdx.z * 65535, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (row >= a.batch * a.beams || is_out(a, row)) return;
    const int b = row / a.beams, w = row - b * a.beams;
    const T* x0 = reinterpret_cast<const T*>(a.logits) + b * a.batch_stride + w * a.beam_stride;
    // Pieces are counted from the 16-byte boundary at or before the row: the first and the last one may be cut.
    const int shift = (int)((reinterpret_cast<uintptr_t>(x0) & 15) / sizeof(T));
    const uint4* pieces = reinterpret_cast<const uint4*>(x0 - shift);
    const int first = blockIdx.x * a.per_chunk, end = min(first + a.per_chunk, (a.vocab + shift + E - 1) / E);
    constexpr uint32_t kNone = sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
    auto load = [&](int p) {
        uint4 u = make_uint4(kNone, kNone, kNone, kNone);
        if (p >= end) return u;
        const int v0 = p * E - shift;
        if (v0 >= 0 && v0 + E <= a.vocab) return pieces[p];
        Vec16<T> part;
        part.u = u;
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (v0 + i >= 0 && v0 + i < a.vocab) part.e[i] = x0[v0 + i];
        return part.u;
    };
    float m = kFloor, sum = 0.0f, last = -INFINITY;   // last: the list's last value once it is full
    int held = 0;
    uint4 raw[kVectors];
#pragma unroll
    for (int i = 0; i < kVectors; ++i) raw[i] = load(first + i * kThreads + tid);
#pragma unroll 1
    for (int p = first; p < end; p += kVectors * kThreads) {
        float x[N];
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
            float y[E];
            unpack16<T, E>(raw[i], y);
#pragma unroll
            for (int j = 0; j < E; ++j) x[i * E + j] = y[j];
        }
#pragma unroll
        for (int i = 0; i < kVectors; ++i) raw[i] = load(p + (kVectors + i) * kThreads + tid);   // the next tile's
        float top = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) top = fmaxf(top, x[i]);
        if (top > m) {
            sum *= exp2_fast((m - top) * kLog2E);
            m = top;
        }
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < N; ++i) s[i & 1] += exp2_fast((x[i] - m) * kLog2E);
        sum += s[0] + s[1];
        // ---- the tile's part of the best.  Places grow from tile to tile, so an equal value comes too late.
        const int above = __syncthreads_count(top > last);
        if (above == 0) continue;
        uint64_t least = 0;                            // 0: whatever is above the list
        auto place = [&](int i) { return (p + (i / E) * kThreads + tid) * E - shift + i % E; };
        if (above > a.count) {
            int at = 0;
#pragma unroll
            for (int i = N - 1; i >= 0; --i) at = x[i] == top ? i : at;
            const uint64_t mine = top > last ? key_of(top, place(at)) : 0;
            maxima[tid] = mine;
            __syncthreads();
            int rank = 0;
#pragma unroll 8
            for (int i = 0; i < kThreads; ++i) rank += maxima[i] > mine;
            if (mine && rank == a.count - 1) bound = mine;
        }
        if (tid < held) keys[tid] = list[tid];
        if (tid == 0) found = held;
        __syncthreads();
        if (above > a.count) least = bound;
        if (top > last) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (x[i] > last) {
                    const uint64_t k = key_of(x[i], place(i));
                    if (k >= least) keys[atomicAdd(&found, 1)] = k;
                }
        }
        __syncthreads();
        const int n = found;
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t k = keys[i];
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j) rank += keys[j] > k;
            if (rank < a.count) list[rank] = k;
        }
        __syncthreads();
        held = min(n, a.count);
        if (held == a.count) last = of_key(list[a.count - 1]).x;
    }
    // ---- the chunk's reference and sum
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, sum, o), top = fmaxf(m, m2);
        sum = sum * exp2_fast((m - top) * kLog2E) + s2 * exp2_fast((m2 - top) * kLog2E);
        m = top;
    }
    if (lane == 0) stats[warp] = Stat{m, sum};
    __syncthreads();
    const int64_t at = (int64_t)row * a.chunks + blockIdx.x;
    if (tid == 0) {
        Stat t = stats[0];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) {
            const float top = fmaxf(t.m, stats[i].m);
            t.sum = t.sum * exp2_fast((t.m - top) * kLog2E) + stats[i].sum * exp2_fast((stats[i].m - top) * kLog2E);
            t.m = top;
        }
        a.stats[at] = t;
    }
    if (tid < a.count) a.best[at * a.count + tid] = tid < held ? of_key(list[tid]) : Candidate{0.0f, -1};
}

// A candidate of a sequence: its total as an ordered number, its place w V + v.
struct Total {
    uint64_t total;   // 0: none
    uint32_t place;
};
__device__ __forceinline__ bool better(const Total& a, const Total& b) { return a.total > b.total || (a.total == b.total && a.place < b.place); }
__device__ __forceinline__ Total total_of(double t, int w, int v, int vocab) {
    if (!(t > -INFINITY)) return Total{0, 0xFFFFFFFFu};
    const uint64_t u = (uint64_t)__double_as_longlong(t + 0.0);   // no negative zero
    return Total{u >> 63 ? ~u : u | (uint64_t)1 << 63, (uint32_t)w * (uint32_t)vocab + (uint32_t)v};
}
__device__ __forceinline__ double value_of(uint64_t o) { return __longlong_as_double((long long)(o >> 63 ? o & 0x7FFFFFFFFFFFFFFFull : ~o)); }

// One CTA a sequence.
__global__ void __launch_bounds__(kThreads) select_join_kernel(const __grid_constant__ SelectArgs a) {
    constexpr int kEach = kMostCandidates / kThreads;             // candidates of a thread
    __shared__ double reference[kMaxBeams], offset[kMaxBeams];    // total = (x - reference) + offset
    __shared__ Total maxima[kThreads];
    __shared__ Total keys[kMaxCount * kEach + kMaxBeams];
    __shared__ Total bound;
    __shared__ int found;
    wait_for_previous();
    const int b = blockIdx.x, tid = threadIdx.x, per_row = a.chunks * a.count, n = a.beams * per_row;
    const Candidate* best = a.best + (int64_t)b * n;
    if (tid < a.beams) {
        const int row = b * a.beams + tid;
        double o = NAN, r = 0.0;
        if (!is_out(a, row)) {
            const Stat* s = a.stats + (int64_t)row * a.chunks;
            float top = kFloor;
            for (int i = 0; i < a.chunks; ++i) top = fmaxf(top, s[i].m);
            double sum = 0.0;
            for (int i = 0; i < a.chunks; ++i) sum += (double)(s[i].sum * exp2_fast((s[i].m - top) * kLog2E));
            r = (double)top;
            o = (double)a.scores[row] - log(sum);
        }
        reference[tid] = r;
        offset[tid] = o;
    }
    if (tid == 0) found = 0;
    __syncthreads();
    auto total_at = [&](int i) {   // candidate i of the sequence
        const int w = i / per_row;
        if (isnan(offset[w])) return Total{0, 0xFFFFFFFFu};
        const Candidate c = best[i];
        return c.v < 0 ? Total{0, 0xFFFFFFFFu} : total_of(((double)c.x - reference[w]) + offset[w], w, c.v, a.vocab);
    };
    Total mine{0, 0xFFFFFFFFu};
    if (tid < a.beams) {   // a finished beam's one candidate
        const int row = b * a.beams + tid;
        if (a.finished && a.finished[row] && fabsf(a.scores[row]) < INFINITY) mine = total_of((double)a.scores[row], tid, a.eos, a.vocab);
    }
    const Total own = mine;
    for (int i = tid; i < n; i += kThreads) {
        const Total t = total_at(i);
        if (better(t, mine)) mine = t;
    }
    maxima[tid] = mine;
    if (tid == 0) bound = Total{1, 0xFFFFFFFFu};   // below every candidate
    __syncthreads();
    if (mine.total) {
        int rank = 0;
#pragma unroll 4
        for (int i = 0; i < kThreads; ++i) rank += better(maxima[i], mine);
        if (rank == a.count - 1) bound = mine;
    }
    __syncthreads();
    const Total least = bound;
    if (mine.total && !better(least, mine)) {
        if (own.total && !better(least, own)) keys[atomicAdd(&found, 1)] = own;
        for (int i = tid; i < n; i += kThreads) {
            const Total t = total_at(i);
            if (t.total && !better(least, t)) keys[atomicAdd(&found, 1)] = t;
        }
    }
    __syncthreads();
    const int m = found;
    const int64_t out = (int64_t)b * a.count;
    for (int i = tid; i < m; i += kThreads) {
        const Total t = keys[i];
        int rank = 0;
        for (int j = 0; j < m; ++j) rank += better(keys[j], t);
        if (rank < a.count) {
            const uint32_t w = t.place / (uint32_t)a.vocab;
            a.out_scores[out + rank] = (float)value_of(t.total);
            a.out_beams[out + rank] = (int)w;
            a.out_tokens[out + rank] = (int)(t.place - w * (uint32_t)a.vocab);
        }
    }
    for (int i = m + tid; i < a.count; i += kThreads) {
        a.out_scores[out + i] = -INFINITY;
        a.out_beams[out + i] = a.out_tokens[out + i] = -1;
    }
}

// How the rows are cut: as many CTAs as the device holds at once, chunks of 256 pieces at least, and no more candidates than the
// joining kernel takes.
struct Split {
    int chunks, per_chunk;   // pieces of a chunk
};
Split split_rows(int64_t rows, int beams, int vocab, int count, int element, int sms) {
    const int pieces = vocab / (16 / element) + 2;   // at most, whatever the row's alignment
    int64_t chunks = std::max<int64_t>(1, (int64_t)sms * kCtas / rows);
    chunks = std::min<int64_t>(chunks, (pieces + kThreads - 1) / kThreads);
    chunks = std::min<int64_t>(chunks, std::max(1, kMostCandidates / (beams * count)));
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
// A CTA serves one cache and one sequence of beams: it reads the sequence's parents, lengths and pages once (three trips to memory
// in a row) and walks over 16-byte pieces.
constexpr int kMaxCaches = 64;   // of a launch

struct CacheRef {
    uint8_t* pages;
    int64_t num_pages;
    int64_t head_bytes;      // of a page
    int32_t heads;
    int32_t parts;           // of a head's page that hold positions: 1 (records), or K and V
    int32_t unit;            // bytes of a part's `per` positions
    int32_t per;
};

struct ReorderArgs {
    CacheRef cache[kMaxCaches];
    int32_t* table;
    const int32_t* lengths;
    const int32_t* parents;
    int32_t* status;
    int64_t groups;
    int num_caches, beams, max_pages, page_shift;
    int split, table_split;   // CTAs of a cache and sequence; of a sequence's table (0: the table stays)
};

template <int W>
__global__ void __launch_bounds__(kThreads) reorder_kernel(const __grid_constant__ ReorderArgs a) {
    __shared__ int parent[W], page[W];
    __shared__ uint32_t children[W];   // beams that go on from this one, itself not among them
    __shared__ int length, bad;
    let_next_start();
    wait_for_previous();
    const int tid = threadIdx.x;
    int64_t unit = blockIdx.x;
    const int64_t copies = a.groups * a.num_caches * a.split;
    const bool is_table = unit >= copies;
    if (is_table) unit -= copies;
    const int parts_of = is_table ? a.table_split : a.split, part = (int)(unit % parts_of);
    unit /= parts_of;
    const int64_t group = unit % a.groups;
    const CacheRef& c = a.cache[is_table ? 0 : (int)(unit / a.groups)];
    if (tid == 0) {
        length = a.lengths[group * a.beams];
        bad = 0;
    }
    if (tid < W) children[tid] = 0;
    __syncthreads();
    const int len = length, column = len >> a.page_shift, rest = len & ((1 << a.page_shift) - 1);
    const bool fits = len >= 0 && (column < a.max_pages || (column == a.max_pages && rest == 0));
    if (tid < a.beams) {
        const int64_t seq = group * a.beams + tid;
        int p = a.parents[seq], pg = -1;
        if (p >= a.beams) {
            raise_status(a.status, TKV_EINVAL);
            p = -1;
        }
        if (a.lengths[seq] != len) atomicOr(&bad, 1);
        if (fits && rest) pg = a.table[seq * a.max_pages + column];
        parent[tid] = p < 0 ? tid : p;   // none: it stays
        page[tid] = pg;
    }
    __syncthreads();
    if (bad || !fits) {
        if (tid == 0 && part == 0) raise_status(a.status, bad ? TKV_EINVAL : TKV_ECAPACITY);
        return;
    }
    if (tid < a.beams && parent[tid] != tid) {
        const int p = parent[tid];
        bool goes = true;
        if (!is_table) {
            goes = page[p] != page[tid];
            if (rest && ((uint32_t)page[p] >= c.num_pages || (uint32_t)page[tid] >= c.num_pages)) {
                if (part == 0) raise_status(a.status, TKV_ECAPACITY);
                goes = false;
            }
        }
        if (goes) atomicOr(&children[p], 1u << tid);
    }
    __syncthreads();
    uint32_t kids[W];
    bool any = false;
#pragma unroll
    for (int p = 0; p < W; ++p) {
        kids[p] = children[p];
        any |= kids[p] != 0;
    }
    if (!any) return;
    const int at = part * kThreads + tid, step = parts_of * kThreads;
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
    const int pieces = (rest + c.per - 1) / c.per * (c.unit / 16);       // of a part
    const int total = pieces * c.parts * c.heads;
    const int64_t part_bytes = c.head_bytes / c.parts, page_bytes = c.head_bytes * c.heads;
    for (int i = at; i < total; i += step) {
        const int q = i / pieces;                                        // head and part
        uint8_t* to = c.pages + q * part_bytes + (int64_t)(i - q * pieces) * 16;
        uint4 v[W];
#pragma unroll
        for (int p = 0; p < W; ++p)
            if (kids[p]) v[p] = *reinterpret_cast<const uint4*>(to + page[p] * page_bytes);
#pragma unroll
        for (int p = 0; p < W; ++p)
            for (uint32_t k = kids[p]; k; k &= k - 1) *reinterpret_cast<uint4*>(to + page[__ffs(k) - 1] * page_bytes) = v[p];
    }
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
    for (int from = 0; from < num_caches && e == cudaSuccess; from += kMaxCaches) {
        a.num_caches = std::min(num_caches - from, kMaxCaches);
        int64_t most = 1;
        for (int i = 0; i < a.num_caches; ++i) {
            const tkv_paged& c = caches[from + i];
            CacheRef& r = a.cache[i];
            const bool records = has_records(c.kv_type);
            r.pages = reinterpret_cast<uint8_t*>(c.pages);
            r.num_pages = c.num_pages;
            r.heads = c.num_kv_heads;
            r.parts = records ? 1 : 2;
            r.per = records ? 16 : 1;
            r.unit = c.kv_type == TKV_INT4 ? 18 * c.head_dim : records ? 32 * c.head_dim + 16 : 2 * c.head_dim;
            r.head_bytes = (int64_t)(c.page_size / r.per) * r.unit * r.parts;
            most = std::max(most, r.head_bytes * r.heads / 16);
        }
        // CTAs: two times what the device holds, none without a piece
        const int64_t wanted = std::max<int64_t>(1, (int64_t)sms * 16 / (a.groups * a.num_caches));
        a.split = (int)std::min(wanted, (most + kThreads - 1) / kThreads);
        a.table_split = from ? 0 : std::max(1, std::min((a.max_pages + kThreads - 1) / kThreads, 16));
        const int64_t grid = a.groups * ((int64_t)a.num_caches * a.split + a.table_split);
        if (grid > 0x7FFFFFFF) return TKV_EINVAL;
        cudaStream_t st = (cudaStream_t)stream;
        e = beams <= 4    ? launch_behind(reorder_kernel<4>, dim3((unsigned)grid), kThreads, 0, st, a)
            : beams <= 8  ? launch_behind(reorder_kernel<8>, dim3((unsigned)grid), kThreads, 0, st, a)
            : beams <= 16 ? launch_behind(reorder_kernel<16>, dim3((unsigned)grid), kThreads, 0, st, a)
                          : launch_behind(reorder_kernel<32>, dim3((unsigned)grid), kThreads, 0, st, a);
    }
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return TKV_ECUDA;
    }
    return TKV_OK;
}
