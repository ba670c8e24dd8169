// Rows into and out of a paged cache: tkv_paged_append (k rotated on the way) and tkv_paged_gather.
//
// A step's rows are ragged: sequence b owns rows cu[b] .. cu[b + 1], which are the last positions of its
// lengths[b].  A thread of the append takes, of a row of K and of V, 16 bytes of channels and the 16 bytes that hold
// their partners (or 16 bytes alone, where k is not rotated by halves), and walks over KV heads: each value is read
// once, and the row's place and the 8 cosines and sines are found once for all its heads; two neighbours share a scale.  A thread of
// the gather writes 16 bytes of K and of V.  So each instruction of a warp reads and writes whole sectors: with 32 bytes
// a thread, in two halves, the gather sent 164 MB to L2 for the 75 MB that it wrote.
//
// What bounds both is memory: 2 bytes a value on one side, 0.5625 (codes and scales) or 2 on the other.
#include <algorithm>
#include <type_traits>

#include "paged_tile.cuh"

using namespace tkv;

namespace {

constexpr int kThreads = 256;
constexpr int kAppendCtas = 4, kGatherCtas = 8;   // on an SM at once, by their registers

struct RowArgs {
    tkv_paged c;
    const void* k;             // append: inputs; gather: outputs
    const void* v;
    const float2* table;       // null: k is not rotated
    const int32_t* positions;  // null: the row's position in the cache
    const int32_t* cu;
    int32_t* status;
    int64_t rows, axis_stride, k_row, k_head, v_row, v_head;
    int pairs, max_positions, num_axes, interleaved;
    bool table_16;             // two pairs of the table lie on 16 bytes
    int lanes;                 // heads that the threads of a row take at once
    int page_shift;
    float sign;
    int units;                 // append: threads of a row
    alignas(16) uint8_t pair_axis[256];
};

// Where row `row` of the step lies: page and position in the page; false for no row (behind the last
// sequence: *page = -2) and for a bad place (*page = -1: the position or the page is outside).
__device__ __forceinline__ bool place_of_row(const RowArgs& a, int64_t row, int64_t* page, int* off, int* position) {
    const int b = sequence_of_row(a.cu, a.c.batch, (int)row);
    *page = -2;
    if (b < 0) return false;
    const int pos = a.c.lengths[b] - (a.cu[b + 1] - (int)row);
    *page = -1;
    *position = pos;
    if (pos < 0 || (pos >> a.page_shift) >= a.c.max_pages) return false;
    const int p = a.c.page_table[(int64_t)b * a.c.max_pages + (pos >> a.page_shift)];
    if (p < 0 || p >= a.c.num_pages) return false;
    *page = p;
    *off = pos & (a.c.page_size - 1);
    return true;
}

// max(|a|, |b|, |c|); NaN if one of them is
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float y;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// The largest |x| of a block, of which 8 values are the neighbouring lane's (xor 1); NaN if one is.  The whole warp calls it
// (but the lanes that have left): a mask of its own for each pair of lanes made the shuffle sixteen times as long.
__device__ __forceinline__ float block_max(const float (&x)[8]) {
    const float m = max3_abs(max3_abs(max3_abs(x[0], x[1], x[2]), x[3], x[4]), max3_abs(x[5], x[6], x[7]), 0.0f);
    return max3_abs(m, __shfl_xor_sync(0xffffffffu, m, 1), 0.0f);
}

// 8 values of a block with that maximum -> 8 codes and the byte of the block's scale.
//   scale = e4m3(max |x| / (7 gain)), to nearest even; q = x / step, step = scale * gain, to nearest even.
// The quotients are products with 1 / (7 gain) and 1 / step, cut towards zero.  Where gain is a power of two, 7 gain and
// step (four bits) have rounded reciprocals that are never below the true ones (for 7 and all eight steps; by less than
// 2^-24), so the cut product of an exact tie is the tie, and it goes to the even side as the quotient would; elsewhere
// only a quotient within 2^-22 of a tie could round to the other side.
// Adding 1.5 * 2^23 + 8 rounds to an integer whose low four bits are q + 8.
// A block that holds an infinity or a NaN gets the NaN scale: it reads as NaN, not as something finite.
__device__ __forceinline__ uint32_t quantise_half(float (&x)[8], float amax, float gain, float inv_7_gain, uint8_t* scale_byte) {
    const bool bad = !(amax < INFINITY);
    const __nv_fp8_storage_t s8 =
        bad ? (__nv_fp8_storage_t)0x7F : __nv_cvt_float_to_fp8(__fmul_rz(amax, inv_7_gain), __NV_SATFINITE, __NV_E4M3);
    *scale_byte = (uint8_t)s8;
    const float step = __fmul_rn(__half2float(__half(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3))), gain);
    const float inv = step > 0.0f ? __frcp_rn(step) : 0.0f;
    if (amax * inv >= 7.5f) {   // a scale that saturated, or was rounded down far below 2^-6; elsewhere |x| <= 7.44 steps
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -7.0f * step), 7.0f * step);
    }
    uint32_t pair[4];
    const F2 inv2 = f2(inv, inv), to_int = f2(12582920.0f, 12582920.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 q = parts(add2(mul2_rz(f2(x[2 * i], x[2 * i + 1]), inv2), to_int));
        pair[i] = __float_as_uint(q.y) * 16u + __float_as_uint(q.x);   // the low byte holds both codes
    }
    const uint32_t codes = __byte_perm(__byte_perm(pair[0], pair[1], 0x0040), __byte_perm(pair[2], pair[3], 0x0040), 0x5410);
    return bad ? 0x88888888u : codes;
}

// 16 bytes as floats, and back.
template <typename T>
__device__ __forceinline__ void unpack(uint4 u, float (&x)[16 / sizeof(T)]) {
    Vec16<T> v;
    v.u = u;
#pragma unroll
    for (int i = 0; i < 16 / (int)sizeof(T); ++i) x[i] = to_float(v.e[i]);
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float* x) {
    Vec16<T> v;
#pragma unroll
    for (int i = 0; i < 16 / (int)sizeof(T); ++i) v.e[i] = from_float<T>(x[i]);
    return v.u;
}

// How k is rotated.
//   kNone      not at all
//   kHalves    pairs % 16 == 0: the partners of 8 channels lie `pairs` channels away, in another block
//   kAdjacent  pairs % 4 == 0: 8 channels hold their own 4 pairs
//   kAny       channel by channel, partners read one at a time
enum Turn { kNone, kHalves, kAdjacent, kAny };

// Channels 8 chunk .. + 7 of head row k, turned one at a time (kAny).
template <typename T>
__device__ __forceinline__ void turn_any(const RowArgs& a, const T* k, int64_t row, int own_position, int chunk, float (&x)[8]) {
    bool bad = false;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
        const int ch = 8 * chunk + i;
        if (ch >= 2 * a.pairs) break;
        const bool first = a.interleaved ? !(ch & 1) : ch < a.pairs;
        const int j = a.interleaved ? ch >> 1 : first ? ch : ch - a.pairs;
        const int p = a.positions ? a.positions[a.pair_axis[j] * a.axis_stride + row] : own_position;
        const float2 cs = table_at(a.table, a.pairs, a.max_positions, p, j, a.sign, &bad);
        const float own = to_float(k[ch]), other = to_float(k[a.interleaved ? ch ^ 1 : first ? ch + a.pairs : ch - a.pairs]);
        const float y = first ? rotate_pair(own, other, cs).x : rotate_pair(other, own, cs).y;
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = c == i ? y : x[c];
    }
    if (bad) raise_status(a.status, TKV_EINVAL);
}

// x (8 values), and y if there is a partner, to their places: 4-bit pages, codes and the byte of the block's scale, `scale`
// bytes behind them; the partner's lie `partner` and `scale_partner` further on.
template <typename T, bool INT4>
__device__ __forceinline__ void put(float (&x)[8], float (&y)[8], bool two, uint8_t* to, int scale, int partner, int scale_partner, bool writes_scale, float gain) {
    if (INT4) {
        const float inv_7_gain = __frcp_rn(__fmul_rn(7.0f, gain));
        const float x_max = block_max(x), y_max = block_max(y);
        uint8_t s;
        *reinterpret_cast<uint32_t*>(to) = quantise_half(x, x_max, gain, inv_7_gain, &s);
        if (writes_scale) to[scale] = s;
        if (two) {
            *reinterpret_cast<uint32_t*>(to + partner) = quantise_half(y, y_max, gain, inv_7_gain, &s);
            if (writes_scale) to[scale + scale_partner] = s;
        }
    } else {
        *reinterpret_cast<uint4*>(to) = pack<T>(x);
        if (two) *reinterpret_cast<uint4*>(to + partner) = pack<T>(y);
    }
}

// blockIdx.y: the first head.  The threads of a row are an even number, so neighbours share its place.  K and V of a head
// one after the other, the next head's values on their way meanwhile: 64 registers, so four CTAs an SM, which cost a
// few spills and were worth it (18,432 rows of 8 heads of 128 into 4-bit pages: 27.3 us, 97 MB, 3.6 TB/s; three CTAs 34.5;
// both at once with three CTAs 32.4).  No unit is at its limit there: about 75 instructions for 8 values are issued in 64 % of
// the cycles, DRAM is busy for 36 %, 42 % of the warps there could be are there, and they wait for memory and for one another.
template <typename T, int D, bool INT4, int TURN>
__global__ void __launch_bounds__(kThreads, kAppendCtas) append_kernel(const __grid_constant__ RowArgs a) {
    let_next_start();
    wait_for_previous();
    const int rows_here = kThreads / a.units;
    const int unit = threadIdx.x % a.units;
    const int64_t row = (int64_t)blockIdx.x * rows_here + threadIdx.x / a.units;
    if (threadIdx.x >= rows_here * a.units || row >= a.rows) return;
    // units of kHalves: the pairs of chunks, then the chunks behind the rotated ones
    const int pair_chunks = TURN == kHalves ? a.pairs / 8 : 0;
    const int chunk = TURN == kHalves && unit >= pair_chunks ? unit + pair_chunks : unit;
    const bool two = TURN == kHalves && unit < pair_chunks;
    const bool turned = TURN != kNone && 8 * chunk < 2 * a.pairs;
    const T* k = reinterpret_cast<const T*>(a.k) + row * a.k_row;
    const T* k_at = k + blockIdx.y * a.k_head + 8 * chunk;
    const T* v_at = reinterpret_cast<const T*>(a.v) + row * a.v_row + blockIdx.y * a.v_head + 8 * chunk;
    // The next head's values are read while the last one's are worked on, the first one's and the positions before the row's
    // place is looked for: what a thread waits for is memory, several times in a row.
    uint4 k_raw[2] = {}, v_raw[2] = {};
    auto read = [&](uint4 (&raw)[2], const T*& at, int64_t stride, int h) {
        if (h >= a.c.num_kv_heads) return;
        raw[0] = *reinterpret_cast<const uint4*>(at);
        if (two) raw[1] = *reinterpret_cast<const uint4*>(at + a.pairs);
        at += a.lanes * stride;
    };
    read(k_raw, k_at, a.k_head, blockIdx.y);
    read(v_raw, v_at, a.v_head, blockIdx.y);
    int p[4] = {0, 0, 0, 0};
    if (turned && a.positions) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (x < a.num_axes) p[x] = a.positions[x * a.axis_stride + row];
    }
    int64_t page;
    int off, position;
    if (!place_of_row(a, row, &page, &off, &position)) {
        if (page == -1 && unit == 0 && blockIdx.y == 0) raise_status(a.status, TKV_ECAPACITY);
        return;
    }
    constexpr int NCS = TURN == kHalves ? 8 : 4;
    float2 cs[NCS];
    if ((TURN == kHalves || TURN == kAdjacent) && turned) {
        if (!a.positions) p[0] = position;
        load_angles<NCS>(a, p, NCS * chunk, cs);
    }
    using R = Record<D>;
    const int64_t head_bytes = INT4 ? (int64_t)(a.c.page_size >> 4) * R::bytes : (int64_t)a.c.page_size * (4 * D);
    // in a head's page: K's place; how far behind it V's lies, and behind each its scale
    const int r = off & 15, block = chunk >> 1;
    uint8_t* to = reinterpret_cast<uint8_t*>(a.c.pages) + (page * a.c.num_kv_heads + blockIdx.y) * head_bytes +
                  (INT4 ? (off >> 4) * R::bytes + r * (D / 2) + 4 * chunk : off * (2 * D) + 16 * chunk);
    const int to_v = INT4 ? R::v_codes : a.c.page_size * (2 * D), partner = (INT4 ? 4 : 16) * pair_chunks;
    const int k_scale = R::k_scales + r * (D / 16) + block - (r * (D / 2) + 4 * chunk);
    const int v_scale = R::v_scales - R::v_codes + block * 16 + r - (r * (D / 2) + 4 * chunk);
    const int64_t next = a.lanes * head_bytes;
#pragma unroll 1
    for (int h = blockIdx.y; h < a.c.num_kv_heads; h += a.lanes) {
        const float k_gain = INT4 && a.c.k_gain ? a.c.k_gain[h] : 1.0f, v_gain = INT4 && a.c.v_gain ? a.c.v_gain[h] : 1.0f;
        float x[8], y[8];
        unpack<T>(k_raw[0], x);
        unpack<T>(k_raw[1], y);
        read(k_raw, k_at, a.k_head, h + a.lanes);
        if (TURN == kHalves && turned) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 z = rotate_pair(x[i], y[i], cs[i % NCS]);
                x[i] = z.x;
                y[i] = z.y;
            }
        } else if (TURN == kAdjacent && turned) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 z = rotate_pair(x[2 * i], x[2 * i + 1], cs[i % NCS]);
                x[2 * i] = z.x;
                x[2 * i + 1] = z.y;
            }
        } else if (TURN == kAny && turned) {
            turn_any(a, k + h * a.k_head, row, position, chunk, x);
        }
        put<T, INT4>(x, y, two, to, k_scale, partner, pair_chunks >> 1, !(chunk & 1), k_gain);
        unpack<T>(v_raw[0], x);
        unpack<T>(v_raw[1], y);
        read(v_raw, v_at, a.v_head, h + a.lanes);
        put<T, INT4>(x, y, two, to + to_v, v_scale, partner, (pair_chunks >> 1) * 16, !(chunk & 1), v_gain);
        to += next;
    }
}

// N codes (4 bits each, from bit 0) -> the values q * scale * gain, one rounding: the pairs of codes i and i + 4 become
// q * scale / 16 in fp16, exactly (as in the attention), and are multiplied by 16 gain in fp32.
template <int N>
__device__ __forceinline__ void expand(uint32_t word, uint8_t scale_byte, float gain, float (&x)[N]) {
    const __half s = __hmul(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)scale_byte, __NV_E4M3)), __float2half(0.0625f));
    const __half2 s2 = __half2half2(s), n1032 = __hmul2(s2, both(-1032.0f)), n72 = __hmul2(s2, both(-72.0f));
    const float g16 = 16.0f * gain;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const uint32_t w = word >> (4 * i);
        const float2 lo = __half22float2(bits_half2(expand_low(w, s2, n1032))), hi = __half22float2(bits_half2(expand_high(w, s2, n72)));
        x[i] = __fmul_rn(lo.x, g16);
        x[i + 1] = __fmul_rn(hi.x, g16);
        if (N == 8) {
            x[(i + 4) % N] = __fmul_rn(lo.y, g16);
            x[(i + 5) % N] = __fmul_rn(hi.y, g16);
        }
    }
}

// TO: element type of the outputs; T: of 16-bit pages.  blockIdx.y: the first head.
// 18,432 rows of 8 heads of 128 out of 4-bit pages: 20.1 us (97 MB, 4.8 TB/s); with 40 registers, six CTAs an SM, 23.5.
template <typename TO, typename T, int D, bool INT4>
__global__ void __launch_bounds__(kThreads, kGatherCtas) gather_kernel(const __grid_constant__ RowArgs a) {
    let_next_start();
    wait_for_previous();
    constexpr int N = 16 / sizeof(TO), NC = D / N;   // values of a thread, threads of a row
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int chunk = (int)(i % NC);
    const int64_t row = i / NC;
    const int lane = blockIdx.y;
    if (row >= a.rows) return;
    int64_t page;
    int off = 0, position;
    const bool good = place_of_row(a, row, &page, &off, &position);
    if (page == -2) return;
    if (!good && chunk == 0 && lane == 0) raise_status(a.status, TKV_ECAPACITY);
    TO* k = reinterpret_cast<TO*>(const_cast<void*>(a.k)) + row * a.k_row + lane * a.k_head + N * chunk;
    TO* v = reinterpret_cast<TO*>(const_cast<void*>(a.v)) + row * a.v_row + lane * a.v_head + N * chunk;
    using R = Record<D>;
    const int r = off & 15, block = N * chunk / 16;
    const int64_t head_bytes = INT4 ? (int64_t)(a.c.page_size >> 4) * R::bytes : (int64_t)a.c.page_size * (4 * D);
    const uint8_t* from = reinterpret_cast<const uint8_t*>(a.c.pages) + ((good ? page : 0) * a.c.num_kv_heads + lane) * head_bytes +
                          (INT4 ? (off >> 4) * R::bytes : off * (2 * D));
    using Raw = typename std::conditional<INT4, typename std::conditional<N == 8, uint32_t, uint16_t>::type,
                                          typename std::conditional<N == 8, uint4, uint2>::type>::type;
    // Heads whose loads go out before the first is stored.  6,139 rows of 4 heads of 128 out of 4-bit and 16-bit pages: as fp32,
    // half as many values a thread, 8.1 and 8.4 us with two, 8.6 and 9.2 with one; as bf16 5.9 and 12.2 (spills) against 5.7 and 6.7.
    constexpr int U = sizeof(TO) == 4 ? 2 : 1;
    const int k_at = INT4 ? R::k_codes + r * (D / 2) : 0, v_at = INT4 ? R::v_codes + r * (D / 2) : a.c.page_size * (2 * D);
    const int64_t next = a.lanes * head_bytes, next_k = a.lanes * a.k_head, next_v = a.lanes * a.v_head;
    for (int h = lane; h < a.c.num_kv_heads; h += U * a.lanes) {
        Raw kr[U], vr[U];
        uint8_t ks[U], vs[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!good || h + u * a.lanes >= a.c.num_kv_heads) break;
            const uint8_t* at = from + u * next;
            kr[u] = reinterpret_cast<const Raw*>(at + k_at)[chunk];
            vr[u] = reinterpret_cast<const Raw*>(at + v_at)[chunk];
            if (INT4) {
                ks[u] = at[R::k_scales + r * (D / 16) + block];
                vs[u] = at[R::v_scales + block * 16 + r];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int hu = h + u * a.lanes;
            if (hu >= a.c.num_kv_heads) break;
            float x[N], y[N];
            if (!good) {
#pragma unroll
                for (int j = 0; j < N; ++j) x[j] = y[j] = __int_as_float(0x7FC00000);
            } else if constexpr (INT4) {
                expand<N>(kr[u], ks[u], a.c.k_gain ? a.c.k_gain[hu] : 1.0f, x);
                expand<N>(vr[u], vs[u], a.c.v_gain ? a.c.v_gain[hu] : 1.0f, y);
            } else {
                union {
                    Raw u;
                    T e[N];
                } ke, ve;
                ke.u = kr[u];
                ve.u = vr[u];
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    x[j] = to_float(ke.e[j]);
                    y[j] = to_float(ve.e[j]);
                }
            }
            *reinterpret_cast<uint4*>(k) = pack<TO>(x);
            *reinterpret_cast<uint4*>(v) = pack<TO>(y);
            k += next_k;
            v += next_v;
        }
        from += U * next;
    }
}

cudaError_t spread(RowArgs& a, int64_t blocks, int ctas) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) a.lanes = spread_heads(blocks, a.c.num_kv_heads, (int64_t)sms * ctas, 8);
    return e;
}

template <typename T, int D, bool INT4>
cudaError_t append_turn(const RowArgs& a, int turn, dim3 grid, cudaStream_t st) {
    return launch_behind(turn == kNone       ? append_kernel<T, D, INT4, kNone>
                         : turn == kHalves   ? append_kernel<T, D, INT4, kHalves>
                         : turn == kAdjacent ? append_kernel<T, D, INT4, kAdjacent>
                                             : append_kernel<T, D, INT4, kAny>,
                         grid, kThreads, 0, st, a);
}

template <typename T>
cudaError_t append_type(const RowArgs& a, int turn, dim3 grid, cudaStream_t st) {
    const bool int4 = a.c.kv_type == TKV_INT4;
    if (a.c.head_dim == 128) return int4 ? append_turn<T, 128, true>(a, turn, grid, st) : append_turn<T, 128, false>(a, turn, grid, st);
    return int4 ? append_turn<T, 64, true>(a, turn, grid, st) : append_turn<T, 64, false>(a, turn, grid, st);
}

template <typename TO, int D>
cudaError_t gather_pages(const RowArgs& a, dim3 grid, cudaStream_t st) {
    return launch_behind(a.c.kv_type == TKV_INT4   ? gather_kernel<TO, __half, D, true>
                         : a.c.kv_type == TKV_FP16 ? gather_kernel<TO, __half, D, false>
                                                   : gather_kernel<TO, __nv_bfloat16, D, false>,
                         grid, kThreads, 0, st, a);
}

template <typename TO>
cudaError_t gather_type(const RowArgs& a, dim3 grid, cudaStream_t st) {
    return a.c.head_dim == 128 ? gather_pages<TO, 128>(a, grid, st) : gather_pages<TO, 64>(a, grid, st);
}

// The checks that append and gather share.
tkv_status row_args(const tkv_paged* c, const void* k, const void* v, int64_t rows, int64_t k_row, int64_t k_head,
                    int64_t v_row, int64_t v_head, int element, const int32_t* cu, int32_t* status, RowArgs* a) {
    if (check_paged(c) != TKV_OK || rows < 0 || rows > 0x7FFFFFFF || !cu || !aligned4(cu) || !aligned4(status)) return TKV_EINVAL;
    if (rows > 0 && (!k || !v)) return TKV_EINVAL;
    const int64_t E = 16 / element;   // blocks are moved in 16-byte pieces
    if (!aligned16(k) || !aligned16(v) || k_row < 0 || k_head < 0 || v_row < 0 || v_head < 0 || k_row % E || k_head % E ||
        v_row % E || v_head % E)
        return TKV_EINVAL;
    a->c = *c;
    a->k = k;
    a->v = v;
    a->cu = cu;
    a->status = status;
    a->rows = rows;
    a->k_row = k_row;
    a->k_head = k_head;
    a->v_row = v_row;
    a->v_head = v_head;
    a->page_shift = __builtin_ctz((unsigned)c->page_size);
    return TKV_OK;
}

}  // namespace

namespace tkv {

tkv_status check_paged(const tkv_paged* c) {
    if (!c || !c->pages || !c->page_table || !c->lengths) return TKV_EINVAL;
    if (c->kv_type != TKV_BF16 && c->kv_type != TKV_FP16 && c->kv_type != TKV_INT4) return TKV_EINVAL;
    if (c->head_dim != 64 && c->head_dim != 128) return TKV_EINVAL;
    if (c->page_size < 16 || c->page_size > 65536 || (c->page_size & (c->page_size - 1))) return TKV_EINVAL;
    if (c->batch < 1 || c->max_pages < 1 || c->num_kv_heads < 1 || c->num_pages < 1) return TKV_EINVAL;
    if ((int64_t)c->max_pages * c->page_size > (int64_t)1 << 30) return TKV_EINVAL;   // positions are int32
    if (!aligned16(c->pages) || !aligned4(c->page_table) || !aligned4(c->lengths) || !aligned4(c->k_gain) || !aligned4(c->v_gain)) return TKV_EINVAL;
    return TKV_OK;
}

}  // namespace tkv

extern "C" tkv_status tkv_paged_append(const tkv_paged* cache, const tkv_rotary* rotary, const void* k, const void* v,
                                       int32_t dtype, int64_t rows, int64_t k_row_stride, int64_t k_head_stride,
                                       int64_t v_row_stride, int64_t v_head_stride, const int32_t* cu_tokens,
                                       int32_t* status, void* stream) {
    RowArgs a{};
    if (dtype != TKV_BF16 && dtype != TKV_FP16) return TKV_EINVAL;
    if (row_args(cache, k, v, rows, k_row_stride, k_head_stride, v_row_stride, v_head_stride, 2, cu_tokens, status, &a) != TKV_OK)
        return TKV_EINVAL;
    if (cache->kv_type != TKV_INT4 && cache->kv_type != dtype) return TKV_EINVAL;
    int turn = kNone;
    if (rotary) {
        if (check_rotary(rotary, cache->head_dim, false) != TKV_OK) return TKV_EINVAL;
        a.table = reinterpret_cast<const float2*>(rotary->table);
        a.positions = rotary->positions;
        a.axis_stride = rotary->axis_stride;
        a.pairs = rotary->pairs;
        a.max_positions = rotary->max_positions;
        a.num_axes = rotary->num_axes;
        a.interleaved = rotary->interleaved != 0;
        a.table_16 = aligned16(rotary->table) && a.pairs % 2 == 0;
        a.sign = rotary->inverse ? -1.0f : 1.0f;
        for (int j = 0; j < 256; ++j) a.pair_axis[j] = j < rotary->pairs ? rotary->pair_axis[j] : 0;
        turn = a.interleaved ? (a.pairs % 4 == 0 ? kAdjacent : kAny) : (a.pairs % 16 == 0 ? kHalves : kAny);
    }
    if (rows == 0) return TKV_OK;
    a.units = cache->head_dim / 8 - (turn == kHalves ? a.pairs / 8 : 0);
    const int rows_a_block = kThreads / a.units;
    cudaError_t e = spread(a, (rows + rows_a_block - 1) / rows_a_block, kAppendCtas);
    if (e == cudaSuccess) {
        const dim3 grid((unsigned)((rows + rows_a_block - 1) / rows_a_block), a.lanes);
        e = dtype == TKV_BF16 ? append_type<__nv_bfloat16>(a, turn, grid, (cudaStream_t)stream)
                              : append_type<__half>(a, turn, grid, (cudaStream_t)stream);
    }
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return TKV_ECUDA;
    }
    return TKV_OK;
}

extern "C" tkv_status tkv_paged_gather(const tkv_paged* cache, void* k, void* v, int32_t dtype, int64_t rows,
                                       int64_t k_row_stride, int64_t k_head_stride, int64_t v_row_stride,
                                       int64_t v_head_stride, const int32_t* cu_tokens, int32_t* status, void* stream) {
    RowArgs a{};
    if (!is_dtype(dtype)) return TKV_EINVAL;
    if (row_args(cache, k, v, rows, k_row_stride, k_head_stride, v_row_stride, v_head_stride, dtype_size(dtype), cu_tokens,
                 status, &a) != TKV_OK)
        return TKV_EINVAL;
    if (!strides_apart(rows, k_row_stride, cache->num_kv_heads, k_head_stride, cache->head_dim) ||
        !strides_apart(rows, v_row_stride, cache->num_kv_heads, v_head_stride, cache->head_dim) || (rows > 0 && k == v))
        return TKV_EINVAL;
    if (rows == 0) return TKV_OK;
    const int64_t threads = rows * (cache->head_dim * dtype_size(dtype) / 16);
    cudaError_t e = spread(a, (threads + kThreads - 1) / kThreads, kGatherCtas);
    if (e == cudaSuccess) {
        const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads), a.lanes);
        cudaStream_t st = (cudaStream_t)stream;
        e = dtype == TKV_BF16   ? gather_type<__nv_bfloat16>(a, grid, st)
            : dtype == TKV_FP16 ? gather_type<__half>(a, grid, st)
                                : gather_type<float>(a, grid, st);
    }
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return TKV_ECUDA;
    }
    return TKV_OK;
}
