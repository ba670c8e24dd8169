// Rotary positions with one or several axes: tkv_rope.
//
// Pair j of a head (of `pairs` rotated ones) turns by the angle of position p = positions[axis(j)][row]:
//   y0 = x0 cos - x1 sin,  y1 = x1 cos + x0 sin
// with cos and sin from the caller's table, row p, column j.  The rotation is orthogonal, so its
// gradient is the rotation by the negated angle: the same kernel with the sine's sign turned.
//
// What bounds it is memory: every value is read and written once and costs three operations.  A thread
// keeps the cosines and sines of its piece of a head in registers and walks over heads of its
// row, so the table (8 bytes a pair, fp32) is read once a row and not once a head.
#include <algorithm>

#include "paged.cuh"

using namespace tkv;

namespace {

constexpr int kThreads = 256;

// CTAs on an SM at once, by their registers.  16-byte pieces, 4,096 rows of 32 heads of 128 in bf16, halves: 13.4 us with five,
// 14.0 with four, 14.6 with six (spills); adjacent pairs, which need half the angles, 16,384 rows of 64 heads: 84 us with
// eight, 92 with six; fp32, 5,003 rows of 13 heads of 80: 8.9 us with six, 9.3 with five, 10.0 with eight.
template <typename T, int BYTES, bool INTERLEAVED>
constexpr int ctas_of() {
    return BYTES < 16 || sizeof(T) == 4 ? 6 : INTERLEAVED ? 8 : 5;
}

template <int BYTES> struct Word;
template <> struct Word<16> { using type = uint4; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<2> { using type = uint16_t; };

struct RopeArgs {
    const void* x;
    void* out;
    const float2* table;
    const int32_t* positions;
    int32_t* status;
    int64_t rows, axis_stride, x_row, x_head, out_row, out_head;
    int heads, head_dim, pairs, max_positions, num_axes, interleaved;
    int lanes;       // heads that the threads of a row take at once
    bool copy_rest;  // channels behind the rotated ones are copied (out is not x)
    bool table_16;   // two pairs of the table lie on 16 bytes
    float sign;
    uint8_t pair_axis[256];
};

// Pieces of BYTES bytes, E elements: 16 bytes where everything allows it, fewer where alignments or numbers of pairs do not
// (16,000 rows of 16 heads of 74 in bf16, pairs 37 apart, in 2-byte pieces: 20 us, 76 MB, 3.8 TB/s, eight times the loads and
// stores of 16-byte pieces; one head at a time 31, a pair a thread 74).  Pieces of a head: with halves, piece i takes channels [i E, i E + E) and their partners `pairs` further on;
// with adjacent pairs, its own E / 2 pairs.  Behind the rotated pieces come the copied ones.  A block holds kThreads /
// pieces rows; blockIdx.y is the first head.  16,384 rows of 64 heads of 128 in bf16, three axes: 89 us (545 MB, 6.1 TB/s).
template <typename T, int BYTES, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, ctas_of<T, BYTES, INTERLEAVED>()) rope_kernel(const __grid_constant__ RopeArgs a) {
    let_next_start();
    wait_for_previous();
    constexpr int E = BYTES / sizeof(T);
    constexpr int NP = INTERLEAVED ? E / 2 : E;   // pairs of a piece
    using W = typename Word<BYTES>::type;
    union Piece {
        W u;
        T e[E];
    };
    const int rotated = a.pairs / NP;
    const int pieces = rotated + (a.copy_rest ? (a.head_dim - 2 * a.pairs) / E : 0);
    const int rows_here = kThreads / pieces;
    const int in_block = threadIdx.x / pieces, piece = threadIdx.x - in_block * pieces;
    const int64_t row = (int64_t)blockIdx.x * rows_here + in_block;
    if (in_block >= rows_here || row >= a.rows) return;
    const bool turned = piece < rotated;
    const int first = turned ? piece * (INTERLEAVED ? E : NP) : 2 * a.pairs + (piece - rotated) * E;
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_row + blockIdx.y * a.x_head + first;
    T* out = reinterpret_cast<T*>(a.out) + row * a.out_row + blockIdx.y * a.out_head + first;
    const bool two = !INTERLEAVED && turned;
    // The next heads' values are read while the last ones' are turned, the first ones' before the angles; of small pieces
    // several heads at once, so that as many bytes are on their way.
    constexpr int U = BYTES == 16 ? 1 : BYTES == 8 ? 2 : 4;
    Piece lo[U], hi[U], next_lo[U], next_hi[U];
    auto read = [&](int h) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h + u * a.lanes >= a.heads) break;
            next_lo[u].u = *reinterpret_cast<const W*>(x);
            next_hi[u].u = two ? *reinterpret_cast<const W*>(x + a.pairs) : W();
            x += a.lanes * a.x_head;
        }
    };
    read(blockIdx.y);
    float2 cs[NP];
    if (turned) {
        int p[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < a.num_axes) p[i] = a.positions[i * a.axis_stride + row];
        load_angles<NP>(a, p, piece * NP, cs);
    }
    for (int h = blockIdx.y; h < a.heads; h += U * a.lanes) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            lo[u] = next_lo[u];
            hi[u] = next_hi[u];
        }
        read(h + U * a.lanes);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h + u * a.lanes >= a.heads) break;
            if (turned) {
#pragma unroll
                for (int k = 0; k < NP; ++k) {
                    T& e0 = INTERLEAVED ? lo[u].e[(2 * k) % E] : lo[u].e[k];
                    T& e1 = INTERLEAVED ? lo[u].e[(2 * k + 1) % E] : hi[u].e[k];
                    const float2 y = rotate_pair(to_float(e0), to_float(e1), cs[k]);
                    e0 = from_float<T>(y.x);
                    e1 = from_float<T>(y.y);
                }
            }
            *reinterpret_cast<W*>(out) = lo[u].u;
            if (two) *reinterpret_cast<W*>(out + a.pairs) = hi[u].u;
            out += a.lanes * a.out_head;
        }
    }
}

// What no piece fits (adjacent pairs that are not aligned to a pair, heads of more pieces than a block has threads): a thread
// takes one pair (or one copied channel) of a head.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_pairs_kernel(const __grid_constant__ RopeArgs a) {
    let_next_start();
    wait_for_previous();
    const int rest = a.copy_rest ? a.head_dim - 2 * a.pairs : 0;
    const uint32_t per_head = a.pairs + rest;
    const int64_t total = a.rows * a.heads * per_head;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int64_t rh = i / per_head;
        const int j = (int)(i - rh * per_head);
        const int64_t row = rh / a.heads;
        const int h = (int)(rh - row * a.heads);
        const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_row + h * a.x_head;
        T* out = reinterpret_cast<T*>(a.out) + row * a.out_row + h * a.out_head;
        if (j >= a.pairs) {
            out[a.pairs + j] = x[a.pairs + j];
            continue;
        }
        bool bad = false;
        const int p = a.positions[(a.num_axes > 1 ? a.pair_axis[j] : 0) * a.axis_stride + row];
        const float2 cs = table_at(a.table, a.pairs, a.max_positions, p, j, a.sign, &bad);
        if (bad) raise_status(a.status, TKV_EINVAL);
        const int i0 = a.interleaved ? 2 * j : j, i1 = a.interleaved ? 2 * j + 1 : j + a.pairs;
        const float2 y = rotate_pair(to_float(x[i0]), to_float(x[i1]), cs);
        out[i0] = from_float<T>(y.x);
        out[i1] = from_float<T>(y.y);
    }
}

template <typename T, int BYTES, bool INTERLEAVED>
cudaError_t launch_pieces(RopeArgs& a, int pieces, int sms, cudaStream_t st) {
    const int rows_here = kThreads / pieces;
    const int64_t blocks = (a.rows + rows_here - 1) / rows_here;
    a.lanes = spread_heads(blocks, a.heads, (int64_t)sms * ctas_of<T, BYTES, INTERLEAVED>(), 16);
    return launch_behind(rope_kernel<T, BYTES, INTERLEAVED>, dim3((unsigned)blocks, a.lanes), kThreads, 0, st, a);
}

// `grain`: the bytes that every address and stride of x and out is a multiple of, as a power of two.
template <typename T>
cudaError_t launch(RopeArgs& a, int grain, cudaStream_t st) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int rest = a.copy_rest ? a.head_dim - 2 * a.pairs : 0, least = a.interleaved ? 2 : 1;
    for (int bytes = std::min(16, grain); bytes >= least * (int)sizeof(T); bytes /= 2) {
        const int E = bytes / (int)sizeof(T), np = E / least;
        if (a.pairs % np || rest % E) continue;
        const int pieces = a.pairs / np + rest / E;
        if (pieces > kThreads) break;
        if (a.interleaved) {
            if (bytes == 16) return launch_pieces<T, 16, true>(a, pieces, sms, st);
            if (bytes == 8) return launch_pieces<T, 8, true>(a, pieces, sms, st);
            if constexpr (sizeof(T) == 2) return launch_pieces<T, 4, true>(a, pieces, sms, st);
        }
        if (bytes == 16) return launch_pieces<T, 16, false>(a, pieces, sms, st);
        if (bytes == 8) return launch_pieces<T, 8, false>(a, pieces, sms, st);
        if (bytes == 4) return launch_pieces<T, 4, false>(a, pieces, sms, st);
        if constexpr (sizeof(T) == 2) return launch_pieces<T, 2, false>(a, pieces, sms, st);
    }
    const int64_t total = a.rows * a.heads * (a.pairs + rest);
    const int grid = (int)std::min<int64_t>((total + kThreads - 1) / kThreads, (int64_t)sms * 64);
    return launch_behind(rope_pairs_kernel<T>, dim3(grid), kThreads, 0, st, a);
}

}  // namespace

namespace tkv {

bool strides_apart(int64_t rows, int64_t row_stride, int64_t heads, int64_t head_stride, int64_t width) {
    if (row_stride < 0 || head_stride < 0) return false;
    if (heads == 1) return rows == 1 || row_stride >= width;
    if (rows == 1) return head_stride >= width;
    if (row_stride >= head_stride) return head_stride >= width && row_stride >= (heads - 1) * head_stride + width;
    return row_stride >= width && head_stride >= (rows - 1) * row_stride + width;
}

tkv_status check_rotary(const tkv_rotary* r, int head_dim, bool need_positions) {
    if (!r || !r->table || (reinterpret_cast<uintptr_t>(r->table) & 7u) || !aligned4(r->positions)) return TKV_EINVAL;
    if (need_positions && !r->positions) return TKV_EINVAL;
    if (r->max_positions < 1 || r->pairs < 1 || r->pairs > 256 || 2 * r->pairs > head_dim) return TKV_EINVAL;
    if (r->num_axes < 1 || r->num_axes > 4 || (r->num_axes > 1 && !r->positions)) return TKV_EINVAL;
    if (r->axis_stride < 0) return TKV_EINVAL;
    for (int j = 0; j < r->pairs; ++j)
        if (r->pair_axis[j] >= r->num_axes) return TKV_EINVAL;
    return TKV_OK;
}

}  // namespace tkv

extern "C" tkv_status tkv_rope(const tkv_rotary* rotary, const void* x, void* out, int32_t dtype, int64_t rows,
                               int32_t heads, int32_t head_dim, int64_t x_row_stride, int64_t x_head_stride,
                               int64_t out_row_stride, int64_t out_head_stride, int32_t* status, void* stream) {
    if (!is_dtype(dtype) || rows < 0 || rows > 0x7FFFFFFF || heads < 1 || head_dim < 2 || head_dim > 65536)
        return TKV_EINVAL;
    if (check_rotary(rotary, head_dim, true) != TKV_OK) return TKV_EINVAL;
    if (rows == 0) return TKV_OK;
    if (!x || !out || x_row_stride < 0 || x_head_stride < 0 || !aligned4(status)) return TKV_EINVAL;
    const uintptr_t size = dtype_size(dtype);
    if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) & (size - 1)) return TKV_EINVAL;
    if (!strides_apart(rows, out_row_stride, heads, out_head_stride, head_dim)) return TKV_EINVAL;
    const bool in_place = x == out;
    if (in_place && ((rows > 1 && x_row_stride != out_row_stride) || (heads > 1 && x_head_stride != out_head_stride)))
        return TKV_EINVAL;
    RopeArgs a{};
    a.x = x;
    a.out = out;
    a.table = reinterpret_cast<const float2*>(rotary->table);
    a.positions = rotary->positions;
    a.status = status;
    a.rows = rows;
    a.axis_stride = rotary->axis_stride;
    a.x_row = x_row_stride;
    a.x_head = x_head_stride;
    a.out_row = out_row_stride;
    a.out_head = out_head_stride;
    a.heads = heads;
    a.head_dim = head_dim;
    a.pairs = rotary->pairs;
    a.max_positions = rotary->max_positions;
    a.num_axes = rotary->num_axes;
    a.interleaved = rotary->interleaved != 0;
    a.copy_rest = !in_place && head_dim > 2 * rotary->pairs;
    a.table_16 = aligned16(rotary->table) && a.pairs % 2 == 0;
    a.sign = rotary->inverse ? -1.0f : 1.0f;
    for (int j = 0; j < 256; ++j) a.pair_axis[j] = j < rotary->pairs ? rotary->pair_axis[j] : 0;
    const uint64_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out) | size * (uint64_t)(x_row_stride | x_head_stride | out_row_stride | out_head_stride) | 16;
    const int grain = (int)(all & (0 - all));
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = dtype == TKV_BF16   ? launch<__nv_bfloat16>(a, grain, st)
                          : dtype == TKV_FP16 ? launch<__half>(a, grain, st)
                                              : launch<float>(a, grain, st);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return TKV_ECUDA;
    }
    return TKV_OK;
}
