// What the kernels that bring rows into and out of a paged cache share: their arguments, the ways of rotating k.
#pragma once

#include "paged_tile.cuh"

namespace tkv {

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
//   kHalves    the partners of 8 channels lie `pairs` channels away, in another piece: pairs % 8 == 0 for 8-bit pages, and for the others
//              pairs % 16 == 0, in another block
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

// Rows into and out of 8-bit pages (paged_cache8.cu); the arguments are checked.
cudaError_t append_e4m3(RowArgs& a, int dtype, cudaStream_t st);
cudaError_t gather_e4m3(RowArgs& a, int dtype, cudaStream_t st);

}  // namespace tkv
