// Rows into and out of a paged cache: tkv_paged_append (k rotated on the way) and tkv_paged_gather.
//
// A step's rows are ragged: sequence b owns rows cu[b] .. cu[b + 1], which are the last positions of its
// lengths[b].  A thread takes one block of 16 channels of a row and walks over KV heads, K and V, so the
// 16 cosines and sines (or none, for V) stay in its registers; the eight (four) threads of a head's
// row and the rows of a record lie next to one another in memory.
//
// What bounds both is memory: 2 bytes a value on one side, 0.5625 (codes and scales) or 2 on the other.
#include <algorithm>

#include "paged.cuh"

using namespace tkv;

namespace {

constexpr int kThreads = 256;

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
    int lanes;                 // heads that the threads of a row take at once
    int page_shift;
    float sign;
    uint8_t pair_axis[256];
};

// Where row `row` of the step lies: page and position in the page; false for no row (behind the last
// sequence: *page = -2) and for a bad place (*page = -1: the position or the page is outside).
__device__ __forceinline__ bool place_of_row(const RowArgs& a, int64_t row, int64_t* page, int* off, int* position) {
    const int b = sequence_of_row(a.cu, a.c.batch, (int)row);
    *page = -2;
    if (b < 0) return false;
    const int pos = __ldg(a.c.lengths + b) - (__ldg(a.cu + b + 1) - (int)row);
    *page = -1;
    *position = pos;
    if (pos < 0 || (pos >> a.page_shift) >= a.c.max_pages) return false;
    const int p = __ldg(a.c.page_table + (int64_t)b * a.c.max_pages + (pos >> a.page_shift));
    if (p < 0 || p >= a.c.num_pages) return false;
    *page = p;
    *off = pos & (a.c.page_size - 1);
    return true;
}

// 16 values -> 16 codes (8 bytes) and the byte of their scale.
//   scale = e4m3(max |x| / (7 gain)), to nearest even; q = round(x / (scale * gain)), to nearest even,
// both quotients divided and not multiplied by a reciprocal, so that a tie stays one.  A block that
// holds an infinity or a NaN gets the NaN scale: it reads as NaN, not as something finite.
__device__ __forceinline__ uint2 quantise_block(const float (&x)[16], float gain, uint8_t* scale_byte) {
    uint32_t top = 0;   // |x| as bits: NaN > infinity > finite
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    const float amax = __uint_as_float(top);
    const bool bad = top >= 0x7F800000u;
    const __nv_fp8_storage_t s8 =
        bad ? (__nv_fp8_storage_t)0x7F : __nv_cvt_float_to_fp8(__fdiv_rn(amax, __fmul_rn(7.0f, gain)), __NV_SATFINITE, __NV_E4M3);
    const __half_raw hr = __nv_cvt_fp8_to_halfraw(s8, __NV_E4M3);
    const float step = __fmul_rn(__half2float(__half(hr)), gain);
    *scale_byte = (uint8_t)s8;
    uint32_t w[2] = {0, 0};
    const bool zero = bad || !(step > 0.0f);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float y = zero ? 0.0f : __fdiv_rn(x[i], step);
        const int q = __float2int_rn(fminf(fmaxf(y, -7.0f), 7.0f)) + 8;
        w[i >> 3] |= (uint32_t)q << (4 * (i & 7));
    }
    return make_uint2(w[0], w[1]);
}

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&x)[16]) {
    Vec16<T> a, b;
    a.u = *reinterpret_cast<const uint4*>(p);
    b.u = *(reinterpret_cast<const uint4*>(p) + 1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = to_float(a.e[i]);
        x[8 + i] = to_float(b.e[i]);
    }
}

template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&x)[16]) {
    constexpr int E = 16 / sizeof(T);
#pragma unroll
    for (int k = 0; k < 16 / E; ++k) {
        Vec16<T> o;
#pragma unroll
        for (int i = 0; i < E; ++i) o.e[i] = from_float<T>(x[k * E + i]);
        *(reinterpret_cast<uint4*>(p) + k) = o.u;
    }
}

// How a block of 16 channels of k is rotated.
//   kNone      not at all
//   kHalves    pairs % 16 == 0: the partners are a whole block, `pairs` channels away
//   kAdjacent  pairs % 8 == 0: the block holds its own 8 pairs
//   kAny       channel by channel, partners read one at a time
enum Turn { kNone, kHalves, kAdjacent, kAny };

// The block's 16 cosines and sines, one a channel (kHalves, kAny) or one a pair (kAdjacent: the first 8).
template <int TURN>
__device__ __forceinline__ void block_angles(const RowArgs& a, const uint8_t* axis_of, int64_t row, int own_position,
                                             int block, float2 (&cs)[16]) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < (TURN == kAdjacent ? 8 : 16); ++i) {
        const int ch = 16 * block + (TURN == kAdjacent ? 2 * i : i);
        cs[i] = make_float2(1.0f, 0.0f);
        if (ch >= 2 * a.pairs) continue;
        const int j = TURN == kAdjacent || (TURN == kAny && a.interleaved) ? ch >> 1 : ch < a.pairs ? ch : ch - a.pairs;
        const int p = a.positions ? __ldg(a.positions + (a.num_axes > 1 ? axis_of[j] : 0) * a.axis_stride + row) : own_position;
        cs[i] = table_at(a.table, a.pairs, a.max_positions, p, j, a.sign, &bad);
    }
    if (bad) raise_status(a.status, TKV_EINVAL);
}

// Block `block` of head row k, rotated.
template <typename T, int TURN>
__device__ __forceinline__ void rotated_block(const RowArgs& a, const T* k, int block, const float2 (&cs)[16], float (&x)[16]) {
    load16(k + 16 * block, x);
    if (TURN == kNone || 16 * block >= 2 * a.pairs) return;
    if (TURN == kHalves) {
        const bool first = 16 * block < a.pairs;
        float y[16];
        load16(k + 16 * block + (first ? a.pairs : -a.pairs), y);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[i] = first ? rotate_pair(x[i], y[i], cs[i]).x : rotate_pair(y[i], x[i], cs[i]).y;
    } else if (TURN == kAdjacent) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 y = rotate_pair(x[2 * i], x[2 * i + 1], cs[i]);
            x[2 * i] = y.x;
            x[2 * i + 1] = y.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int ch = 16 * block + i;
            if (ch >= 2 * a.pairs) continue;
            const bool first = a.interleaved ? !(ch & 1) : ch < a.pairs;
            const float other = to_float(k[a.interleaved ? ch ^ 1 : first ? ch + a.pairs : ch - a.pairs]);
            x[i] = first ? rotate_pair(x[i], other, cs[i]).x : rotate_pair(other, x[i], cs[i]).y;
        }
    }
}

template <typename T, int D, bool INT4, int TURN>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ RowArgs a) {
    constexpr int NB = D / 16;
    __shared__ uint8_t axis_of[256];
    if (TURN != kNone && a.num_axes > 1) {
        axis_of[threadIdx.x] = a.pair_axis[threadIdx.x];
        __syncthreads();
    }
    // block fastest, then the row, then the head lane: eight threads a head's row, whole records a warp
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int block = (int)(i % NB);
    const int64_t row = i / NB;
    const int lane = blockIdx.y;
    if (row >= a.rows) return;
    int64_t page;
    int off, position;
    if (!place_of_row(a, row, &page, &off, &position)) {
        if (page == -1 && block == 0 && lane == 0) raise_status(a.status, TKV_ECAPACITY);
        return;
    }
    float2 cs[16];
    if (TURN != kNone && 16 * block < 2 * a.pairs) block_angles<TURN>(a, axis_of, row, position, block, cs);
    const T* k = reinterpret_cast<const T*>(a.k) + row * a.k_row;
    const T* v = reinterpret_cast<const T*>(a.v) + row * a.v_row;
    for (int h = lane; h < a.c.num_kv_heads; h += a.lanes) {
        float x[16], y[16];
        rotated_block<T, TURN>(a, k + h * a.k_head, block, cs, x);
        load16(v + h * a.v_head + 16 * block, y);
        if (INT4) {
            using R = Record<D>;
            const int r = off & 15;
            uint8_t* rec = reinterpret_cast<uint8_t*>(a.c.pages) +
                           ((page * a.c.num_kv_heads + h) * (a.c.page_size / kGroup) + (off >> 4)) * R::bytes;
            const float kg = a.c.k_gain ? __ldg(a.c.k_gain + h) : 1.0f, vg = a.c.v_gain ? __ldg(a.c.v_gain + h) : 1.0f;
            uint8_t s;
            const uint2 kc = quantise_block(x, kg, &s);
            *reinterpret_cast<uint2*>(rec + R::k_codes + r * (D / 2) + 8 * block) = kc;
            rec[R::k_scales + r * NB + block] = s;
            const uint2 vc = quantise_block(y, vg, &s);
            *reinterpret_cast<uint2*>(rec + R::v_codes + r * (D / 2) + 8 * block) = vc;
            rec[R::v_scales + block * 16 + r] = s;
        } else {
            T* base = reinterpret_cast<T*>(a.c.pages) + ((page * a.c.num_kv_heads + h) * 2 * a.c.page_size + off) * D + 16 * block;
            store16(base, x);
            store16(base + (int64_t)a.c.page_size * D, y);
        }
    }
}

// 8 bytes of codes -> the values q * scale * gain: the product of code and scale is exact, one rounding.
__device__ __forceinline__ void expand_block(uint2 w, uint8_t scale_byte, float gain, float (&x)[16]) {
    const __half_raw hr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)scale_byte, __NV_E4M3);
    const float s = __half2float(__half(hr));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int q = (int)(((i < 8 ? w.x : w.y) >> (4 * (i & 7))) & 15u) - 8;
        x[i] = __fmul_rn(__fmul_rn((float)q, s), gain);
    }
}

// TO: element type of the outputs; T: of 16-bit pages.
template <typename TO, typename T, int D, bool INT4>
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ RowArgs a) {
    constexpr int NB = D / 16;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int block = (int)(i % NB);
    const int64_t row = i / NB;
    const int lane = blockIdx.y;
    if (row >= a.rows) return;
    int64_t page;
    int off = 0, position;
    const bool good = place_of_row(a, row, &page, &off, &position);
    if (page == -2) return;
    if (!good && block == 0 && lane == 0) raise_status(a.status, TKV_ECAPACITY);
    TO* k = reinterpret_cast<TO*>(const_cast<void*>(a.k)) + row * a.k_row;
    TO* v = reinterpret_cast<TO*>(const_cast<void*>(a.v)) + row * a.v_row;
    for (int h = lane; h < a.c.num_kv_heads; h += a.lanes) {
        float x[16], y[16];
        if (!good) {
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = y[j] = __int_as_float(0x7FC00000);
        } else if (INT4) {
            using R = Record<D>;
            const int r = off & 15;
            const uint8_t* rec = reinterpret_cast<const uint8_t*>(a.c.pages) +
                                 ((page * a.c.num_kv_heads + h) * (a.c.page_size / kGroup) + (off >> 4)) * R::bytes;
            const uint2 kc = *reinterpret_cast<const uint2*>(rec + R::k_codes + r * (D / 2) + 8 * block);
            const uint2 vc = *reinterpret_cast<const uint2*>(rec + R::v_codes + r * (D / 2) + 8 * block);
            const uint8_t ks = rec[R::k_scales + r * NB + block], vs = rec[R::v_scales + block * 16 + r];
            expand_block(kc, ks, a.c.k_gain ? __ldg(a.c.k_gain + h) : 1.0f, x);
            expand_block(vc, vs, a.c.v_gain ? __ldg(a.c.v_gain + h) : 1.0f, y);
        } else {
            const T* base = reinterpret_cast<const T*>(a.c.pages) + ((page * a.c.num_kv_heads + h) * 2 * a.c.page_size + off) * D + 16 * block;
            load16(base, x);
            load16(base + (int64_t)a.c.page_size * D, y);
        }
        store16(k + h * a.k_head + 16 * block, x);
        store16(v + h * a.v_head + 16 * block, y);
    }
}

// Threads of a launch: a row's blocks in x, heads at once in y.  A thread walks over up to 8 heads
// as long as a wave of threads is left (the table and the row's place are then read once for them).
cudaError_t geometry(RowArgs& a, dim3* grid) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int64_t blocks = a.rows * (a.c.head_dim / 16);
    const int hkv = a.c.num_kv_heads;
    const int per_thread = (int)std::min<int64_t>(8, std::max<int64_t>(1, blocks * hkv / ((int64_t)sms * 1024)));
    a.lanes = std::min(65535, (hkv + per_thread - 1) / per_thread);
    *grid = dim3((unsigned)((blocks + kThreads - 1) / kThreads), a.lanes);
    return cudaSuccess;
}

template <typename T, int D, bool INT4>
void append_turn(const RowArgs& a, int turn, dim3 grid, cudaStream_t st) {
    if (turn == kNone) append_kernel<T, D, INT4, kNone><<<grid, kThreads, 0, st>>>(a);
    else if (turn == kHalves) append_kernel<T, D, INT4, kHalves><<<grid, kThreads, 0, st>>>(a);
    else if (turn == kAdjacent) append_kernel<T, D, INT4, kAdjacent><<<grid, kThreads, 0, st>>>(a);
    else append_kernel<T, D, INT4, kAny><<<grid, kThreads, 0, st>>>(a);
}

template <typename T>
void append_type(const RowArgs& a, int turn, dim3 grid, cudaStream_t st) {
    const bool int4 = a.c.kv_type == TKV_INT4;
    if (a.c.head_dim == 128)
        int4 ? append_turn<T, 128, true>(a, turn, grid, st) : append_turn<T, 128, false>(a, turn, grid, st);
    else
        int4 ? append_turn<T, 64, true>(a, turn, grid, st) : append_turn<T, 64, false>(a, turn, grid, st);
}

template <typename TO, int D>
void gather_pages(const RowArgs& a, dim3 grid, cudaStream_t st) {
    if (a.c.kv_type == TKV_INT4) gather_kernel<TO, __half, D, true><<<grid, kThreads, 0, st>>>(a);
    else if (a.c.kv_type == TKV_FP16) gather_kernel<TO, __half, D, false><<<grid, kThreads, 0, st>>>(a);
    else gather_kernel<TO, __nv_bfloat16, D, false><<<grid, kThreads, 0, st>>>(a);
}

template <typename TO>
void gather_type(const RowArgs& a, dim3 grid, cudaStream_t st) {
    if (a.c.head_dim == 128) gather_pages<TO, 128>(a, grid, st);
    else gather_pages<TO, 64>(a, grid, st);
}

// The checks that append and gather share.
tkv_status row_args(const tkv_paged* c, const void* k, const void* v, int64_t rows, int64_t k_row, int64_t k_head,
                    int64_t v_row, int64_t v_head, int element, const int32_t* cu, RowArgs* a) {
    if (check_paged(c) != TKV_OK || rows < 0 || rows > 0x7FFFFFFF || !cu) return TKV_EINVAL;
    if (rows > 0 && (!k || !v)) return TKV_EINVAL;
    const int64_t E = 16 / element;   // blocks are moved in 16-byte pieces
    if (!aligned16(k) || !aligned16(v) || k_row < 0 || k_head < 0 || v_row < 0 || v_head < 0 || k_row % E || k_head % E ||
        v_row % E || v_head % E)
        return TKV_EINVAL;
    a->c = *c;
    a->k = k;
    a->v = v;
    a->cu = cu;
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
    if (!aligned16(c->pages)) return TKV_EINVAL;
    return TKV_OK;
}

}  // namespace tkv

extern "C" tkv_status tkv_paged_append(const tkv_paged* cache, const tkv_rotary* rotary, const void* k, const void* v,
                                       int32_t dtype, int64_t rows, int64_t k_row_stride, int64_t k_head_stride,
                                       int64_t v_row_stride, int64_t v_head_stride, const int32_t* cu_tokens,
                                       int32_t* status, void* stream) {
    RowArgs a{};
    if (dtype != TKV_BF16 && dtype != TKV_FP16) return TKV_EINVAL;
    if (row_args(cache, k, v, rows, k_row_stride, k_head_stride, v_row_stride, v_head_stride, 2, cu_tokens, &a) != TKV_OK)
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
        a.sign = rotary->inverse ? -1.0f : 1.0f;
        for (int j = 0; j < 256; ++j) a.pair_axis[j] = j < rotary->pairs ? rotary->pair_axis[j] : 0;
        turn = a.interleaved ? (a.pairs % 8 == 0 ? kAdjacent : kAny) : (a.pairs % 16 == 0 ? kHalves : kAny);
    }
    if (rows == 0) return TKV_OK;
    a.status = status;
    dim3 grid;
    cudaError_t e = geometry(a, &grid);
    if (e == cudaSuccess) {
        if (dtype == TKV_BF16) append_type<__nv_bfloat16>(a, turn, grid, (cudaStream_t)stream);
        else append_type<__half>(a, turn, grid, (cudaStream_t)stream);
        e = cudaGetLastError();
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
                 &a) != TKV_OK)
        return TKV_EINVAL;
    if (!strides_apart(rows, k_row_stride, cache->num_kv_heads, k_head_stride, cache->head_dim) ||
        !strides_apart(rows, v_row_stride, cache->num_kv_heads, v_head_stride, cache->head_dim) || (rows > 0 && k == v))
        return TKV_EINVAL;
    if (rows == 0) return TKV_OK;
    a.status = status;
    dim3 grid;
    cudaError_t e = geometry(a, &grid);
    if (e == cudaSuccess) {
        cudaStream_t st = (cudaStream_t)stream;
        if (dtype == TKV_BF16) gather_type<__nv_bfloat16>(a, grid, st);
        else if (dtype == TKV_FP16) gather_type<__half>(a, grid, st);
        else gather_type<float>(a, grid, st);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return TKV_ECUDA;
    }
    return TKV_OK;
}
