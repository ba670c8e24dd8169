// Rows into and out of 8-bit pages (the records are described in paged.cuh): the E4M3 side of tkv_paged_append and tkv_paged_gather.
//
// A block of 16 positions of a KV head has one exponent for K and one for V.  A step brings it new rows at offsets [f, g):
//   a = max |x| over what is finite of them (k after its rotation),  e_new = least e with a <= 448 2^e, within -32 .. 31
//   e = e_new if f = 0, else max(e, e_new);  code = e4m3(x 2^-e), to nearest even, saturating; an infinity or a NaN is NaN
// and where e grows the rows [0, f) are written anew: value 2^-e, rounded once more (exact but for what becomes subnormal).
// So a block and not a row is what one CTA owns: four warps take its K, two or four its V, and walk over KV heads; a thread has
// two rows of 8 channels, whose cosines and sines it finds once for all heads, and the CTA meets once a head, for the
// maxima.
//
// A CTA's block.  A sequence's n rows touch at most (n + 14) / 16 + 1 blocks, so the slots from (cu[b] >> 4) + 2 b up to
// (cu[b + 1] >> 4) + 2 (b + 1) hold them all wherever they begin: slots are CTAs, the sequence of a slot is found by a search over cu,
// 32 lanes at a time (one trip to memory up to 32 sequences, two up to 1,024), and at most 2 slots a sequence stay idle.
//
// What bounds both is memory: 2 bytes a value on one side, 1 on the other.
#include "paged_rows.cuh"

using namespace tkv;

namespace {

constexpr int kAppendCtas = 3, kGatherCtas = 6;   // on an SM at once, by their registers

template <int D>
struct Threads {
    static constexpr int k = 128, v = D, all = k + v;   // 16 rows of D / 8 pieces of 8 channels: two (of K at d 64: one) a thread of K, two of V
};

// A block of a step: its new rows are those at offsets [lo, hi), row0 + offset in the step's tensors.
struct Block {
    int64_t first, row0, page;   // position of offset 0; page -1: it has no place
    int lo, hi;
};

// The block of a slot; false: the slot has none.  Every lane of the warp calls it.
__device__ __forceinline__ bool find_block(const RowArgs& a, int64_t slot, Block* k) {
    const int lane = threadIdx.x & 31;
    int begin = 0, len = a.c.batch;   // sequences [begin, begin + len) are not known yet; those before begin at or before the slot
    while (len > 0) {
        const int step = (len + 31) / 32, at = lane * step;
        const bool before = at < len && (int64_t)(a.cu[begin + at] >> 4) + 2 * (int64_t)(begin + at) <= slot;
        const int n = __popc(__ballot_sync(0xffffffffu, before));
        if (n == 0) break;
        const int known = (n - 1) * step + 1;
        begin += known;
        len = min(step - 1, len - known);
    }
    const int b = begin - 1;
    if (b < 0) return false;
    const int64_t c0 = a.cu[b], c1 = a.cu[b + 1], length = a.c.lengths[b];
    const int64_t p0 = length - (c1 - c0);   // position of the sequence's first row
    const int64_t block = (p0 >> 4) + (slot - ((c0 >> 4) + 2 * (int64_t)b));
    k->first = block * 16;
    if (c1 <= c0 || k->first >= length || slot < (c0 >> 4) + 2 * (int64_t)b) return false;
    k->lo = (int)max((int64_t)0, p0 - k->first);
    k->hi = (int)min((int64_t)16, length - k->first);
    k->row0 = c0 + (k->first - p0);
    k->lo = (int)max((int64_t)k->lo, min((int64_t)16, -k->row0));          // the rows that there are, whatever cu holds
    k->hi = (int)min((int64_t)k->hi, max((int64_t)0, a.rows - k->row0));
    if (k->lo >= k->hi) return false;
    k->page = -1;
    const int64_t column = k->first >> a.page_shift;
    if (k->first >= 0 && column < a.c.max_pages) {
        const int p = a.c.page_table[(int64_t)b * a.c.max_pages + column];
        if (p >= 0 && p < a.c.num_pages) k->page = p;
    }
    return true;
}

// The least e with amax <= 448 * 2^e (448 = 1.75 * 2^8), within the format's range.
__device__ __forceinline__ int exponent_for(float amax) {
    return block_exponent(((int)(__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 127 - 8);
}

// Two values as codes, the first in the low byte.
__device__ __forceinline__ uint32_t code_pair(float a, float b) { return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3); }

// Four codes as values.
__device__ __forceinline__ void decode4(uint32_t w, float scale, float (&x)[4]) {
    const float2 a = __half22float2(e4m3_pair((uint16_t)w)), b = __half22float2(e4m3_pair((uint16_t)(w >> 16)));
    x[0] = a.x * scale;
    x[1] = a.y * scale;
    x[2] = b.x * scale;
    x[3] = b.y * scale;
}

// A thread's pieces of a record: 8 channels from `channel` on, of the rows r[0] and r[1] (16: none), and where they lie.
struct Pieces {
    int channel, r[2], at[2];
    bool is_k;
};

template <int D>
__device__ __forceinline__ Pieces pieces_of_thread() {
    Pieces p;
    p.is_k = threadIdx.x < Threads<D>::k;
    if (p.is_k) {
        const int t = threadIdx.x, chunk = t & (D / 8 - 1);
        p.channel = 8 * chunk;
        p.r[0] = t / (D / 8);
        p.r[1] = D == 128 ? p.r[0] + 8 : 16;
#pragma unroll
        for (int i = 0; i < 2; ++i) p.at[i] = (chunk >> 3) * 1024 + p.r[i] * 64 + (chunk & 7) * 8;
    } else {
        const int t = threadIdx.x - Threads<D>::k, chunk = (t >> 2) & (D / 8 - 1), half = t / (D / 2);
        p.channel = 8 * chunk;
        p.r[0] = half * 8 + (t & 3) * 2;
        p.r[1] = p.r[0] + 1;
        p.at[0] = Record8<D>::v_codes + half * (8 * D) + chunk * 64 + (t & 3) * 16;
        p.at[1] = p.at[0] + 1;   // every other byte each
    }
    return p;
}

// blockIdx.y: the first head.
template <typename T, int D, int TURN>
__global__ void __launch_bounds__(Threads<D>::all, kAppendCtas) append8_kernel(const __grid_constant__ RowArgs a) {
    let_next_start();
    wait_for_previous();
    using R = Record8<D>;
    Block blk;
    if (!find_block(a, blockIdx.x, &blk)) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (blk.page < 0) {
        if (tid == 0 && blockIdx.y == 0) raise_status(a.status, TKV_ECAPACITY);
        return;
    }
    __shared__ uint32_t maxima[2][Threads<D>::all / 32];
    const Pieces p = pieces_of_thread<D>();
    const bool is_new[2] = {p.r[0] >= blk.lo && p.r[0] < blk.hi, p.r[1] >= blk.lo && p.r[1] < blk.hi};
    const int64_t stride = p.is_k ? a.k_row : a.v_row, head = p.is_k ? a.k_head : a.v_head;
    const T* from[2];
    uint4 raw[2] = {};
#pragma unroll
    for (int i = 0; i < 2; ++i) from[i] = reinterpret_cast<const T*>(p.is_k ? a.k : a.v) + (blk.row0 + p.r[i]) * stride + blockIdx.y * head + p.channel;
    auto read = [&](int h) {   // the next head's values, while the last one's are worked on
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (is_new[i] && h < a.c.num_kv_heads) raw[i] = *reinterpret_cast<const uint4*>(from[i]);
            from[i] += a.lanes * head;
        }
    };
    read(blockIdx.y);
    // the angles of the thread's rows: halves: with the sign that the partner's product has
    constexpr int NCS = TURN == kHalves ? 8 : TURN == kAdjacent ? 4 : 1;
    const bool turned = TURN != kNone && p.is_k && p.channel < 2 * a.pairs, first = p.channel < a.pairs;
    float2 cs[2][NCS];
    if ((TURN == kHalves || TURN == kAdjacent) && turned) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!is_new[i]) continue;
            int pos[4] = {(int)(blk.first + p.r[i]), 0, 0, 0};
            if (a.positions) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (x < a.num_axes) pos[x] = a.positions[x * a.axis_stride + blk.row0 + p.r[i]];
            }
            load_angles<NCS>(a, pos, TURN == kHalves ? (first ? p.channel : p.channel - a.pairs) : p.channel / 2, cs[i]);
            if (TURN == kHalves && first) {
#pragma unroll
                for (int j = 0; j < NCS; ++j) cs[i][j].y = -cs[i][j].y;
            }
        }
    }
    const int64_t head_bytes = (int64_t)(a.c.page_size >> 4) * R::bytes;
    uint8_t* rec = reinterpret_cast<uint8_t*>(a.c.pages) + (blk.page * a.c.num_kv_heads + blockIdx.y) * head_bytes +
                   (((int)blk.first & (a.c.page_size - 1)) >> 4) * R::bytes;
    const int partner = lane + (first ? a.pairs / 8 : -(a.pairs / 8));
    int turn = 0;
#pragma unroll 1
    for (int h = blockIdx.y; h < a.c.num_kv_heads; h += a.lanes, rec += a.lanes * head_bytes, turn ^= 1) {
        int* exponent = reinterpret_cast<int*>(rec + R::exponents) + !p.is_k;
        int e_old = kLowestExponent;
        if (blk.lo > 0) e_old = block_exponent(*exponent);
        float x[2][8];
        const uint4 now[2] = {raw[0], raw[1]};
        unpack<T>(now[0], x[0]);
        unpack<T>(now[1], x[1]);
        read(h + a.lanes);
        if (TURN == kHalves && p.is_k) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint4 other;
                other.x = __shfl_sync(0xffffffffu, now[i].x, partner);
                other.y = __shfl_sync(0xffffffffu, now[i].y, partner);
                other.z = __shfl_sync(0xffffffffu, now[i].z, partner);
                other.w = __shfl_sync(0xffffffffu, now[i].w, partner);
                if (turned && is_new[i]) {
                    float y[8];
                    unpack<T>(other, y);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[i][j] = __fadd_rn(__fmul_rn(x[i][j], cs[i][j % NCS].x), __fmul_rn(y[j], cs[i][j % NCS].y));
                }
            }
        } else if (TURN == kAdjacent && turned) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (is_new[i]) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 z = rotate_pair(x[i][2 * j], x[i][2 * j + 1], cs[i][j % NCS]);
                        x[i][2 * j] = z.x;
                        x[i][2 * j + 1] = z.y;
                    }
                }
        } else if (TURN == kAny && turned) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int64_t row = blk.row0 + p.r[i];
                if (is_new[i]) turn_any(a, reinterpret_cast<const T*>(a.k) + row * a.k_row + h * a.k_head, row, (int)(blk.first + p.r[i]), p.channel >> 3, x[i]);
            }
        }
        // the largest of the block: NaN counts for nothing here, and neither does an infinity, which becomes one
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (is_new[i]) {
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[i][j]));
            }
        if (top == INFINITY) {
            top = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (fabsf(x[i][j]) == INFINITY) x[i][j] = __int_as_float(0x7FC00000);
                    if (is_new[i]) top = fmaxf(top, fabsf(x[i][j]));
                }
        }
        const uint32_t warp_max = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
        if (lane == 0) maxima[turn][warp] = warp_max;
        __syncthreads();   // the next head's maxima lie in the other half, so once a head is enough
        uint32_t most = 0;
        if (p.is_k) {
#pragma unroll
            for (int w = 0; w < Threads<D>::k / 32; ++w) most = max(most, maxima[turn][w]);
        } else {
#pragma unroll
            for (int w = 0; w < Threads<D>::v / 32; ++w) most = max(most, maxima[turn][Threads<D>::k / 32 + w]);
        }
        const int e_new = exponent_for(__uint_as_float(most)), e = max(e_old, e_new);
        const bool grows = blk.lo > 0 && e_new > e_old;
        bool writes[2] = {is_new[0], is_new[1]};
        if (grows) {   // the rows that were there before, from their codes
            const float scale = power_of_two(e_old);
            if (p.is_k) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (p.r[i] < blk.lo) {
                        const uint2 w = *reinterpret_cast<const uint2*>(rec + p.at[i]);
                        float y[4];
                        decode4(w.x, scale, y);
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[i][j] = y[j];
                        decode4(w.y, scale, y);
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[i][4 + j] = y[j];
                        writes[i] = true;
                    }
            } else if (p.r[0] < blk.lo) {
                const uint4 w4 = *reinterpret_cast<const uint4*>(rec + p.at[0]);
                const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float y[4];
                    decode4(w[q], scale, y);
                    x[0][2 * q] = y[0];
                    x[0][2 * q + 1] = y[2];
                    if (p.r[1] < blk.lo) {
                        x[1][2 * q] = y[1];
                        x[1][2 * q + 1] = y[3];
                    }
                }
                writes[0] = true;
                writes[1] = writes[1] || p.r[1] < blk.lo;
            }
        }
        const float inv = power_of_two(-e);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] *= inv;
        if (p.is_k) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (writes[i])
                    *reinterpret_cast<uint2*>(rec + p.at[i]) = make_uint2(code_pair(x[i][0], x[i][1]) | code_pair(x[i][2], x[i][3]) << 16,
                                                                          code_pair(x[i][4], x[i][5]) | code_pair(x[i][6], x[i][7]) << 16);
        } else if (writes[0] && writes[1]) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = code_pair(x[0][2 * q], x[1][2 * q]) | code_pair(x[0][2 * q + 1], x[1][2 * q + 1]) << 16;
            *reinterpret_cast<uint4*>(rec + p.at[0]) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (writes[i]) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) rec[p.at[i] + 2 * j] = (uint8_t)code_pair(x[i][j], 0.0f);
                }
        }
        if ((tid == 0 || tid == Threads<D>::k) && (blk.lo == 0 || grows)) *exponent = e;
    }
}

// 8 values to their row, as TO.
template <typename TO>
__device__ __forceinline__ void put8(TO* to, const float (&x)[8]) {
    constexpr int N = 16 / sizeof(TO);
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) reinterpret_cast<uint4*>(to)[i] = pack<TO>(x + N * i);
}

template <typename TO, int D>
__global__ void __launch_bounds__(Threads<D>::all, kGatherCtas) gather8_kernel(const __grid_constant__ RowArgs a) {
    let_next_start();
    wait_for_previous();
    using R = Record8<D>;
    Block blk;
    if (!find_block(a, blockIdx.x, &blk)) return;
    const bool good = blk.page >= 0;
    if (!good && threadIdx.x == 0 && blockIdx.y == 0) raise_status(a.status, TKV_ECAPACITY);
    const Pieces p = pieces_of_thread<D>();
    const bool wanted[2] = {p.r[0] >= blk.lo && p.r[0] < blk.hi, p.r[1] >= blk.lo && p.r[1] < blk.hi};
    if (!wanted[0] && !wanted[1]) return;
    const int64_t stride = p.is_k ? a.k_row : a.v_row, head = p.is_k ? a.k_head : a.v_head;
    TO* to = reinterpret_cast<TO*>(const_cast<void*>(p.is_k ? a.k : a.v)) + blockIdx.y * head + p.channel;
    const int64_t head_bytes = (int64_t)(a.c.page_size >> 4) * R::bytes;
    const uint8_t* rec = reinterpret_cast<const uint8_t*>(a.c.pages) + ((good ? blk.page : 0) * a.c.num_kv_heads + blockIdx.y) * head_bytes +
                         (((int)blk.first & (a.c.page_size - 1)) >> 4) * R::bytes;
    uint4 w = {}, next = {};
    int e = 0, next_e = 0;
    auto read = [&](int h) {   // K: 8 bytes of each row; V: 16 bytes of both
        if (!good || h >= a.c.num_kv_heads) return;
        if (p.is_k) {
            const uint2 u = wanted[0] ? *reinterpret_cast<const uint2*>(rec + p.at[0]) : make_uint2(0, 0);
            const uint2 v = wanted[1] ? *reinterpret_cast<const uint2*>(rec + p.at[1]) : make_uint2(0, 0);
            next = make_uint4(u.x, u.y, v.x, v.y);
        } else {
            next = *reinterpret_cast<const uint4*>(rec + p.at[0]);
        }
        next_e = reinterpret_cast<const int*>(rec + R::exponents)[!p.is_k];
        rec += a.lanes * head_bytes;
    };
    read(blockIdx.y);
#pragma unroll 1
    for (int h = blockIdx.y; h < a.c.num_kv_heads; h += a.lanes, to += a.lanes * head) {
        w = next;
        e = next_e;
        read(h + a.lanes);
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
        const float scale = good ? power_of_two(block_exponent(e)) : __int_as_float(0x7FC00000);
        float x[2][8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float y[4];
            decode4(v[q], scale, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (p.is_k) x[q >> 1][4 * (q & 1) + j] = y[j];
                else x[j & 1][2 * q + (j >> 1)] = y[j];
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (wanted[i]) put8(to + (blk.row0 + p.r[i]) * stride, x[i]);
    }
}

// Slots of a step: the place behind the last sequence's, cu[batch] <= rows.
int64_t slots_of(const RowArgs& a) { return (a.rows >> 4) + 2 * (int64_t)a.c.batch; }

cudaError_t spread(RowArgs& a, int ctas) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) a.lanes = spread_heads(slots_of(a), a.c.num_kv_heads, (int64_t)sms * ctas, 8);
    return e;
}

template <typename T, int D>
cudaError_t append_turn(const RowArgs& a, cudaStream_t st) {
    const int turn = !a.table ? kNone : a.interleaved ? (a.pairs % 4 == 0 ? kAdjacent : kAny) : a.pairs % 8 == 0 ? kHalves : kAny;
    return launch_behind(turn == kNone       ? append8_kernel<T, D, kNone>
                         : turn == kHalves   ? append8_kernel<T, D, kHalves>
                         : turn == kAdjacent ? append8_kernel<T, D, kAdjacent>
                                             : append8_kernel<T, D, kAny>,
                         dim3((unsigned)slots_of(a), a.lanes), Threads<D>::all, 0, st, a);
}

template <typename TO>
cudaError_t gather_type(const RowArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)slots_of(a), a.lanes);
    return a.c.head_dim == 128 ? launch_behind(gather8_kernel<TO, 128>, grid, Threads<128>::all, 0, st, a)
                               : launch_behind(gather8_kernel<TO, 64>, grid, Threads<64>::all, 0, st, a);
}

}  // namespace

namespace tkv {

cudaError_t append_e4m3(RowArgs& a, int dtype, cudaStream_t st) {
    const cudaError_t e = spread(a, kAppendCtas);
    if (e != cudaSuccess) return e;
    if (dtype == TKV_BF16) return a.c.head_dim == 128 ? append_turn<__nv_bfloat16, 128>(a, st) : append_turn<__nv_bfloat16, 64>(a, st);
    return a.c.head_dim == 128 ? append_turn<__half, 128>(a, st) : append_turn<__half, 64>(a, st);
}

cudaError_t gather_e4m3(RowArgs& a, int dtype, cudaStream_t st) {
    const cudaError_t e = spread(a, kGatherCtas);
    if (e != cudaSuccess) return e;
    return dtype == TKV_BF16 ? gather_type<__nv_bfloat16>(a, st) : dtype == TKV_FP16 ? gather_type<__half>(a, st) : gather_type<float>(a, st);
}

}  // namespace tkv
