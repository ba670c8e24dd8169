// Rows into and out of 8-bit pages (the records are described in paged.cuh): the E4M3 side of tkv_paged_append and tkv_paged_gather.
//
// A block of 16 positions of a KV head has one exponent for K and one for V.  A step brings it new rows at offsets [f, g):
//   a = max |x| over what is finite of them (k after its rotation),  e_new = least e with a <= 448 2^e, within -32 .. 31
//   e = e_new if f = 0, else max(e, e_new);  code = e4m3(x 2^-e), to nearest even, saturating; an infinity or a NaN is NaN
// and where e grows the rows [0, f) are written anew: value 2^-e, rounded once more (exact but for what becomes subnormal).
// So a block and not a row is what one CTA owns: half of its warps take K, the others V, and walk over KV heads; a thread has 16 values
// of each head, and half of the CTA meets once a head, for the maxima.  Of K they are a row's 8 channels and the 8 that hold their
// partners, whose cosines and sines are found once for all heads; of V 8 channels of two rows, which are written together.
//
// A CTA's block.  A sequence's n rows touch at most (n + 14) / 16 + 1 blocks, so the slots from (cu[b] >> 4) + 2 b up to
// (cu[b + 1] >> 4) + 2 (b + 1) hold them all wherever they begin: slots are CTAs, the sequence of a slot is found by a search over cu,
// 32 lanes at a time (one trip to memory up to 32 sequences, two up to 1,024), and at most 2 slots a sequence stay idle.  What a CTA
// waits for at its begin is memory: the search, then the page together with the first head's values and the positions, then the
// angles; in a prompt each of its two rounds of CTAs spent 4.7 of 14 us there while the page was asked for first.
//
// What bounds both is memory: 2 bytes a value on one side, 1 on the other.
#include "paged_rows.cuh"

using namespace tkv;

namespace {

// D threads for K and D for V, 16 values each.  CTAs on an SM at once, by their registers: the gather of 18,432 rows of 8 heads of 128
// takes 18.3 us with eight and 21.2 with six; 402 rows of 5 heads of 64 2.7 us with twelve and 3.2 with sixteen.
template <int D>
constexpr int append_ctas() { return 512 / D; }
template <int D>
constexpr int gather_ctas() { return D == 128 ? 8 : 12; }

// A block of a step: its new rows are those at offsets [lo, hi), row0 + offset in the step's tensors.
struct Block {
    int64_t first, row0;   // position of offset 0
    int lo, hi, page;      // page: as the table has it, or -1; on its way when find_block returns
};

// The block of a slot; false: the slot has none.  Every lane of the warp calls it.
__device__ __forceinline__ bool find_block(const RowArgs& a, int64_t slot, Block* k) {
    const int lane = threadIdx.x & 31;
    int begin = 0, len = a.c.batch;   // sequences [begin, begin + len) are not known yet; those before begin at or before the slot
    int64_t c0 = 0, c1 = 0, length = 0;
    bool known = false;
    while (len > 0) {
        const int step = (len + 31) / 32, at = lane * step;
        const int mine = at < len ? a.cu[begin + at] : 0;
        int next = 0, its = 0;
        if (step == 1 && at < len) {   // the last round: what is wanted of the sequence comes along
            next = a.cu[begin + at + 1];
            its = a.c.lengths[begin + at];
        }
        const bool before = at < len && (int64_t)(mine >> 4) + 2 * (int64_t)(begin + at) <= slot;
        const int n = __popc(__ballot_sync(0xffffffffu, before));
        if (n == 0) break;
        if (step == 1) {
            c0 = __shfl_sync(0xffffffffu, mine, n - 1);
            c1 = __shfl_sync(0xffffffffu, next, n - 1);
            length = __shfl_sync(0xffffffffu, its, n - 1);
            known = true;
        }
        const int behind = (n - 1) * step + 1;
        begin += behind;
        len = min(step - 1, len - behind);
    }
    const int b = begin - 1;
    if (b < 0) return false;
    if (!known) {
        c0 = a.cu[b];
        c1 = a.cu[b + 1];
        length = a.c.lengths[b];
    }
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
    const int64_t column = k->first >> a.page_shift;
    k->page = k->first >= 0 && column < a.c.max_pages ? a.c.page_table[(int64_t)b * a.c.max_pages + column] : -1;
    return true;
}

__device__ __forceinline__ bool has_place(const RowArgs& a, const Block& k) { return k.page >= 0 && k.page < a.c.num_pages; }

// Where the block's record of the CTA's first head lies (of page 0, if it has no place).
template <int D>
__device__ __forceinline__ int64_t record_at(const RowArgs& a, const Block& k, int64_t head_bytes) {
    return ((has_place(a, k) ? (int64_t)k.page : 0) * a.c.num_kv_heads + blockIdx.y) * head_bytes + (((int)k.first & (a.c.page_size - 1)) >> 4) * Record8<D>::bytes;
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
    const float2 c = parts(mul2(f2(a.x, a.y), f2(scale, scale))), d = parts(mul2(f2(b.x, b.y), f2(scale, scale)));
    x[0] = c.x;
    x[1] = c.y;
    x[2] = d.x;
    x[3] = d.y;
}

// The largest of three magnitudes; NaN counts for nothing.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float y;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// The largest magnitude of a thread's 16 values.
__device__ __forceinline__ float largest(const float (&x)[2][8]) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 8; j += 2) top = max_abs(x[i][j], x[i][j + 1], top);
    return top;
}

// Infinities become NaN, which their codes are then.
__device__ __forceinline__ void no_infinities(const float (&x)[2][8], float (&z)[2][8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) z[i][j] = fabsf(x[i][j]) == INFINITY ? __int_as_float(0x7FC00000) : x[i][j];
}

// The largest over the D threads of K (half 0) or V (half 1), which are whole warps and meet at a barrier of their own.
template <int D>
__device__ __forceinline__ float largest_of_half(float top, int half, uint32_t (&maxima)[D / 32]) {
    const uint32_t warp_max = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
    if ((threadIdx.x & 31) == 0) maxima[(threadIdx.x >> 5) & (D / 32 - 1)] = warp_max;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + half), "n"(D) : "memory");
    uint32_t most = 0;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) most = max(most, maxima[w]);
    return __uint_as_float(most);
}

__device__ __forceinline__ void scaled(const float (&x)[8], float f, float (&y)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 z = parts(mul2(f2(x[j], x[j + 1]), f2(f, f)));
        y[j] = z.x;
        y[j + 1] = z.y;
    }
}

// Chunks of 8 channels.  Unit u of a row: where k is turned by halves the first pairs / 8 units are chunk u and its partner, otherwise
// two neighbours.
struct Chunks {
    int c[2];
    bool turned;
};
template <int TURN>
__device__ __forceinline__ Chunks chunks_of(int u, int pairs) {
    const int pc = TURN == kHalves ? pairs >> 3 : 0;
    if (u < pc) return Chunks{{u, u + pc}, true};
    const int c = 2 * pc + 2 * (u - pc);
    return Chunks{{c, c + 1}, TURN != kNone && TURN != kHalves};
}
__device__ __forceinline__ int k_place(int row, int chunk) { return (chunk >> 3) * 1024 + row * 64 + (chunk & 7) * 8; }

__device__ __forceinline__ void put_k(uint8_t* rec, int r, const Chunks& ch, const float (&x)[2][8], int e) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float y[8];
        scaled(x[i], power_of_two(-e), y);
        *reinterpret_cast<uint2*>(rec + k_place(r, ch.c[i])) =
            make_uint2(code_pair(y[0], y[1]) | code_pair(y[2], y[3]) << 16, code_pair(y[4], y[5]) | code_pair(y[6], y[7]) << 16);
    }
}

__device__ __forceinline__ void put_v(uint8_t* to, const float (&x)[2][8], int e, bool first, bool second) {
    float y[8], z[8];
    scaled(x[0], power_of_two(-e), y);
    scaled(x[1], power_of_two(-e), z);
    if (first && second) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = code_pair(y[2 * q], z[2 * q]) | code_pair(y[2 * q + 1], z[2 * q + 1]) << 16;
        *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if (first || second) {
#pragma unroll
        for (int j = 0; j < 8; ++j) to[(second ? 1 : 0) + 2 * j] = (uint8_t)code_pair(second ? z[j] : y[j], 0.0f);
    }
}

// K of a block: a thread has 16 channels of one row.
template <typename T, int D, int TURN>
__device__ __forceinline__ void append_k(const RowArgs& a, const Block& blk, uint32_t (&maxima)[3][D / 32]) {
    const int t = threadIdx.x, r = t / (D / 16);
    const Chunks ch = chunks_of<TURN>(t & (D / 16 - 1), a.pairs);
    const bool is_new = r >= blk.lo && r < blk.hi;
    const int64_t row = blk.row0 + r;
    const T* from = reinterpret_cast<const T*>(a.k) + row * a.k_row + blockIdx.y * a.k_head;
    uint4 raw[2] = {};
    auto read = [&](int h) {   // the next head's values, while the last one's are worked on
        if (is_new && h < a.c.num_kv_heads) {
            raw[0] = *reinterpret_cast<const uint4*>(from + 8 * ch.c[0]);
            raw[1] = *reinterpret_cast<const uint4*>(from + 8 * ch.c[1]);
        }
        from += a.lanes * a.k_head;
    };
    read(blockIdx.y);
    constexpr int NCS = TURN == kHalves || TURN == kAdjacent ? 8 : 1;
    float2 cs[NCS];
    bool turned[2] = {ch.turned, ch.turned};   // adjacent pairs: a chunk holds its own four
    if (TURN == kAdjacent || TURN == kAny) {
#pragma unroll
        for (int i = 0; i < 2; ++i) turned[i] = 8 * ch.c[i] < 2 * a.pairs;
    }
    if (NCS == 8 && is_new && (turned[0] || turned[1])) {
        int pos[4] = {(int)(blk.first + r), 0, 0, 0};
        if (a.positions) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (x < a.num_axes) pos[x] = a.positions[x * a.axis_stride + row];
        }
        if (TURN == kHalves) {
            load_angles<NCS>(a, pos, 8 * ch.c[0], cs);
        } else {
            float2 four[4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (turned[i]) {
                    load_angles<4>(a, pos, 4 * ch.c[i], four);
#pragma unroll
                    for (int j = 0; j < 4; ++j) cs[(4 * i + j) % NCS] = four[j];
                }
        }
    }
    if (!has_place(a, blk)) {
        if (t == 0 && blockIdx.y == 0) raise_status(a.status, TKV_ECAPACITY);
        return;
    }
    const int64_t head_bytes = (int64_t)(a.c.page_size >> 4) * Record8<D>::bytes, next_rec = a.lanes * head_bytes;
    uint8_t* rec = reinterpret_cast<uint8_t*>(a.c.pages) + record_at<D>(a, blk, head_bytes);
    int side = 0;
#pragma unroll 1
    for (int h = blockIdx.y; h < a.c.num_kv_heads; h += a.lanes, rec += next_rec, side ^= 1) {
        int* exponent = reinterpret_cast<int*>(rec + Record8<D>::exponents);
        int e_old = kLowestExponent;
        if (blk.lo > 0) e_old = block_exponent(*exponent);
        float x[2][8];
        unpack<T>(raw[0], x[0]);
        unpack<T>(raw[1], x[1]);
        read(h + a.lanes);
        if (TURN == kHalves && ch.turned && is_new) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 z = rotate_pair(x[0][j], x[1][j], cs[j % NCS]);
                x[0][j] = z.x;
                x[1][j] = z.y;
            }
        } else if (TURN == kAdjacent && is_new) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (turned[i]) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 z = rotate_pair(x[i][2 * j], x[i][2 * j + 1], cs[(4 * i + j) % NCS]);
                        x[i][2 * j] = z.x;
                        x[i][2 * j + 1] = z.y;
                    }
                }
        } else if (TURN == kAny && is_new) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (turned[i]) turn_any(a, reinterpret_cast<const T*>(a.k) + row * a.k_row + h * a.k_head, row, (int)(blk.first + r), ch.c[i], x[i]);
        }
        // What is rare (an infinity in the block, rows whose scale grows) works on values of its own, so that the common path has no
        // register that two paths write: 24.2 us instead of 26.4 for 18,432 rows of 8 heads of 128.
        float most = largest_of_half<D>(largest(x), 0, maxima[side]);   // rows that are not new are zeros here
        auto finish = [&](const float (&x)[2][8]) {
            const int e_new = exponent_for(most), e = max(e_old, e_new);
            const bool grows = blk.lo > 0 && e_new > e_old;
            if (is_new) {
                put_k(rec, r, ch, x, e);
            } else if (grows && r < blk.lo) {   // the rows that were there before, from their codes
                float z[2][8];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint2 w = *reinterpret_cast<const uint2*>(rec + k_place(r, ch.c[i]));
                    float y[4];
                    decode4(w.x, power_of_two(e_old), y);
#pragma unroll
                    for (int j = 0; j < 4; ++j) z[i][j] = y[j];
                    decode4(w.y, power_of_two(e_old), y);
#pragma unroll
                    for (int j = 0; j < 4; ++j) z[i][4 + j] = y[j];
                }
                put_k(rec, r, ch, z, e);
            }
            if (t == 0 && (blk.lo == 0 || grows)) *exponent = e;   // everyone has read the old one before the barrier
        };
        if (most < INFINITY) {
            finish(x);
        } else {
            float z[2][8];
            no_infinities(x, z);
            most = largest_of_half<D>(largest(z), 0, maxima[2]);
            finish(z);
        }
    }
}

// V of a block: a thread has 8 channels of two rows, every other byte of 16 each.
template <typename T, int D>
__device__ __forceinline__ void append_v(const RowArgs& a, const Block& blk, uint32_t (&maxima)[3][D / 32]) {
    const int t = threadIdx.x - D, chunk = (t >> 2) & (D / 8 - 1), r = t / (D / 2) * 8 + (t & 3) * 2;
    const bool is_new[2] = {r >= blk.lo && r < blk.hi, r + 1 >= blk.lo && r + 1 < blk.hi};
    const T* from = reinterpret_cast<const T*>(a.v) + (blk.row0 + r) * a.v_row + blockIdx.y * a.v_head + 8 * chunk;
    uint4 raw[2] = {};
    auto read = [&](int h) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (is_new[i] && h < a.c.num_kv_heads) raw[i] = *reinterpret_cast<const uint4*>(from + i * a.v_row);
        from += a.lanes * a.v_head;
    };
    read(blockIdx.y);
    if (!has_place(a, blk)) return;
    const int64_t head_bytes = (int64_t)(a.c.page_size >> 4) * Record8<D>::bytes, next_rec = a.lanes * head_bytes;
    const int at = Record8<D>::v_codes + t / (D / 2) * (8 * D) + chunk * 64 + (t & 3) * 16, to_exponent = Record8<D>::exponents + 4 - at;
    uint8_t* rec = reinterpret_cast<uint8_t*>(a.c.pages) + record_at<D>(a, blk, head_bytes) + at;
    int side = 0;
#pragma unroll 1
    for (int h = blockIdx.y; h < a.c.num_kv_heads; h += a.lanes, rec += next_rec, side ^= 1) {
        int* exponent = reinterpret_cast<int*>(rec + to_exponent);
        int e_old = kLowestExponent;
        if (blk.lo > 0) e_old = block_exponent(*exponent);
        float x[2][8];
        unpack<T>(raw[0], x[0]);
        unpack<T>(raw[1], x[1]);
        read(h + a.lanes);
        float most = largest_of_half<D>(largest(x), 1, maxima[side]);
        auto finish = [&](const float (&x)[2][8]) {
            const int e_new = exponent_for(most), e = max(e_old, e_new);
            const bool grows = blk.lo > 0 && e_new > e_old;
            if (grows && r < blk.lo) {
                float z[2][8];
                const uint4 w4 = *reinterpret_cast<const uint4*>(rec);
                const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
                const bool both = r + 1 < blk.lo;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float y[4];
                    decode4(w[q], power_of_two(e_old), y);
                    z[0][2 * q] = y[0];
                    z[0][2 * q + 1] = y[2];
                    z[1][2 * q] = both ? y[1] : x[1][2 * q];
                    z[1][2 * q + 1] = both ? y[3] : x[1][2 * q + 1];
                }
                put_v(rec, z, e, true, both || is_new[1]);
            } else {
                put_v(rec, x, e, is_new[0], is_new[1]);
            }
            if (t == 0 && (blk.lo == 0 || grows)) *exponent = e;
        };
        if (most < INFINITY) {
            finish(x);
        } else {
            float z[2][8];
            no_infinities(x, z);
            most = largest_of_half<D>(largest(z), 1, maxima[2]);
            finish(z);
        }
    }
}

// blockIdx.y: the first head.
template <typename T, int D, int TURN>
__global__ void __launch_bounds__(2 * D, append_ctas<D>()) append8_kernel(const __grid_constant__ RowArgs a) {
    let_next_start();
    wait_for_previous();
    __shared__ uint32_t maxima[2][3][D / 32];   // of K and V; one head's and the next's in turn, so one barrier a head is enough
    Block blk;
    if (!find_block(a, blockIdx.x, &blk)) return;
    if (threadIdx.x < D) append_k<T, D, TURN>(a, blk, maxima[0]);
    else append_v<T, D>(a, blk, maxima[1]);
}

// 8 values to their row, as TO.
template <typename TO>
__device__ __forceinline__ void put8(TO* to, const float (&x)[8]) {
    constexpr int N = 16 / sizeof(TO);
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) reinterpret_cast<uint4*>(to)[i] = pack<TO>(x + N * i);
}

template <typename TO, int D>
__global__ void __launch_bounds__(2 * D, gather_ctas<D>()) gather8_kernel(const __grid_constant__ RowArgs a) {
    let_next_start();
    wait_for_previous();
    using R = Record8<D>;
    Block blk;
    if (!find_block(a, blockIdx.x, &blk)) return;
    const bool good = has_place(a, blk), is_k = threadIdx.x < D;
    if (!good && threadIdx.x == 0 && blockIdx.y == 0) raise_status(a.status, TKV_ECAPACITY);
    // 8 channels of two rows a thread, 8 apart of K and neighbours of V: with 16 channels of one each store writes half of its sectors
    // (22.7 us instead of 18.3 for 18,432 rows of 8 heads of 128 as bf16)
    const int t = threadIdx.x & (D - 1), chunk = is_k ? t & (D / 8 - 1) : (t >> 2) & (D / 8 - 1);
    const int r = is_k ? t / (D / 8) : t / (D / 2) * 8 + (t & 3) * 2, apart = is_k ? 8 : 1;
    const bool wanted[2] = {r >= blk.lo && r < blk.hi, r + apart >= blk.lo && r + apart < blk.hi};
    if (!wanted[0] && !wanted[1]) return;
    const int64_t stride = is_k ? a.k_row : a.v_row, head = is_k ? a.k_head : a.v_head, second = apart * stride;
    TO* to = reinterpret_cast<TO*>(const_cast<void*>(is_k ? a.k : a.v)) + (blk.row0 + r) * stride + blockIdx.y * head + 8 * chunk;
    const int64_t head_bytes = (int64_t)(a.c.page_size >> 4) * R::bytes;
    const int at = is_k ? k_place(r, chunk) : R::v_codes + t / (D / 2) * (8 * D) + chunk * 64 + (t & 3) * 16;
    const int to_exponent = R::exponents + (is_k ? 0 : 4) - at;
    const uint8_t* from = reinterpret_cast<const uint8_t*>(a.c.pages) + record_at<D>(a, blk, head_bytes) + at;
    // V's bytes in turn belong to the two rows: put beside those of their row
    const uint32_t low = is_k ? 0x3210u : 0x6420u, high = is_k ? 0x7654u : 0x7531u;
    uint4 next = {};
    int next_e = 0;
    auto read = [&](int h) {
        if (!good || h >= a.c.num_kv_heads) return;
        if (is_k) {
            const uint2 u = *reinterpret_cast<const uint2*>(from), v = *reinterpret_cast<const uint2*>(from + 8 * 64);
            next = make_uint4(u.x, u.y, v.x, v.y);
        } else {
            next = *reinterpret_cast<const uint4*>(from);
        }
        next_e = *reinterpret_cast<const int*>(from + to_exponent);
        from += a.lanes * head_bytes;
    };
    read(blockIdx.y);
#pragma unroll 1
    for (int h = blockIdx.y; h < a.c.num_kv_heads; h += a.lanes, to += a.lanes * head) {
        const float scale = good ? power_of_two(block_exponent(next_e)) : __int_as_float(0x7FC00000);
        // words of the first piece (row), then of the second
        const uint32_t first[2] = {__byte_perm(next.x, next.y, low), __byte_perm(next.x, next.y, high)};
        const uint32_t last[2] = {__byte_perm(next.z, next.w, low), __byte_perm(next.z, next.w, high)};
        const uint32_t w[2][2] = {{first[0], is_k ? first[1] : last[0]}, {is_k ? last[0] : first[1], last[1]}};
        read(h + a.lanes);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float x[8], y[4];
            decode4(w[i][0], scale, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = y[j];
            decode4(w[i][1], scale, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[4 + j] = y[j];
            if (wanted[i]) put8(to + i * second, x);
        }
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
                         dim3((unsigned)slots_of(a), a.lanes), 2 * D, 0, st, a);
}

template <typename TO>
cudaError_t gather_type(const RowArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)slots_of(a), a.lanes);
    return a.c.head_dim == 128 ? launch_behind(gather8_kernel<TO, 128>, grid, 256, 0, st, a)
                               : launch_behind(gather8_kernel<TO, 64>, grid, 128, 0, st, a);
}

}  // namespace

namespace tkv {

cudaError_t append_e4m3(RowArgs& a, int dtype, cudaStream_t st) {
    const cudaError_t e = spread(a, a.c.head_dim == 128 ? append_ctas<128>() : append_ctas<64>());
    if (e != cudaSuccess) return e;
    if (dtype == TKV_BF16) return a.c.head_dim == 128 ? append_turn<__nv_bfloat16, 128>(a, st) : append_turn<__nv_bfloat16, 64>(a, st);
    return a.c.head_dim == 128 ? append_turn<__half, 128>(a, st) : append_turn<__half, 64>(a, st);
}

cudaError_t gather_e4m3(RowArgs& a, int dtype, cudaStream_t st) {
    const cudaError_t e = spread(a, a.c.head_dim == 128 ? gather_ctas<128>() : gather_ctas<64>());
    if (e != cudaSuccess) return e;
    return dtype == TKV_BF16 ? gather_type<__nv_bfloat16>(a, st) : dtype == TKV_FP16 ? gather_type<__half>(a, st) : gather_type<float>(a, st);
}

}  // namespace tkv
