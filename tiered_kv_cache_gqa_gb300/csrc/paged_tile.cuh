// One tile of positions of the attention over a paged cache: S^T = K q^T, the softmax's running sums, O^T += V^T P^T.
//
// For a KV head, the rows of a step (query t of a sequence, query head g of its group: row t G + g) are the columns of
// two small matrix products a tile of positions:
//   S^T = K q^T       (positions x rows; K from the cache, q in registers)
//   O^T += V^T P^T    (channels x rows; P = 2^(z - m), z = S scale log2 e)
// Every warp keeps, for each row, a reference m, the sum l of its p and O, in fp32.  m is not the running maximum but a
// number that the maximum has not passed by more than kTop (in powers of two): p stays within fp16's range, the
// common tile needs no exchange between lanes, and O is rescaled only where that room is used up.
// Transposed like this, a group of 8 heads fills the 8 columns of mma.m16n8k16 with nothing wasted; the operation is
// bound by memory there (at 8 heads and 4 bits, 28 operations a byte), so mma.sync is enough for it.  With more rows it is not:
// the tiles of 16 or 32 rows are held up by expanding the codes again for each and by O in registers.
//
// 4 bits to fp16, exactly.  (w & 0x000F000F) | 0x64006400 is the pair (1024 + n, 1024 + n') of two codes n = q + 8, and
// (w & 0x00F000F0) | 0x54005400 the pair (64 + n, 64 + n'); one fused multiply-add with s = scale / 16 gives
// (1024 + n) s - 1032 s = q s (and (64 + n) s - 72 s).  Every operand and result is exact in fp16: scale has 4 bits,
// 129 * 15 < 2^11, and 1032 * 448 / 16 is below its largest number.  So K and V enter the products as stored; what is
// rounded is p (to fp16, 2^-11; for bf16 pages to two bf16 parts, 2^-16) and, for rows of q in bf16, what lies 2^-29 below
// a row's largest channel (q is scaled by a power of two into fp16's range).
// 8 bits: E4M3 codes are fp16 numbers by one conversion a pair.  A block's exponents stay out of the products: z = S scale log2 e 2^e_k
// + e_v and p = 2^(z - m), which is the weight times V's scale, so O^T += V^T P^T adds up blocks of different scales; l += p 2^-e_v.
// With e_v in -32 .. 31 what p loses below 2^-126 is below 2^-60 of the largest weight, and what it loses in fp16 is, times its
// code, below 2^-29 of the largest weight times V's scale.
// The channels that a lane holds of a position are those of its own bytes: K's products sum over all channels, so q is
// laid out to match; for V the lanes' channels are rows of O^T.
#pragma once

#include "paged.cuh"
#include "tkv_internal.cuh"

namespace tkv {

constexpr float kTop = 15.0f;                      // p = 2^(z - m) <= 2^15; in fp16 the smallest is 2^-24
constexpr float kLift = 5.0f;                      // a new reference lies this far below the maximum: 10 are left to grow
constexpr float kLowest = -3.402823466e38f;        // a reference before anything is seen: 2^(-inf - it) = 0, no NaN

enum PageKind { kInt4, kBf16, kFp16, kE4m3 };
// pages of records, copied whole; their lanes hold neighbouring channels of O
constexpr bool in_records(int kind) { return kind == kInt4 || kind == kE4m3; }

template <int D, int KIND>
struct TileOf {
    static constexpr int groups = KIND == kInt4 || (KIND == kE4m3 && D == 64) ? 2 : 1;     // of 16 positions
    static constexpr int positions = 16 * groups;
    static constexpr int row = 2 * D + 16;                   // 16 bits: bytes of a row, 16 more than it has, so that the
                                                             // rows of a fragment lie in different banks
    static constexpr int record = KIND == kInt4 ? Record<D>::bytes : KIND == kE4m3 ? Record8<D>::bytes : 2 * 16 * row;
    static constexpr int bytes = groups * record;
};

// ------------------------------------------------------------------ PTX
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
// 8 x 8 16-bit matrix, a row's pair a lane -> its transpose
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
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
__device__ __forceinline__ uint32_t bf162_bits(__nv_bfloat162 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 both(float x) { return __half2half2(__float2half(x)); }
__device__ __forceinline__ __half2 e4m3_pair(uint16_t w) { return __half2(__nv_cvt_fp8x2_to_halfraw2(w, __NV_E4M3)); }

// Four codes a half of the word -> q s of codes 0, 1 of each half (first) or 2, 3 (second): s, -1032 s, -72 s.
__device__ __forceinline__ uint32_t expand_low(uint32_t x, __half2 s, __half2 n1032) {
    return half2_bits(__hfma2(bits_half2(and_or(x, 0x000F000Fu, 0x64006400u)), s, n1032));
}
__device__ __forceinline__ uint32_t expand_high(uint32_t x, __half2 s, __half2 n72) {
    return half2_bits(__hfma2(bits_half2(and_or(x, 0x00F000F0u, 0x54005400u)), s, n72));
}

// The query of a row of its sequence: row / group, by a multiplication that is at most one too small.
__device__ __forceinline__ int query_of(int row, int group, uint32_t mul) {
    const int t = (int)__umulhi((uint32_t)row, mul);
    return row - t * group >= group ? t + 1 : t;
}

// ------------------------------------------------------------------ what a warp holds
// The rows of a piece: which positions they see.
struct Rows {
    int h, first_row, n;        // KV head; the sequence's first row of the step, and its queries
    int row0, seq_rows;         // this tile of rows starts here; rows of the sequence, n * group
    int len, last0;             // positions [0, len) exist; query t sees those <= last0 + t
    int all_from, all_until;    // positions in between are seen by every row,
    int any_from, any_until;    // those outside [any_from, any_until) by none
};

template <int D, int NT>
struct Sums {
    float o[NT][D / 16][4], m[NT][2], l[NT][2];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = kLowest;
            l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.0f;
        }
    }
};

// Fragments of q^T: column r of row tile nt.  4 bits: channels in the order of the codes' pairs.
// Where they would take 64 registers the lane keeps them in shared memory, every 32nd uint2 of its own.
template <int D, int NT>
struct Query {
    static constexpr bool kShared = D * NT > 256;
    static constexpr int words = kShared ? NT * (D / 16) * 32 : 1;   // uint2s of a warp
    uint32_t f[kShared ? 1 : NT][kShared ? 1 : D / 16][2];
    uint2* s;
    float z0[NT], z1[NT];      // S -> z, columns 2 cq and 2 cq + 1
    __device__ __forceinline__ uint2 get(int nt, int i) const {
        if constexpr (kShared) return s[(nt * (D / 16) + i) * 32];
        else return make_uint2(f[nt][i][0], f[nt][i][1]);
    }
    __device__ __forceinline__ void set(int nt, int i, uint32_t a, uint32_t b) {
        if constexpr (kShared) {
            s[(nt * (D / 16) + i) * 32] = make_uint2(a, b);
        } else {
            f[nt][i][0] = a;
            f[nt][i][1] = b;
        }
    }
};

// The position, within a group of 16, that row i of a fragment stands for.  4 bits: 0 1 3 2 4 5 7 6 8 .., so that the
// lanes of a quarter warp (K) and of half a warp (V) read from different banks.
template <int KIND>
__device__ __forceinline__ int slot_position(int i) { return KIND == kInt4 ? i ^ ((i >> 1) & 1) : i; }

// The lane's four V positions of a group (columns 2 cq, 2 cq + 1 and + 8): bit i set if position i lies in [from, to).
template <int KIND>
__device__ __forceinline__ uint32_t v_bits(int cq, int base, int from, int to) {
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int p = base + slot_position<KIND>(2 * cq + (i & 1)) + (i >> 1) * 8;
        bits |= p >= from && p < to ? 1u << i : 0u;
    }
    return bits;
}

// ------------------------------------------------------------------ K
// z += K q^T of a group: each lane expands its own bytes of rows r and r + 8.
template <int D, int NT>
__device__ __forceinline__ void scores_int4(const uint8_t* rec, int r, int cq, const Query<D, NT>& q, float (&z)[NT][4]) {
    using Rec = Record<D>;
    constexpr int W = D / 32;                 // words of codes, 8 channels each
    const int pr = slot_position<kInt4>(r);
    uint32_t wa[W], wb[W];
    __half2 sa[W / 2], sb[W / 2];             // scale / 16 of the lane's blocks, twice each
    if (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(rec + pr * 64 + cq * 16);
        const uint4 y = *reinterpret_cast<const uint4*>(rec + (pr + 8) * 64 + cq * 16);
        wa[0] = x.x; wa[1] = x.y; wa[W - 2] = x.z; wa[W - 1] = x.w;
        wb[0] = y.x; wb[1] = y.y; wb[W - 2] = y.z; wb[W - 1] = y.w;
        const __half2 fa = __hmul2(e4m3_pair(*reinterpret_cast<const uint16_t*>(rec + Rec::k_scales + pr * 8 + cq * 2)), both(0.0625f));
        const __half2 fb = __hmul2(e4m3_pair(*reinterpret_cast<const uint16_t*>(rec + Rec::k_scales + (pr + 8) * 8 + cq * 2)), both(0.0625f));
        sa[0] = __low2half2(fa); sa[W / 2 - 1] = __high2half2(fa);
        sb[0] = __low2half2(fb); sb[W / 2 - 1] = __high2half2(fb);
    } else {
        const uint2 x = *reinterpret_cast<const uint2*>(rec + pr * 32 + cq * 8);
        const uint2 y = *reinterpret_cast<const uint2*>(rec + (pr + 8) * 32 + cq * 8);
        wa[0] = x.x; wa[1] = x.y;
        wb[0] = y.x; wb[1] = y.y;
        const __half_raw ha = __nv_cvt_fp8_to_halfraw(rec[Rec::k_scales + pr * 4 + cq], __NV_E4M3);
        const __half_raw hb = __nv_cvt_fp8_to_halfraw(rec[Rec::k_scales + (pr + 8) * 4 + cq], __NV_E4M3);
        sa[0] = __hmul2(__half2half2(__half(ha)), both(0.0625f));
        sb[0] = __hmul2(__half2half2(__half(hb)), both(0.0625f));
    }
#pragma unroll
    for (int k = 0; k < W / 2; ++k) {
        const __half2 a1032 = __hmul2(sa[k], both(-1032.0f)), a72 = __hmul2(sa[k], both(-72.0f));
        const __half2 b1032 = __hmul2(sb[k], both(-1032.0f)), b72 = __hmul2(sb[k], both(-72.0f));
#pragma unroll
        for (int w = 2 * k; w < 2 * k + 2; ++w)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t x = wa[w] >> (8 * i), y = wb[w] >> (8 * i);
                const uint32_t f0 = expand_low(x, sa[k], a1032), f2 = expand_high(x, sa[k], a72);
                const uint32_t f1 = expand_low(y, sb[k], b1032), f3 = expand_high(y, sb[k], b72);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint2 b = q.get(nt, 2 * w + i);
                    mma_f16(z[nt], f0, f1, f2, f3, b.x, b.y);
                }
            }
    }
}

// The same from 8-bit codes: the lane's 16 channels of rows r and r + 8 in every 64.
template <int D, int NT>
__device__ __forceinline__ void scores_e4m3(const uint8_t* rec, int r, int cq, const Query<D, NT>& q, float (&z)[NT][4]) {
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
        const uint4 x = *reinterpret_cast<const uint4*>(rec + h * 1024 + r * 64 + cq * 16);
        const uint4 y = *reinterpret_cast<const uint4*>(rec + h * 1024 + (r + 8) * 64 + cq * 16);
        const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t f0 = half2_bits(e4m3_pair((uint16_t)wx[w])), f2 = half2_bits(e4m3_pair((uint16_t)(wx[w] >> 16)));
            const uint32_t f1 = half2_bits(e4m3_pair((uint16_t)wy[w])), f3 = half2_bits(e4m3_pair((uint16_t)(wy[w] >> 16)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint2 b = q.get(nt, 4 * h + w);
                mma_f16(z[nt], f0, f1, f2, f3, b.x, b.y);
            }
        }
    }
}

// The same from 16-bit rows.
template <int D, int NT, int KIND>
__device__ __forceinline__ void scores_16(uint32_t k_at, int lane, const Query<D, NT>& q, float (&z)[NT][4]) {
    const int row = (lane & 7) + (lane & 8);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        uint32_t f[4];
        ldmatrix4(f, k_at + row * TileOf<D, KIND>::row + (2 * i + (lane >> 4)) * 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const uint2 b = q.get(nt, i);
            if (KIND == kBf16) mma_bf16(z[nt], f[0], f[1], f[2], f[3], b.x, b.y);
            else mma_f16(z[nt], f[0], f[1], f[2], f[3], b.x, b.y);
        }
    }
}

// ------------------------------------------------------------------ V
template <int NT>
struct Weights {   // fragments of P^T; bf16: p = hi + lo
    uint32_t hi[NT][2], lo[NT][2];
};

__device__ __forceinline__ uint32_t pair_mask(uint32_t bits) { return (bits & 1 ? 0xFFFFu : 0u) | (bits & 2 ? 0xFFFF0000u : 0u); }

// The scales of the lane's two pairs of V positions, in the order of the slots (the bytes lie in that of the positions).
template <int D>
__device__ __forceinline__ uint32_t v_scale_pair(const uint8_t* rec, int r, int cq, int i) {
    const uint8_t* vs = rec + Record<D>::v_scales + (D == 128 ? r : r >> 1) * 16 + 2 * cq;
    return __byte_perm(half2_bits(e4m3_pair(*reinterpret_cast<const uint16_t*>(vs + 8 * i))), 0, cq & 1 ? 0x1032u : 0x3210u);
}

// acc += V^T P^T of a group.  MASKED: V is taken as 0 where `keep` has no bit.
template <int D, int NT, bool MASKED>
__device__ __forceinline__ void values_int4(const uint8_t* rec, int r, int cq, uint32_t keep, const Weights<NT>& p, float (&acc)[NT][D / 16][4]) {
    using Rec = Record<D>;
    __half2 s[2], n1032[2], n72[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t x = v_scale_pair<D>(rec, r, cq, i);
        if (MASKED) x &= pair_mask(keep >> (2 * i));
        s[i] = __hmul2(bits_half2(x), both(0.0625f));
        n1032[i] = __hmul2(s[i], both(-1032.0f));
        n72[i] = __hmul2(s[i], both(-72.0f));
    }
    constexpr int W = D / 64;                     // words of 8 channels a position
    uint32_t w[4][W];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint8_t* at = rec + Rec::v_codes + (slot_position<kInt4>(2 * cq + (i & 1)) + (i >> 1) * 8) * (D / 2) + r * (D / 16);
        if (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(at);
            w[i][0] = x.x;
            w[i][W - 1] = x.y;
        } else {
            w[i][0] = *reinterpret_cast<const uint32_t*>(at);
        }
    }
#pragma unroll
    for (int wi = 0; wi < W; ++wi)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            // the low (high) halves of the words of two positions side by side: four channels of the pair
            const uint32_t x0 = __byte_perm(w[0][wi], w[1][wi], half ? 0x7632 : 0x5410), y0 = __byte_perm(w[2][wi], w[3][wi], half ? 0x7632 : 0x5410);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t x = x0 >> (8 * i), y = y0 >> (8 * i);
                const uint32_t f0 = expand_low(x, s[0], n1032[0]), f1 = expand_high(x, s[0], n72[0]);
                const uint32_t f2 = expand_low(y, s[1], n1032[1]), f3 = expand_high(y, s[1], n72[1]);
                const int j = 4 * wi + 2 * half + i;   // rows r and r + 8 of the fragment: channels (D / 8) r + 2 j and + 1
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt][j], f0, f1, f2, f3, p.hi[nt][0], p.hi[nt][1]);
            }
        }
}

// Fragment j of V^T: rows r and r + 8 are channels 8 (r + 8 (j / 4)) + 2 (j % 4) and + 1; word j % 4 of the lane's pieces.
__device__ __forceinline__ void v_codes8(uint32_t (&f)[4], uint32_t x, uint32_t y, uint32_t m0, uint32_t m1) {
    f[0] = half2_bits(e4m3_pair((uint16_t)x)) & m0;
    f[1] = half2_bits(e4m3_pair((uint16_t)(x >> 16))) & m0;
    f[2] = half2_bits(e4m3_pair((uint16_t)y)) & m1;
    f[3] = half2_bits(e4m3_pair((uint16_t)(y >> 16))) & m1;
}

template <int D, int NT, bool MASKED>
__device__ __forceinline__ void values_e4m3(const uint8_t* rec, int r, int cq, uint32_t keep, const Weights<NT>& p, float (&acc)[NT][D / 16][4]) {
    const uint32_t m0 = MASKED ? pair_mask(keep) : ~0u, m1 = MASKED ? pair_mask(keep >> 2) : ~0u;
    const uint8_t* at = rec + Record8<D>::v_codes + r * 64 + cq * 16;
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
        const uint4 x = *reinterpret_cast<const uint4*>(at + h * 512), y = *reinterpret_cast<const uint4*>(at + 8 * D + h * 512);
        const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t f[4];
            v_codes8(f, wx[w], wy[w], m0, m1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt][4 * h + w], f[0], f[1], f[2], f[3], p.hi[nt][0], p.hi[nt][1]);
        }
    }
}

// Block j of V^T (channels 16 j .. 16 j + 15) from 16-bit rows.
template <int D>
__device__ __forceinline__ void v_block(uint32_t (&f)[4], uint32_t v_at, int lane, int j, uint32_t m0, uint32_t m1) {
    const int row = (lane & 7) + ((lane >> 4) << 3);
    ldmatrix4_trans(f, v_at + row * TileOf<D, kBf16>::row + (2 * j + ((lane >> 3) & 1)) * 16);
    f[0] &= m0; f[1] &= m0; f[2] &= m1; f[3] &= m1;
}

template <int D, int NT, int KIND, bool MASKED>
__device__ __forceinline__ void values_16(uint32_t v_at, int lane, uint32_t keep, const Weights<NT>& p, float (&acc)[NT][D / 16][4]) {
    const uint32_t m0 = MASKED ? pair_mask(keep) : ~0u, m1 = MASKED ? pair_mask(keep >> 2) : ~0u;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        uint32_t f[4];
        v_block<D>(f, v_at, lane, j, m0, m1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (KIND == kBf16) {
                mma_bf16(acc[nt][j], f[0], f[1], f[2], f[3], p.hi[nt][0], p.hi[nt][1]);
                mma_bf16(acc[nt][j], f[0], f[1], f[2], f[3], p.lo[nt][0], p.lo[nt][1]);
            } else {
                mma_f16(acc[nt][j], f[0], f[1], f[2], f[3], p.hi[nt][0], p.hi[nt][1]);
            }
        }
    }
}

template <int D, int NT, int KIND, bool MASKED>
__device__ __forceinline__ void values(const uint8_t* tile, uint32_t tile_s, int g, int lane, uint32_t keep, const Weights<NT>& p,
                                       float (&acc)[NT][D / 16][4]) {
    if (KIND == kInt4) values_int4<D, NT, MASKED>(tile + g * Record<D>::bytes, lane >> 2, lane & 3, keep, p, acc);
    else if (KIND == kE4m3) values_e4m3<D, NT, MASKED>(tile + g * Record8<D>::bytes, lane >> 2, lane & 3, keep, p, acc);
    else values_16<D, NT, KIND, MASKED>(tile_s + 16 * TileOf<D, KIND>::row, lane, keep, p, acc);
}

// Whether the lane's part of V where `keep` has a bit holds an infinity or a NaN.
template <int D, int KIND>
__device__ __forceinline__ bool not_finite(const uint8_t* tile, uint32_t tile_s, int g, int lane, uint32_t keep) {
    constexpr uint32_t ex = KIND == kBf16 ? 0x7F80u : 0x7C00u;
    const uint32_t m0 = pair_mask(keep), m1 = pair_mask(keep >> 2);
    auto odd = [](uint32_t x) { return (x & ex) == ex || (x & (ex << 16)) == (ex << 16); };
    if (KIND == kInt4) {
        const uint8_t* rec = tile + g * Record<D>::bytes;
        return odd(v_scale_pair<D>(rec, lane >> 2, lane & 3, 0) & m0) || odd(v_scale_pair<D>(rec, lane >> 2, lane & 3, 1) & m1);
    }
    if (KIND == kE4m3) {   // a NaN is a byte 0x7F or 0xFF; the bytes of two positions alternate
        const uint8_t* at = tile + g * Record8<D>::bytes + Record8<D>::v_codes + (lane >> 2) * 64 + (lane & 3) * 16;
        uint32_t found = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t bytes = (keep >> (2 * i) & 1 ? 0x007F007Fu : 0u) | (keep >> (2 * i) & 2 ? 0x7F007F00u : 0u);
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                const uint4 x = *reinterpret_cast<const uint4*>(at + i * (8 * D) + h * 512);
                found |= ((x.x & bytes) + 0x01010101u) | ((x.y & bytes) + 0x01010101u) | ((x.z & bytes) + 0x01010101u) | ((x.w & bytes) + 0x01010101u);
            }
        }
        return found & 0x80808080u;
    }
    bool any = false;
#pragma unroll 1
    for (int j = 0; j < D / 16; ++j) {
        uint32_t f[4];
        v_block<D>(f, tile_s + 16 * TileOf<D, KIND>::row, lane, j, m0, m1);
        any |= odd(f[0]) || odd(f[1]) || odd(f[2]) || odd(f[3]);
    }
    return any;
}

// The values of V that row j of the lane's fragments stands for (two channels), at slot i of a group; 4 bits: q scale / 16; 8 bits: the code.
template <int D, int KIND>
__device__ __forceinline__ float2 v_values(const uint8_t* tile, int g, int r, int i, int j) {
    const int p = slot_position<KIND>(i);
    if (KIND == kInt4) {
        const uint8_t* rec = tile + g * Record<D>::bytes;
        const int c = (D / 8) * r + 2 * j, codes = rec[Record<D>::v_codes + p * (D / 2) + c / 2];
        const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(rec[Record<D>::v_scales + (c / 16) * 16 + p], __NV_E4M3))) * 0.0625f;
        return make_float2((float)((codes & 15) - 8) * s, (float)((codes >> 4) - 8) * s);
    }
    if (KIND == kE4m3) {
        const uint8_t* at = tile + g * Record8<D>::bytes + Record8<D>::v_codes + (p >> 3) * (8 * D) + (r + 8 * (j >> 2)) * 64 + ((p & 7) >> 1) * 16 +
                            (j & 3) * 4 + (p & 1);
        return __half22float2(e4m3_pair((uint16_t)(at[0] | at[2] << 8)));
    }
    const uint16_t* row = reinterpret_cast<const uint16_t*>(tile + (16 + p) * TileOf<D, KIND>::row);
    const uint32_t w = row[16 * j + r] | (uint32_t)row[16 * j + r + 8] << 16;
    return KIND == kBf16 ? bf16x2_to_float2(w) : __half22float2(bits_half2(w));
}

// ------------------------------------------------------------------ a tile
// NG groups of 16 positions from p0 on.  PLAIN: every row sees every one of them; bad: their page is none.
template <int D, int NT, int KIND, int NG, bool PLAIN>
__device__ __forceinline__ void attend_tile(const uint8_t* tile, uint32_t tile_s, int lane, int p0, bool bad, const Rows& rows,
                                            int group, uint32_t mul, int window, const Query<D, NT>& q, Sums<D, NT>& a) {
    constexpr int KM = D / 16;
    const int r = lane >> 2, cq = lane & 3;
    float z[NG][NT][4];
    float un[NG];        // 8 bits: 2^-e_v of a group
    uint32_t keep[NG];   // which of the lane's four V positions of a group any row sees
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) z[g][nt][0] = z[g][nt][1] = z[g][nt][2] = z[g][nt][3] = 0.0f;
        if (KIND == kInt4) scores_int4<D, NT>(tile + g * Record<D>::bytes, r, cq, q, z[g]);
        else if (KIND == kE4m3) scores_e4m3<D, NT>(tile + g * Record8<D>::bytes, r, cq, q, z[g]);
        else scores_16<D, NT, KIND>(tile_s, lane, q, z[g]);
        if (KIND == kE4m3) {
            const int2 e = *reinterpret_cast<const int2*>(tile + g * Record8<D>::bytes + Record8<D>::exponents);
            const float ks = power_of_two(block_exponent(e.x)), ev = (float)block_exponent(e.y);
            un[g] = power_of_two(-block_exponent(e.y));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {   // S 2^e_k first, which is within 2^-65 .. 2^62: z0 2^e_k may be infinite, and 0 times that NaN
                const F2 k2 = f2(ks, ks), q2 = f2(q.z0[nt], q.z1[nt]), v2 = f2(ev, ev);
                const float2 x = parts(fma2(mul2(f2(z[g][nt][0], z[g][nt][1]), k2), q2, v2));
                const float2 y = parts(fma2(mul2(f2(z[g][nt][2], z[g][nt][3]), k2), q2, v2));
                z[g][nt][0] = x.x;
                z[g][nt][1] = x.y;
                z[g][nt][2] = y.x;
                z[g][nt][3] = y.y;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT && KIND != kE4m3; ++nt) {
            z[g][nt][0] *= q.z0[nt];
            z[g][nt][1] *= q.z1[nt];
            z[g][nt][2] *= q.z0[nt];
            z[g][nt][3] *= q.z1[nt];
        }
        keep[g] = 15;
        if (!PLAIN) {
            const bool here = !bad;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int to = rows.last0 + query_of(rows.row0 + nt * 8 + 2 * cq + c, group, mul);   // the last position that this row sees
                    const int before = to >= 0 ? to - window : 0;   // and the one before its window (with to < 0 it sees nothing)
#pragma unroll
                    for (int e = c; e < 4; e += 2) {
                        const int p = p0 + 16 * g + slot_position<KIND>(r) + (e >> 1) * 8;
                        if (!here || p >= rows.len || p > to || (window > 0 && p <= before)) z[g][nt][e] = -INFINITY;
                    }
                }
            // the others may hold anything: their V is taken as 0
            keep[g] = here ? v_bits<KIND>(cq, p0 + 16 * g, rows.any_from, rows.any_until) : 0u;
        }
    }
    // ---- the references
    bool over = false;
    float top[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x = fmaxf(z[0][nt][e], z[0][nt][e + 2]);
            if (NG == 2) x = fmaxf(x, fmaxf(z[NG - 1][nt][e], z[NG - 1][nt][e + 2]));
            top[nt][e] = x;
            over |= x - a.m[nt][e] > kTop;
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
                const float m = fmaxf(a.m[nt][e], x - kLift);
                const float f = exp2_approx(a.m[nt][e] - m);
                a.m[nt][e] = m;
                a.l[nt][e] *= f;
#pragma unroll
                for (int j = 0; j < KM; ++j) {
                    a.o[nt][j][e] *= f;
                    a.o[nt][j][e + 2] *= f;
                }
            }
    }
    // ---- p, and O^T += V^T P^T
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        Weights<NT> p;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float p00 = exp2_approx(z[g][nt][0] - a.m[nt][0]), p01 = exp2_approx(z[g][nt][1] - a.m[nt][1]);
            const float p10 = exp2_approx(z[g][nt][2] - a.m[nt][0]), p11 = exp2_approx(z[g][nt][3] - a.m[nt][1]);
            if (KIND == kE4m3) {
                a.l[nt][0] = fmaf(p00 + p10, un[g], a.l[nt][0]);
                a.l[nt][1] = fmaf(p01 + p11, un[g], a.l[nt][1]);
            } else {
                a.l[nt][0] += p00 + p10;
                a.l[nt][1] += p01 + p11;
            }
            if (KIND == kBf16) {
                // bf16 keeps 8 bits: p as a sum of two, which the products add up in fp32
                const __nv_bfloat162 h0 = __floats2bfloat162_rn(p00, p01), h1 = __floats2bfloat162_rn(p10, p11);
                const float2 f0 = __bfloat1622float2(h0), f1 = __bfloat1622float2(h1);
                p.hi[nt][0] = transpose8(bf162_bits(h0));
                p.hi[nt][1] = transpose8(bf162_bits(h1));
                p.lo[nt][0] = transpose8(bf162_bits(__floats2bfloat162_rn(p00 - f0.x, p01 - f0.y)));
                p.lo[nt][1] = transpose8(bf162_bits(__floats2bfloat162_rn(p10 - f1.x, p11 - f1.y)));
            } else {
                p.hi[nt][0] = transpose8(half2_bits(__floats2half2_rn(p00, p01)));
                p.hi[nt][1] = transpose8(half2_bits(__floats2half2_rn(p10, p11)));
            }
        }
        if (!PLAIN && rows.n > 1 && __any_sync(0xffffffffu, not_finite<D, KIND>(tile, tile_s, g, lane, keep[g]))) {
            // An infinity or a NaN in V where some rows look and others may not: 0 times it is no 0.  The rare tile is
            // added up position by position, each row only where it looks (its p is sent as -1 where it does not).
#pragma unroll 1
            for (int i = 0; i < 16; ++i) {
                float w[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = z[g][nt][i < 8 ? e : e + 2];
                        w[nt][e] = __shfl_sync(0xffffffffu, x == -INFINITY ? -1.0f : exp2_approx(x - a.m[nt][e]), (i & 7) * 4 + cq);
                    }
#pragma unroll
                for (int j = 0; j < KM; ++j) {
                    const float2 v = v_values<D, KIND>(tile, g, r, i, j);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (!(w[nt][e] < 0.0f)) {
                                a.o[nt][j][e] += w[nt][e] * v.x;
                                a.o[nt][j][e + 2] += w[nt][e] * v.y;
                            }
                }
            }
        } else {
            values<D, NT, KIND, !PLAIN>(tile, tile_s, g, lane, keep[g], p, a.o);
        }
    }
}

// ------------------------------------------------------------------ q
// q16: the rows of q, 16-bit elements; gain: of the head's keys (1 for 16-bit pages).
template <int D, int NT, int KIND>
__device__ __forceinline__ void load_query(const uint16_t* q16, int64_t row_stride, int64_t head_stride, bool fp16, int group, uint32_t mul,
                                           float scale_log2, float gain, int lane, const Rows& rows, Query<D, NT>& q) {
    constexpr int KM = D / 16;
    const int r = lane >> 2, cq = lane & 3;
    uint4 raw[KIND == kE4m3 ? NT : 1][D / 32];   // 8 bits: all rows at once, 16 channels of every 64
    if (KIND == kE4m3) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = rows.row0 + nt * 8 + r, t = row < rows.seq_rows ? query_of(row, group, mul) : 0;
            const uint16_t* x16 = q16 + (rows.first_row + t) * row_stride + (rows.h * group + row - t * group) * head_stride + 16 * cq;
#pragma unroll
            for (int w = 0; w < D / 32; ++w)
                raw[KIND == kE4m3 ? nt : 0][w] = row < rows.seq_rows ? *reinterpret_cast<const uint4*>(x16 + 64 * (w >> 1) + 8 * (w & 1)) : make_uint4(0, 0, 0, 0);
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int row = rows.row0 + nt * 8 + r;
        const bool is_row = row < rows.seq_rows;
        const int t = is_row ? query_of(row, group, mul) : 0, g = is_row ? row - t * group : 0;
        const uint16_t* x16 = q16 + (rows.first_row + t) * row_stride + (rows.h * group + g) * head_stride;
        if (KIND == kInt4) {
            constexpr int W = D / 32;                    // words of codes, 8 channels each
            float x[8 * W];
            float top = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (is_row) v = *reinterpret_cast<const uint4*>(x16 + (D / 4) * cq + 8 * w);
                const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = fp16 ? __half22float2(bits_half2(e[i])) : bf16x2_to_float2(e[i]);
                    x[8 * w + 2 * i] = f.x;
                    x[8 * w + 2 * i + 1] = f.y;
                    top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // the largest channel into [2^14, 2^15): a power of two, undone in z0 and z1
            const int ex = min(254, max(1, 268 - (int)(__float_as_uint(top) >> 23)));
            const float up = __uint_as_float((uint32_t)ex << 23);
#pragma unroll
            for (int i = 0; i < KM; ++i) {
                const int w = i >> 1, c = (i & 1) * 2;
                q.set(nt, i, half2_bits(__floats2half2_rn(x[8 * w + c] * up, x[8 * w + c + 4] * up)),
                      half2_bits(__floats2half2_rn(x[8 * w + c + 1] * up, x[8 * w + c + 5] * up)));
            }
            const float z = scale_log2 * gain * 16.0f / up;
            q.z0[nt] = __shfl_sync(0xffffffffu, z, 8 * cq);
            q.z1[nt] = __shfl_sync(0xffffffffu, z, 8 * cq + 4);
        } else if (KIND == kE4m3) {
            float x[D / 4];
            float top = 0.0f;
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const uint4 v = raw[KIND == kE4m3 ? nt : 0][w];
                const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = fp16 ? __half22float2(bits_half2(e[i])) : bf16x2_to_float2(e[i]);
                    x[8 * w + 2 * i] = f.x;
                    x[8 * w + 2 * i + 1] = f.y;
                    top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = min(254, max(1, 268 - (int)(__float_as_uint(top) >> 23)));   // as above
            const float up = __uint_as_float((uint32_t)ex << 23);
#pragma unroll
            for (int i = 0; i < KM; ++i)
                q.set(nt, i, half2_bits(__floats2half2_rn(x[4 * i] * up, x[4 * i + 1] * up)), half2_bits(__floats2half2_rn(x[4 * i + 2] * up, x[4 * i + 3] * up)));
            const float z = scale_log2 / up;
            q.z0[nt] = __shfl_sync(0xffffffffu, z, 8 * cq);
            q.z1[nt] = __shfl_sync(0xffffffffu, z, 8 * cq + 4);
        } else {
#pragma unroll
            for (int i = 0; i < KM; ++i) {
                q.set(nt, i, is_row ? *reinterpret_cast<const uint32_t*>(x16 + 16 * i + 2 * cq) : 0u,
                      is_row ? *reinterpret_cast<const uint32_t*>(x16 + 16 * i + 2 * cq + 8) : 0u);
            }
            q.z0[nt] = q.z1[nt] = scale_log2;
        }
    }
}

}  // namespace tkv
