// Definitions shared by the operators over a caller-owned paged cache (append, gather, attention)
// and the rotation of positions.
//
// 4-bit pages.  A page holds, for every KV head, page_size / 16 records of 16 positions:
//   K codes [16][d/2] | K scales [16][d/16] | V codes [16][d/2] | V scales [d/16][16]
// 18 d bytes: 2,304 at d = 128, 1,152 at d = 64.  A record is the unit that attention copies (one
// contiguous, 128-byte aligned piece of memory for 16 keys and 16 values of a head) and the 16 rows
// of one matrix instruction.  The V scales lie the other way round than the K scales: K's products
// run over the channels of one position, V's over the positions of one channel, and each then finds
// the scales that it multiplies with next to one another.
// A code is q + 8 with q in -7..7; channel 2 j in the low half of byte j, 2 j + 1 in the high half.
// The value is q * scale * gain: scale an E4M3 number >= 0 of a block of 16 channels, gain a power of
// two or any other positive fp32 number of the KV head.  Uniform codes and not E2M1: they expand to
// fp16, times their scale, with one logic and one fused multiply-add instruction a pair, exactly.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/tkv.h"

namespace tkv {

template <int D>
struct Record {
    static constexpr int k_codes = 0, k_scales = 8 * D, v_codes = 9 * D, v_scales = 17 * D, bytes = 18 * D;
};

template <typename T> __device__ __forceinline__ float to_float(T x);
template <> __device__ __forceinline__ float to_float<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_float<__half>(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// 16 bytes as elements of T
template <typename T>
union Vec16 {
    uint4 u;
    T e[16 / sizeof(T)];
};

// One pair by its angle: (x0 + i x1)(c + i s), each product and each sum rounded once, so that the
// rotation on its own and the one on the way into the cache give the same bits.
__device__ __forceinline__ float2 rotate_pair(float x0, float x1, float2 cs) {
    return make_float2(__fsub_rn(__fmul_rn(x0, cs.x), __fmul_rn(x1, cs.y)),
                       __fadd_rn(__fmul_rn(x1, cs.x), __fmul_rn(x0, cs.y)));
}

// Two fp32 numbers an instruction.  A packed product and a packed sum of the same rounding may be fused into one; these two
// have different ones.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 parts(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 mul2_rz(F2 a, F2 b) {
    F2 r;
    asm("mul.rz.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// (cos, sin) of pair j at position p; NaN outside the table, where *bad is set.
__device__ __forceinline__ float2 table_at(const float2* table, int pairs, int max_positions, int p, int j,
                                           float sign, bool* bad) {
    if ((uint32_t)p >= (uint32_t)max_positions) {
        *bad = true;
        return make_float2(__int_as_float(0x7FC00000), __int_as_float(0x7FC00000));
    }
    float2 cs = table[(int64_t)p * pairs + j];
    cs.y *= sign;
    return cs;
}

// The status word holds the largest code that a kernel met.
__device__ __forceinline__ void raise_status(int32_t* status, int code) {
    if (status) atomicMax(status, code);
}

// cs[i] = (cos, sin) of pair j0 + i at a row's positions p, one an axis; j0 is a multiple of N.
template <int N, typename Args>
__device__ __forceinline__ void load_angles(const Args& a, const int (&p)[4], int j0, float2 (&cs)[N]) {
    bool bad = false;
    if (N > 1 && a.num_axes == 1 && a.table_16) {
        const bool in = (uint32_t)p[0] < (uint32_t)a.max_positions;
        const float4* at = reinterpret_cast<const float4*>(a.table + (int64_t)(in ? p[0] : 0) * a.pairs + j0);
        const float nan = __int_as_float(0x7FC00000);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float4 v = at[i];
            cs[2 * i] = in ? make_float2(v.x, v.y * a.sign) : make_float2(nan, nan);
            cs[2 * i + 1] = in ? make_float2(v.z, v.w * a.sign) : make_float2(nan, nan);
        }
        bad = !in;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int x = a.pair_axis[j0 + i];
            cs[i] = table_at(a.table, a.pairs, a.max_positions, x == 0 ? p[0] : x == 1 ? p[1] : x == 2 ? p[2] : p[3], j0 + i, a.sign, &bad);
        }
    }
    if (bad) raise_status(a.status, TKV_EINVAL);
}

// The sequence that row `row` of a step belongs to: cu[b] <= row < cu[b + 1]; -1 behind the last.
__device__ __forceinline__ int sequence_of_row(const int32_t* cu, int batch, int row) {
    if (row < cu[0] || row >= cu[batch]) return -1;
    int lo = 0, hi = batch;   // cu[lo] <= row < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= row) lo = mid; else hi = mid;
    }
    return lo;
}

// The operators' kernels start while the kernel before them in the stream ends (programmatic launches): each reads and writes
// memory only behind wait_for_previous, which lasts until the kernel before it is done and its writes can be seen.  A
// kernel that calls let_next_start first lets its successor start although its predecessor still runs: the successor
// then may not read anything before its own wait.  One kernel does: the one that joins an attention's pieces reads lengths and
// cu_tokens early, so the attention's main kernel lets it start only behind its own wait.
// Every load is an ordinary one.  The read-only path (__ldg, ld.global.nc) is for memory that nothing writes while the kernel
// exists, and these kernels exist before what precedes them has finished: the wait does not hold such a load back, nor does
// it renew a line that the SM read through that path for a kernel still running when this one came.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename Args, typename... Rest>
cudaError_t launch_behind(void (*kernel)(Args, Rest...), dim3 grid, int threads, int smem, cudaStream_t st, const Args& args, Rest... rest) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args, rest...);
}

// How many heads the threads of a row take at once, each thread walking over up to `most`: the row's place and angles are then
// found once for them, which costs about as much as a head.  A call takes as long as its waves of CTAs (`at_once` of them,
// `blocks` a head), and the last one is rarely full: 4,096 rows of 32 heads to rotate took 18.5 us with two waves and a half
// of threads, 13.4 like this.
inline int spread_heads(int64_t blocks, int64_t heads, int64_t at_once, int most) {
    int64_t best = 0;
    int chosen = 1;
    for (int per_thread = most; per_thread >= 1; --per_thread) {
        int64_t lanes = (heads + per_thread - 1) / per_thread;
        if (lanes > 65535) lanes = 65535;
        const int64_t cost = (blocks * lanes + at_once - 1) / at_once * ((heads + lanes - 1) / lanes + 1);
        if (best && cost >= best) continue;
        best = cost;
        chosen = (int)lanes;
    }
    return chosen;
}

// Host-side checks shared by the entry points; TKV_OK or TKV_EINVAL.
tkv_status check_rotary(const tkv_rotary* r, int head_dim, bool need_positions);
tkv_status check_paged(const tkv_paged* c);
// element (row, head, channel) -> memory: rows and heads do not overlap, strides >= 0
bool strides_apart(int64_t rows, int64_t row_stride, int64_t heads, int64_t head_stride, int64_t width);
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline int dtype_size(int t) { return t == TKV_FP32 ? 4 : 2; }
inline bool is_dtype(int t) { return t == TKV_BF16 || t == TKV_FP16 || t == TKV_FP32; }

}  // namespace tkv
