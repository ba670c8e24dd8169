/*
 * tkv.h -- tiered KV-cache decode attention for one GB300 GPU (sm_103a).
 *
 * The method ("Not All Thoughts Need HBM: Semantics-Aware Memory Hierarchy
 * for LLM Reasoning"; gist.science summary and fugumt.com abstract) keeps
 * every token of a reasoning chain in one of four tiers:
 *
 *   T0  HBM, full precision (bf16)          -- protected tokens and the most
 *                                              important reasoning tokens
 *   T1  pinned host DDR, full precision     -- fetched back into HBM before
 *                                              each attention step (or read
 *                                              from an HBM copy the re-tier
 *                                              keeps: TKV_T1_RESIDENT)
 *   T2  8-bit (FP8-E4M3, one fp32 scale per token, layer and KV head, for K
 *       and for V), kept in HBM or in pinned host memory (TKV_T2_HOST) and
 *       dequantised inside the attention load
 *   T3  evicted (dropped from every store)
 *
 * ranked by the cumulative attention score
 *     s_i(t) = s_i(t-1) + (1/|L|) sum_l (1/H) sum_h alpha_{l,h}(t)[i]
 * ("Importance scoring") and re-tiered every Delta decode steps ("System
 * implementation", Delta = 64).  The prompt, the first `num_sinks` tokens and
 * the last `recent_window` tokens are protected and always in T0
 * ("Four-tier classification").
 *
 * Conventions for every call:
 *   - Device pointers are caller-owned CUDA device memory (e.g. a torch
 *     tensor's data_ptr()) and must stay valid until the work enqueued on the
 *     context's compute stream has completed.  Host pointers are caller-owned
 *     and are only read or written during the call.
 *   - All GPU work is enqueued asynchronously on the context's streams; calls
 *     return without waiting unless their comment says they synchronise.
 *   - No call aborts or traps.  Argument errors return TKV_EINVAL and change
 *     nothing.  The first CUDA error (or a device-side status word set by a
 *     kernel) poisons the context: that call returns TKV_ECUDA / TKV_ETIMEOUT /
 *     TKV_ECAPACITY and every later call except tkv_destroy, tkv_get_stats and
 *     tkv_status_string returns TKV_ESTATE.
 *   - One context is used from one host thread at a time.
 *   - Fault injection (a test hook for the error paths, host side only): if
 *     the environment variable TKV_FAULT_INJECT is set when tkv_create runs,
 *       "hostalloc"  makes that context's pinned host allocations fail
 *                    (tkv_create returns TKV_ENOMEM and frees what it took);
 *       "call:N"     makes the N-th checked CUDA call of that context (counted
 *                    from 1 after creation) report failure after it ran:
 *                    the call returns TKV_ECUDA, the context is poisoned
 *                    (tkv_stats.cuda_error = cudaErrorUnknown) and no device
 *                    work goes wrong.
 *
 * Shapes: L layers, B sequences, Hq query heads, Hkv KV heads, G = Hq / Hkv,
 * d = head_dim (64 or 128).  Query head h reads KV head h / G (GQA).
 * All sequences of a batch advance together: they hold the same number N of
 * positions.
 */
#ifndef TKV_H
#define TKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TKV_OK = 0,
    TKV_EINVAL = 1,     /* bad argument or call out of order; nothing changed */
    TKV_ENOMEM = 2,     /* device or pinned host allocation failed */
    TKV_ECUDA = 3,      /* a CUDA runtime call failed; context poisoned */
    TKV_ECAPACITY = 4,  /* a tier store or the position capacity is full */
    TKV_ETIMEOUT = 5,   /* a bounded device-side wait ran out; context poisoned */
    TKV_ESTATE = 6      /* context poisoned by an earlier error */
} tkv_status;

typedef struct tkv_ctx tkv_ctx;

/* T1 transports (tkv_config.t1_transport): the same bytes land in the same
 * staging rows either way, so results do not depend on the choice.
 *   TKV_T1_COPY_ENGINE  one cudaMemcpy2DAsync per layer on the copy stream
 *   TKV_T1_SM_COPY      a copy kernel on the copy stream whose threads load
 *                       the pinned host rows directly (zero-copy) and store
 *                       them to staging
 *   TKV_T1_SPLIT        half the rows by the copy engine, half by the copy
 *                       kernel on a second stream, concurrently
 *   TKV_T1_MULTI_CE     the rows split four ways over four copy streams, so
 *                       that several copy engines run at once
 *   TKV_T1_RESIDENT     the other reading of "System implementation": an HBM
 *                       copy of every layer's T1 rows is kept next to the host
 *                       store and updated by the re-tier's moves, so only the
 *                       delta crosses the host link (no per-step T1 stream;
 *                       T1 then occupies HBM like T0) */
enum { TKV_T1_COPY_ENGINE = 0, TKV_T1_SM_COPY = 1, TKV_T1_SPLIT = 2, TKV_T1_MULTI_CE = 3,
       TKV_T1_RESIDENT = 4 };

/* Where the T2 rows (E4M3 codes + fp32 scales) live (tkv_config.t2_placement):
 *   TKV_T2_HBM   in an HBM pool that the attention kernel reads in place
 *   TKV_T2_HOST  in pinned host memory, the placement "Four-tier
 *                classification" gives T2: each layer's T2 records are copied
 *                with its T1 rows into an HBM staging ring before its attention.
 * The same bytes reach the kernel either way, so the results are identical. */
enum { TKV_T2_HBM = 0, TKV_T2_HOST = 1 };

/* How the pinned host stores (T1 rows, full-precision copies of T2 rows, host
 * T2 records) are allocated (tkv_config.host_alloc):
 *   TKV_HOST_HUGE_ARENA    an anonymous mapping aligned to and populated with
 *                          transparent huge pages, bound to the host NUMA node
 *                          closest to the device when the host has several,
 *                          registered with cudaHostRegister (mapped, portable);
 *                          falls back to cudaHostAlloc if a step fails.  Huge
 *                          pages keep the host link's DMA translations few, so
 *                          the per-step copy of a store of tens of GB keeps to
 *                          the link's rate.
 *   TKV_HOST_PINNED_ALLOC  cudaHostAlloc (mapped, portable).
 *   TKV_HOST_AUTO          the huge-page arena for stores of 1 GiB or more,
 *                          cudaHostAlloc below (default).
 * The bytes stored are the same either way. */
enum { TKV_HOST_AUTO = 0, TKV_HOST_PINNED_ALLOC = 1, TKV_HOST_HUGE_ARENA = 2 };

typedef struct {
    int32_t num_layers;       /* L >= 1 */
    int32_t num_q_heads;      /* Hq, a multiple of num_kv_heads, Hq / Hkv <= 8 */
    int32_t num_kv_heads;     /* Hkv >= 1 */
    int32_t head_dim;         /* d: 64 or 128 */
    int32_t batch;            /* B >= 1 */
    int32_t max_tokens;       /* capacity of positions per sequence, <= 65536 */
    int32_t prompt_len;       /* protected prompt [0, prompt_len) */
    int32_t num_sinks;        /* protected attention sinks [0, num_sinks) */
    int32_t recent_window;    /* protected recent window [N - W, N) */
    int32_t retier_interval;  /* Delta; informational for callers (tkv_retier is explicit) */
    float ratio_t0;           /* tier shares of N; held internally as parts per million */
    float ratio_t1;
    float ratio_t2;
    float ratio_t3;
    int32_t t0_capacity;      /* HBM T0 slots per sequence; 0 = max_tokens */
    int32_t t1_capacity;      /* pinned-host T1 slots per sequence (and HBM staging rows); 0 = max_tokens */
    int32_t t2_capacity;      /* T2 slots per sequence; 0 = max_tokens if ratio_t2 > 0, else 0 */
    int32_t t1_transport;     /* how T1 rows reach the attention kernel: TKV_T1_COPY_ENGINE,
                                 TKV_T1_SM_COPY, TKV_T1_SPLIT, TKV_T1_MULTI_CE or TKV_T1_RESIDENT
                                 (see above) */
    int32_t device;           /* CUDA device ordinal */
    void* compute_stream;     /* cudaStream_t for attention, append, fold, re-tier; NULL = create a
                                 non-blocking one (then order the caller's work with tkv_sync);
                                 cudaStreamLegacy / cudaStreamPerThread are accepted */
    void* copy_stream;        /* cudaStream_t for T1 prefetch and delta prefetch; NULL = create one */
    int32_t t2_placement;     /* where T2 rows live: TKV_T2_HBM (0, default) or TKV_T2_HOST */
    int32_t host_alloc;       /* host stores: TKV_HOST_AUTO (0, default), TKV_HOST_PINNED_ALLOC or
                                 TKV_HOST_HUGE_ARENA (see above) */
} tkv_config;

typedef struct {
    int64_t num_tokens;            /* N: positions per sequence so far */
    int64_t step;                  /* decode steps completed */
    int64_t retiers;               /* re-tiers completed */
    int64_t tier_count[4];         /* tokens per tier, summed over the batch */
    int64_t t1_rows_streamed;      /* T1 slots copied per layer per sequence per step (high-water mark) */
    int64_t last_promoted;         /* last re-tier: tokens moved into T0 from T1/T2 (summed over batch) */
    int64_t last_demoted_t1;       /* last re-tier: tokens moved T0 -> T1 */
    int64_t last_quantised;        /* last re-tier: tokens moved into T2 */
    int64_t last_evicted;          /* last re-tier: tokens newly evicted */
    int64_t last_t2_to_t1;         /* last re-tier: tokens moved T2 -> T1 */
    int64_t h2d_bytes_t1_stream;   /* cumulative bytes of the per-layer T1 stream */
    int64_t h2d_bytes_delta;       /* cumulative bytes of delta prefetch (promotions) */
    int64_t d2h_bytes_writeback;   /* cumulative bytes written back to the host stores */
    int64_t hbm_bytes_allocated;   /* device bytes held by the context */
    int64_t host_bytes_allocated;  /* pinned host bytes held by the context */
    int64_t hbm_bytes_kv_resident; /* KV bytes in HBM now: T0 rows + T2 rows (or their two staged layers)
                                      + T1 staging (or the resident T1 copy) */
    int64_t kv_bytes_full_cache;   /* bf16 KV bytes of all N positions (no tiering) */
    int64_t kernel_launches;       /* kernels this context has launched (all kinds) */
    int32_t status;                /* tkv_status of the context */
    int32_t attn_splits;           /* CTAs of the last attention launch */
    int64_t h2d_bytes_t2_stream;   /* cumulative bytes of the per-layer T2 stream (TKV_T2_HOST) */
    int64_t host_huge_bytes;       /* bytes of the host stores backed by huge pages */
    int32_t host_numa_node;        /* NUMA node the host stores are bound to, -1 = none */
    int32_t cuda_error;            /* cudaError_t of the CUDA call that poisoned the context, 0 = none */
    int32_t cuda_error_line;       /* source line of that call in the library (diagnostics) */
    int32_t pad0;
} tkv_stats;

/* Creates a context: device pools for T0 (bf16), T2 (fp8 + scales) and the
 * two-deep T1 staging ring, pinned mapped host stores for T1 and for the
 * full-precision copy of T2 rows, page tables and the score vector s.
 * Every position starts in T0.  Ownership of *out passes to the caller.
 * Errors: TKV_EINVAL (shape/ratio checks), TKV_ENOMEM, TKV_ECUDA. */
tkv_status tkv_create(const tkv_config* cfg, tkv_ctx** out);

/* Frees everything the context holds (after synchronising its streams). */
void tkv_destroy(tkv_ctx* ctx);

/* Appends n_tokens new positions for one layer ("Four-tier classification":
 * new tokens fall in the recent window, so they enter T0).
 * k, v: device bf16 [B][n_tokens][Hkv][d].
 * k and v must be 16-byte aligned (TKV_EINVAL otherwise).
 * Protocol: a group of n tokens opens with layer 0 and every layer is
 * appended in order 0..L-1.  With n_tokens == 1 the group is a decode step:
 * tkv_decode_step(layer) follows tkv_append(layer), and the step closes after
 * tkv_decode_step(L-1).  A decode token's rows are written into T0 by the
 * attention kernel of that tkv_decode_step (no launch of their own), so k and v
 * must stay valid and unchanged until that call's work has run on the compute
 * stream.  With n_tokens > 1 (prefill) the rows are copied on the compute
 * stream at once and the positions are committed when layer L-1 is appended;
 * pre-filled positions start with s = 0 and are not scored.
 * Errors: TKV_EINVAL (layer out of order, NULL pointers, n_tokens < 1),
 * TKV_ECAPACITY (max_tokens or T0 capacity would be exceeded; nothing changes). */
tkv_status tkv_append(tkv_ctx* ctx, int32_t layer, const void* k, const void* v,
                      int32_t n_tokens);

/* Enqueues, on the copy stream, the fetch of `layer`'s T1 rows (full
 * precision, pinned host -> HBM staging slot layer % 2) and, on the first step
 * after a re-tier, the delta prefetch of the rows newly promoted into T0 for
 * that layer ("Zero-approximation-error offloading": T1 rows are fetched
 * before each attention step; "System implementation": asynchronous delta
 * prefetch of newly promoted tokens only).  Call it for layer l+1 before
 * tkv_decode_step(l) so the copy overlaps layer l's attention; if it was not
 * called, tkv_decode_step(layer) issues it itself.  Layers may be prefetched
 * in any order (at most two layers ahead of the attention): each layer's
 * delta is enqueued, once, before that layer's fetch completes.
 * Errors: TKV_EINVAL (layer out of range, or called twice for one layer in
 * one step). */
tkv_status tkv_prefetch(tkv_ctx* ctx, int32_t layer);

/* Decode attention of one layer for the open decode step, over all retained
 * positions (T0, T1, T2; T3 excluded) in logical order, with the softmax
 * scale 1/sqrt(d).  Also emits, per retained position, the sum over this
 * layer's query heads of the attention weights, and on the last layer folds
 * them into s ("Importance scoring").  The result does not depend on which of
 * T0 / T1 a token sits in (Proposition 1): the work split and the order of
 * every sum depend only on the retained set.
 * q: device bf16 [B][Hq][d].  out: device fp32 [B][Hq][d].
 * Errors: TKV_EINVAL (no open decode step, layer not yet appended, or out of
 * order), TKV_ECUDA. */
tkv_status tkv_decode_step(tkv_ctx* ctx, int32_t layer, const void* q, float* out);

/* Re-tiers every sequence by its current scores ("System implementation":
 * every Delta = 64 decode steps; the caller calls it when step % Delta == 0,
 * after tkv_decode_step(L-1)).  Ranking key: s descending, lower position
 * first on exact ties.  Counts: n_k = floor(ratio_k * N) with ratios held in
 * parts per million; T0's count includes the protected set; T3 is cumulative
 * and never gives a token back; after evictions T0, then T2, take their
 * targets from the ranked list and T1 takes the remainder (T1 shrinks first,
 * then T2, if the protected set is too large).
 * Rows leaving T0 are written back to the host store or quantised here; rows
 * entering T0 are fetched by the next step's tkv_prefetch.  Synchronises the
 * compute stream once (reads back the move counts).
 * Errors: TKV_EINVAL (a decode step or prefill group is open),
 * TKV_ECAPACITY (a tier store is full; context poisoned), TKV_ECUDA. */
tkv_status tkv_retier(tkv_ctx* ctx);

/* Copies s to the host: dst [B][N] fp32.  Synchronises. */
tkv_status tkv_get_scores(tkv_ctx* ctx, float* dst_host);

/* Replaces s from the host: src [B][N] fp32 (test hook: feed given scores to
 * the re-tier).  Synchronises. */
tkv_status tkv_set_scores(tkv_ctx* ctx, const float* src_host);

/* Copies the tier of every position to the host: dst [B][N] uint8 (0..3).
 * Synchronises. */
tkv_status tkv_get_tiers(tkv_ctx* ctx, uint8_t* dst_host);

/* Moves every position to the given tier (test hook, e.g. for Proposition 1:
 * same T3 set, different T0/T1 splits): src [B][N] uint8.  Data moves exactly
 * as in tkv_retier.  An evicted position cannot be given back a tier, and a
 * protected position (sinks, prompt, recent window at the current N) cannot be
 * evicted (TKV_EINVAL, nothing changes).  Synchronises. */
tkv_status tkv_set_tiers(tkv_ctx* ctx, const uint8_t* src_host);

/* Inspection hook: copies the stored K and V rows of one position of one
 * layer and sequence, from wherever its tier keeps them, to the host, and
 * returns its tier in *tier_out.
 *   T0 / T1: dst_host receives bf16 [2][Hkv][d] (K rows, then V rows) from
 *            the HBM T0 pool or the pinned host T1 store; scales untouched.
 *   T2:      dst_host receives the E4M3 codes uint8 [2][Hkv][d] and
 *            scales_host the fp32 scales [2][Hkv] from the HBM T2 pool.
 *   T3:      nothing is copied.
 * dst_host must hold 2*Hkv*d*2 bytes; scales_host 2*Hkv floats (may be NULL
 * when the caller knows the position is not in T2).  Synchronises.
 * Errors: TKV_EINVAL (indices out of range). */
tkv_status tkv_get_row(tkv_ctx* ctx, int32_t layer, int32_t seq, int32_t pos, void* dst_host,
                       float* scales_host, int32_t* tier_out);

/* Time and bytes of one kind of work between tkv_profile_begin and _end. */
typedef struct {
    double ms;          /* summed CUDA-event time of the timed launches or copies */
    int64_t count;      /* launches or copies timed */
    double bytes;       /* algorithmic bytes they moved */
} tkv_prof_entry;

/* Kernel and copy timing.  tkv_profile_begin clears the counters and, until
 * tkv_profile_end, brackets with CUDA events (at most 16384 of each kind):
 *   attn   -- every launch of the attention main kernel, on the compute
 *             stream, right around the kernel (after its wait for the T1
 *             fetch).  Bytes per launch and sequence: 4*Hkv*d per T0/T1 row,
 *             2*Hkv*d + 8*Hkv per T2 row (codes + two fp32 scales), plus q
 *             (bf16);
 *   combine -- every launch of the attention combine kernel that follows it
 *             (the bracket between the two kernels keeps them from
 *             overlapping while timed); bytes: out (fp32) plus, per retained
 *             row and KV head, its logits and its alpha running sum;
 *   t1     -- every per-layer T1 copy (pinned host -> HBM staging) on the
 *             copy stream; bytes = rows copied * 4*Hkv*d;
 *   delta  -- every delta-prefetch gather of promoted rows on the copy stream;
 *             bytes = rows gathered * 4*Hkv*d.
 * tkv_profile_end synchronises, stops recording and fills the entries (any
 * pointer may be NULL). */
tkv_status tkv_profile_begin(tkv_ctx* ctx);
tkv_status tkv_profile_end(tkv_ctx* ctx, tkv_prof_entry* attn, tkv_prof_entry* combine,
                           tkv_prof_entry* t1, tkv_prof_entry* delta);

/* Allocation-free decode step for callers that cannot let a library allocate
 * device memory: runtimes whose caching allocator owns the whole memory
 * budget, and decode loops that cannot afford the device-wide stalls that
 * cudaMalloc / cudaFree may cause.  The paper has no counterpart: this is a
 * packaging of the same attention kernel and score fold as tkv_decode_step,
 * over a dense cache in which every position is retained and resident.
 *   q:   device bf16 [L][B][Hq][d]
 *   kv:  device bf16 [L][2][B][Hkv][R][d]   (K rows, then V rows; positions
 *        0..R-1 in logical order, the decoded token included), 16-byte aligned
 *   out: device fp32 [L][B][Hq][d]
 *   s:   device fp32 [B][R], read and updated in place: s += the step's mean
 *        over layers and query heads of the attention weights
 *   stream: cudaStream_t to enqueue on (NULL = the legacy default stream)
 * Scratch lives in fixed file-scope device arrays (about 34 MiB), held by
 * every GPU that loads the library until exit: B*Hkv*R <= 131,072,
 * B*R <= 131,072, B <= 256; larger sizes return TKV_ECAPACITY before anything
 * is enqueued.
 * It calls no cudaMalloc, cudaFree or other allocating routine.  The first
 * call on a device (with that device current) resolves the scratch addresses
 * and should come before any stream capture.  All calls share the scratch and
 * leave their contents in it, so calls that overlap on the GPU race.  The call
 * enqueues work and returns without waiting.
 * Errors: TKV_EINVAL (NULL pointers, a misaligned kv, shapes), TKV_ECAPACITY
 * (beyond the limits above), TKV_ECUDA. */
tkv_status tkv_decode_dense_noalloc(const void* q, const void* kv, float* out, float* s,
                                    int32_t num_layers, int32_t batch, int32_t num_q_heads,
                                    int32_t num_kv_heads, int32_t head_dim, int32_t num_positions,
                                    void* stream);

/* CUDA-graph decode steps.  The pages have no counterpart: this is how a
 * serving loop takes the host-side cost of the per-layer calls (and the gaps
 * between launches) off a decode step.
 * tkv_capture_begin: between decode steps, with no delta prefetch pending
 * (i.e. not on the first step after a re-tier), profiling off and any T1
 * transport but TKV_T1_SPLIT.  The caller then makes one
 * decode step's calls (tkv_append / tkv_prefetch / tkv_decode_step for every
 * layer) as usual: they are recorded into a graph, on an internal stream, and
 * nothing runs.  tkv_capture_end instantiates the graph, puts the context back
 * to its state before the step and sets *steps_valid to the number of
 * replays the graph stays valid for (the launch geometry covers the retained
 * counts; capacity).  tkv_replay launches the graph on the compute stream: one
 * decode step, with the pointers given at capture (the caller refills those
 * buffers before each replay).  Any re-tier, tkv_set_tiers or prefill append
 * discards the graph.
 * Errors: TKV_EINVAL (call order, conditions above, no valid graph, the
 * captured calls were not exactly one decode step), TKV_ECUDA. */
tkv_status tkv_capture_begin(tkv_ctx* ctx);
tkv_status tkv_capture_end(tkv_ctx* ctx, int32_t* steps_valid);
tkv_status tkv_replay(tkv_ctx* ctx);

/* Measurement hook (no counterpart on the pages, which quote PCIe Gen5 x16 for
 * their prototype's host link): the bandwidth of this device's host link as
 * seen by the two ways the library moves host rows.  Allocates `bytes` of
 * pinned mapped host memory and of device memory, times the best of three
 * passes of each kind with CUDA events on a stream of its own, frees both and
 * synchronises:
 *   h2d_ce_gbs  one cudaMemcpyAsync, pinned host -> device (the copy engine
 *               that carries the per-layer T1 stream);
 *   h2d_sm_gbs  the library's copy kernel loading the mapped host buffer
 *               (zero-copy; the path the delta prefetch and TKV_T1_SM_COPY use);
 *   d2h_ce_gbs  one cudaMemcpyAsync, device -> pinned host.
 * GB/s = 1e9 bytes per second.  Any output pointer may be NULL.
 * Errors: TKV_EINVAL (bytes < 1 MiB or not a multiple of 16, device < 0),
 * TKV_ENOMEM, TKV_ECUDA. */
tkv_status tkv_measure_host_link(int32_t device, int64_t bytes, double* h2d_ce_gbs, double* h2d_sm_gbs,
                                 double* d2h_ce_gbs);

/* ------------------------------------------------------------------------
 * Operators over a paged cache that the caller owns.
 *
 * The pages have no counterpart for these calls: they are what a decode layer
 * around the attention needs when its cache is not a tiered context -- the
 * rotation of positions, rows into a paged cache with the rotation of k on the
 * way, attention over that cache held in 4 bits, in 8 or in 16, rows back out,
 * and beam search: the choice of the beams' continuations, and caches that follow
 * the beams that were chosen.
 *
 * Conventions of these calls, beyond those at the top of this file:
 *   - They have no context and keep nothing: the caller owns every buffer, they
 *     allocate nothing, never synchronise, can be captured into a CUDA graph, and
 *     may be called from several host threads.  Their work is enqueued on
 *     `stream` (NULL = the legacy default stream) of the current device, on
 *     which all pointers must lie.
 *   - A step's rows are ragged.  cu_tokens: device int32 [batch + 1],
 *     not descending; sequence b owns rows cu_tokens[b] .. cu_tokens[b + 1] - 1 of
 *     k, v, q and out, and they are its last positions: row cu_tokens[b] + i
 *     is position lengths[b] - n_b + i, n_b = cu_tokens[b + 1] - cu_tokens[b].
 *     `rows` is the extent of the tensors; rows behind cu_tokens[batch] are
 *     left as they were (a captured step can be padded).  lengths counts the
 *     step's own tokens, so one array serves append and attention.  Both launches
 *     of an attention read lengths and cu_tokens.
 *   - Strides count elements; the channels of a head are contiguous.  Inputs
 *     may be broadcast (stride 0); the elements of an output may not overlap.
 *   - The device arrays (positions, page table, lengths, cu_tokens) cannot be
 *     checked by the host.  No kernel reads or writes outside the buffers for
 *     any value in them.  What is wrong is left out as each call says and
 *     reported in `status`: a device int32 that the caller clears (or NULL),
 *     raised to TKV_EINVAL (a position outside the rotary table; in the attention
 *     a sequence whose cu_tokens descend or leave the rows), TKV_ECAPACITY
 *     (a page or a position outside the cache) or TKV_ETIMEOUT (in the attention a
 *     wait for a copy of the kernel's own ran out: the rows that it was for are NaN),
 *     the largest.  With NULL none of them is reported. */

/* Element types.  TKV_INT4 and TKV_E4M3 are types of pages only. */
enum { TKV_BF16 = 0, TKV_FP16 = 1, TKV_FP32 = 2, TKV_INT4 = 3, TKV_E4M3 = 4 };

/* A rotation of positions.  Of a head's channels the first 2 * pairs are
 * turned in pairs, (j, j + pairs) or, if interleaved, (2j, 2j + 1):
 *   y0 = x0 cos - x1 sin,  y1 = x1 cos + x0 sin
 * by the angle that the table holds for pair j at position
 * positions[pair_axis[j]][row]: with one axis, text; with several (time,
 * height, width), each section of the pairs follows its own axis.  inverse
 * turns by the negated angle, which is the gradient of the forward call. */
typedef struct {
    const float* table;         /* device fp32 [max_positions][pairs][2]: cos, sin; 8-byte aligned */
    const int32_t* positions;   /* device int32 [num_axes][axis_stride], the row innermost; may be NULL in
                                   tkv_paged_append with one axis: the row's position in the cache */
    int64_t axis_stride;        /* elements from one axis to the next */
    int32_t max_positions;      /* rows of the table */
    int32_t pairs;              /* 1 .. 256, 2 * pairs <= head_dim */
    int32_t num_axes;           /* 1 .. 4 */
    int32_t interleaved;        /* 0: pair j is channels j, j + pairs; 1: channels 2j, 2j + 1 */
    int32_t inverse;            /* 0: forward, 1: by the negated angle */
    uint8_t pair_axis[256];     /* axis of each pair, below num_axes */
} tkv_rotary;

/* A paged cache.  Position p of sequence b lies in page page_table[b][p /
 * page_size].  Pages, by kv_type:
 *   TKV_BF16, TKV_FP16  [num_pages][Hkv][2][page_size][d]   (2 = K, V)
 *   TKV_INT4            [num_pages][Hkv][page_size / 16][18 d] bytes: records of
 *       16 positions, K codes [16][d/2] | K scales [16][d/16] | V codes [16][d/2] |
 *       V scales [d/16][16].  A code is q + 8, q in -7..7, in four bits (channel
 *       2j in the low half of byte j); a scale is the E4M3 number of 16
 *       channels; the value is q * scale * gain of the KV head.  The append
 *       writes scale = amax / (7 gain), to nearest even, saturating at 448, and
 *       q = x / (scale gain), to nearest even; a block with an infinity or a
 *       NaN reads as NaN.  A quotient within 2^-22 of a tie may go to either side
 *       where gain is not a power of two.  Choose gain so that amax / (7 gain) falls in E4M3's
 *       normal range, 2^-6 .. 448: amax / 1024 of what the head is expected to
 *       hold leaves room on both sides.
 *   TKV_E4M3            [num_pages][Hkv][page_size / 16][32 d + 16] bytes: records of
 *       16 positions, K codes [d/64][16][64] | V codes [2][d/8][4][8][2] | int32 e_k,
 *       e_v | 8 unused bytes.  K: 64 channels of 16 positions at a time; V: half of the
 *       positions, channel / 8, pair of positions, channel, position of the pair.  The
 *       value is E4M3(code) * 2^e, with one e for the 16 positions of a block and
 *       head, of K and of V (e outside -32 .. 31 counts as the nearer of these).
 *       The append finds the least e in that range with amax <= 448 * 2^e, amax the largest
 *       finite magnitude of the block's new rows; where rows of the block precede
 *       them, e never falls, and if it grows their codes are rounded anew: only what falls below
 *       2^-6 of the new scale can change.  A code is x 2^-e to nearest even, saturating (at
 *       448 * 2^31); an infinity or a NaN is stored as NaN, and the block's other values stay
 *       what they are.  The rows of a block that come after the step's are as good as free:
 *       sequences that share a block's page may not append to it.  Rows that are taken back
 *       (lengths set back behind drafted tokens) leave their block's e behind: a drafted row with a
 *       magnitude 2^k times the others' leaves the rows that stay, and those that come, on a scale
 *       that is 2^k as coarse, until the block's first position is written again. */
typedef struct {
    void* pages;                /* device, 16-byte aligned */
    const int32_t* page_table;  /* device int32 [batch][max_pages] */
    const int32_t* lengths;     /* device int32 [batch]: positions of each sequence, the step's included */
    const float* k_gain;        /* device fp32 [Hkv], > 0; TKV_INT4 only; NULL = 1 */
    const float* v_gain;
    int64_t num_pages;
    int32_t kv_type;            /* TKV_BF16, TKV_FP16, TKV_INT4 or TKV_E4M3 */
    int32_t num_kv_heads;       /* Hkv >= 1 */
    int32_t head_dim;           /* d: 64 or 128 */
    int32_t page_size;          /* a power of two, 16 .. 65536 */
    int32_t batch;              /* B >= 1 */
    int32_t max_pages;          /* pages a sequence; max_pages * page_size <= 2^30 */
} tkv_paged;

/* Rotates x into out, which may be x itself (same strides) and may not overlap it otherwise.
 * x, out: device [rows][heads][head_dim] of dtype (TKV_BF16, TKV_FP16 or
 * TKV_FP32), rows up to 2^31 - 1, any strides that keep out's elements apart; channels behind the
 * rotated ones are copied.  Computed in fp32, rounded once.  Fastest
 * where everything starts on 16-byte boundaries.  A position outside the table turns
 * its pairs into NaN and raises status to TKV_EINVAL.
 * Errors: TKV_EINVAL, TKV_ECUDA. */
tkv_status tkv_rope(const tkv_rotary* rotary, const void* x, void* out, int32_t dtype, int64_t rows,
                    int32_t heads, int32_t head_dim, int64_t x_row_stride, int64_t x_head_stride,
                    int64_t out_row_stride, int64_t out_head_stride, int32_t* status, void* stream);

/* Writes a step's k and v into their pages; k is rotated on the way if rotary is
 * not NULL (before it is rounded to the pages' type).
 * k, v: device [rows][Hkv][d] of dtype TKV_BF16 or TKV_FP16 (the pages' own type if
 * they are 16-bit), 16-byte aligned, strides multiples of 8.
 * A row whose position is negative or beyond the page table, or whose page is
 * not in [0, num_pages), is dropped and raises status to TKV_ECAPACITY.  Two
 * rows that the page table sends to the same place race: one of them stays, or
 * a mixture.  Errors: TKV_EINVAL, TKV_ECUDA. */
tkv_status tkv_paged_append(const tkv_paged* cache, const tkv_rotary* rotary, const void* k, const void* v,
                            int32_t dtype, int64_t rows, int64_t k_row_stride, int64_t k_head_stride,
                            int64_t v_row_stride, int64_t v_head_stride, const int32_t* cu_tokens,
                            int32_t* status, void* stream);

/* The reverse: reads positions out of the pages into k and v, addressed like an
 * append (lengths[b] = the end of the range, n_b its extent).
 * k, v: device [rows][Hkv][d] of dtype TKV_BF16, TKV_FP16 or TKV_FP32, 16-byte
 * aligned, strides multiples of 16 bytes; a 4-bit or 8-bit value is rounded to fp32,
 * and every value from there to dtype.  A row
 * without a place (see the append) reads as NaN and raises status.
 * Errors: TKV_EINVAL, TKV_ECUDA. */
tkv_status tkv_paged_gather(const tkv_paged* cache, void* k, void* v, int32_t dtype, int64_t rows,
                            int64_t k_row_stride, int64_t k_head_stride, int64_t v_row_stride,
                            int64_t v_head_stride, const int32_t* cu_tokens, int32_t* status, void* stream);

/* Attention of a step's queries over the paged cache: one query a sequence in
 * plain decoding, several where drafted tokens are checked or a prompt is
 * continued.  Query row cu_tokens[b] + i, at position p = lengths[b] - n_b + i,
 * sees the positions <= p and, with window > 0, > p - window.  Query head h
 * reads KV head h / (num_q_heads / Hkv).
 *   out = softmax(scale q.k) v in q's type, lse = log of the sum of
 *   exp(scale q.k) (natural; NULL = not wanted; joins partial results over
 *   several caches); a query that sees nothing gets out = 0, lse = -infinity.
 * q, out: device [rows][num_q_heads][d] of dtype TKV_BF16 or TKV_FP16 (the pages'
 * own type if they are 16-bit), 16-byte aligned, strides multiples of 8, not
 * overlapping; lse:
 * device fp32 [rows][num_q_heads], contiguous.
 * A step's size is limited: (rows * num_q_heads / Hkv / 8 + batch) * Hkv *
 * (max_pages * page_size / 32, rounded up) tiles (16 positions a tile with 16-bit
 * pages, and with 8-bit pages of d 128) are at most 2 * 10^9; a longer prompt enters in parts.
 * max_new and max_len are the host's estimates of the largest n_b and the largest
 * length.  They choose how the work is split, not what is computed: any
 * values >= 1 give right results, better ones faster.
 * workspace: device memory of tkv_paged_attention_workspace(...) bytes, 16-byte
 * aligned, contents irrelevant; calls that may run at the same time need one
 * each.  Results of one call's inputs are the same every time; a
 * sequence's last bits may depend on the lengths of the others (they move
 * the places where its sums are split).  Positions in a page outside
 * [0, num_pages), and a sequence's positions beyond the page table, are left
 * out and raise status to TKV_ECAPACITY.  A sequence whose cu_tokens descend or
 * leave the rows is left out and raises it to TKV_EINVAL.
 * Errors: TKV_EINVAL, TKV_ECAPACITY (workspace too small), TKV_ECUDA. */
tkv_status tkv_paged_attention(const tkv_paged* cache, const void* q, void* out, float* lse, int32_t dtype,
                               int64_t rows, int32_t num_q_heads, int64_t q_row_stride, int64_t q_head_stride,
                               int64_t out_row_stride, int64_t out_head_stride, const int32_t* cu_tokens,
                               int32_t max_new, int32_t max_len, int32_t window, float scale, void* workspace,
                               int64_t workspace_bytes, int32_t* status, void* stream);

/* Bytes of workspace that tkv_paged_attention needs on the current device for
 * this cache, num_q_heads and max_new (0 if the arguments are refused).  Does
 * not depend on lengths. */
int64_t tkv_paged_attention_workspace(const tkv_paged* cache, int32_t num_q_heads, int32_t max_new);

/* Beam search: the best continuations of each sequence's beams.
 *   total[b][w][v] = scores[b][w] + logits[b][w][v] - log sum_v exp(logits[b][w][v])
 * and the outputs are the `count` largest over (w, v), in descending order, ties to the
 * lowest w * vocab + v: the total, the beam w and the token v.  Totals are compared in 64 bits.
 * Within a beam the order is that of the logits, even where their totals are equal in 64 bits.
 * finished (device uint8 [batch][beams], or NULL): a beam where it is not 0 offers
 * one candidate, token eos with the beam's own score; its logits are not read.
 * A beam with a score that is not finite, or with a NaN or +infinity among its logits, offers
 * none, and no candidate has a logit of -infinity or a total below the lowest fp32 number.
 * Places that are left over get score -infinity, beam -1 and token -1.  A row's log of its sum is
 * good to about 2^-20, and the same for equal rows.
 * logits: device [batch][beams][vocab] of dtype TKV_BF16, TKV_FP16 or TKV_FP32, the
 * vocabulary contiguous, strides in elements (any alignment); scores: device fp32
 * [batch][beams]; out_scores, out_beams, out_tokens: device [batch][count].
 * Limits: beams and count 1 .. 64, beams * vocab < 2^31 - 256; tkv_paged_reorder follows 32 beams at most.
 * workspace: tkv_beam_select_workspace(...) bytes on the current device, 16-byte aligned,
 * contents irrelevant; calls that may run at the same time need one each.
 * Errors: TKV_EINVAL (eos outside the vocabulary with `finished` among them), TKV_ECAPACITY
 * (workspace too small), TKV_ECUDA. */
tkv_status tkv_beam_select(const void* logits, int32_t dtype, int64_t batch, int32_t beams, int32_t vocab, int64_t batch_stride,
                           int64_t beam_stride, const float* scores, const uint8_t* finished, int32_t eos, int32_t count,
                           float* out_scores, int32_t* out_beams, int32_t* out_tokens, void* workspace, int64_t workspace_bytes,
                           void* stream);

/* Bytes of workspace of tkv_beam_select on the current device (0 if the arguments are refused, or batch is 0). */
int64_t tkv_beam_select_workspace(int32_t dtype, int64_t batch, int32_t beams, int32_t vocab, int32_t count);

/* The caches of a model's layers follow the chosen beams: sequence g * beams + w goes on
 * from sequence g * beams + parents[g * beams + w].
 * caches: host array of num_caches descriptors that share page_table, lengths, batch,
 * max_pages and page_size; types, heads and head_dim may differ, and no two have the same pages.  parents:
 * device int32 [batch]; a negative one means that the sequence keeps what it has.
 * The columns of the page table before a sequence's current page (lengths / page_size) become
 * its parent's, so beams share pages that are full; what the current, partly filled
 * page holds (whole records of 4-bit and 8-bit pages) is copied, in every cache, from the parent's page into
 * the sequence's own.  The table's columns from the current one on stay as they are, and the pages
 * in them have to be each sequence's own.  So a prompt that one sequence has appended is given to its
 * group by parents of that sequence; a child that keeps its parent costs nothing.
 * What is wrong is reported in status, and left as it was: a parent >= beams (TKV_EINVAL, as if
 * negative), a group whose sequences differ in length (TKV_EINVAL), lengths outside the table and pages
 * outside [0, num_pages) (TKV_ECAPACITY; the table's columns are exchanged all the same in the
 * latter case).  The page table is written, although the descriptor's pointer is const.
 * Limits: beams 1 .. 32, page_size * Hkv < 2^26.  Errors: TKV_EINVAL, TKV_ECUDA. */
tkv_status tkv_paged_reorder(const tkv_paged* caches, int32_t num_caches, const int32_t* parents, int32_t beams, int32_t* status,
                             void* stream);

/* Waits for all enqueued work and reports any device-side status word. */
tkv_status tkv_sync(tkv_ctx* ctx);

/* Counters and sizes; valid on a poisoned context too. */
tkv_status tkv_get_stats(tkv_ctx* ctx, tkv_stats* out);

/* Static string for a status code. */
const char* tkv_status_string(tkv_status s);

#ifdef __cplusplus
}
#endif

#endif /* TKV_H */
