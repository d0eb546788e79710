/*
 * ep.h -- C ABI of the single-GPU MoE expert-parallel token shuffle
 * (get_dispatch_layout -> dispatch -> combine) for GB300 (sm_103a).
 *
 * The operations are the high-throughput expert-parallel kernels described in
 * "[Not ready] MSCCLPP EP implementation" (mscclpp pull request 852), section
 * "Scope": get_dispatch_layout, intranode_dispatch and intranode_combine (the
 * DeepEP kernels, there ported onto MSCCL++ channels), plus the kUseFP8
 * payload cast of the low-latency dispatch<kUseFP8,...> kernel.  Here all R
 * logical ranks live on one GPU: rank s owns tokens [s*T_r, (s+1)*T_r) of
 * one call and experts [s*E_l, (s+1)*E_l), and every destination rank's
 * receive buffer is a range of rows of one packed device buffer.  The
 * "exchange" is the scatter kernel's own HBM writes; there is no peer
 * traffic and no collective.
 *
 * Notation: T tokens (T % R == 0, T_r = T/R), K top-k slots, E experts
 * (E % R == 0, E_l = E/R), H hidden channels, R ranks, P = number of
 * (token, destination rank) pairs = rows of the receive buffer.
 * src(t) = t / T_r, rank(e) = e / E_l.
 *
 * Conventions shared by every entry point
 *   - Pointers marked "device" are CUDA device pointers (or managed memory);
 *     "host" pointers are ordinary host memory.  The library never
 *     allocates or frees memory: the caller owns every buffer.
 *   - Every call is enqueued on `stream` (NULL = the legacy default stream)
 *     and returns without synchronising, except ep_layout_total_rows.
 *   - Argument checks are done on the host before anything is enqueued; a
 *     failed check returns EP_ERR_INVALID_ARG and enqueues nothing.
 *   - Problems that only the data reveal are reported through an optional
 *     device error word (int32, nullable): the kernels OR EP_ERRBIT_* bits
 *     into it with atomicOr.  The caller zeroes it; the library never clears
 *     it.  No kernel traps.
 *   - All buffers must be 16-byte aligned; x / recv_x / y / out rows are
 *     moved in 16-byte vectors and 1-D bulk (TMA) copies.
 *   - Limits: 1 <= R <= EP_MAX_RANKS, 1 <= K <= EP_MAX_TOPK,
 *     1 <= E <= EP_MAX_EXPERTS, H % 8 == 0 (H % 128 == 0 for FP8),
 *     T * R < 2^31.
 *   - The first call of each kind on a device does a one-time set-up on
 *     the host (kernel attributes, occupancy and cluster-size queries,
 *     cached per device; thread-safe).  Later calls repeat none of it: they
 *     check arguments and launch, so a sequence of calls can be captured
 *     into a CUDA graph once each kind has run eagerly on that device.
 */
#ifndef EP_H_
#define EP_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same opaque type as cudaStream_t / CUstream, so no CUDA header is needed. */
typedef struct CUstream_st* ep_stream_t;

typedef enum {
  EP_OK = 0,
  EP_ERR_INVALID_ARG = 1, /* a host-side argument check failed; nothing enqueued */
  EP_ERR_CAPACITY = 2,    /* a caller-provided buffer is too small (host-visible size) */
  EP_ERR_CUDA = 3,        /* a CUDA runtime call failed (launch, copy, sync) */
  EP_ERR_TIMEOUT = 4      /* reserved: a bounded device wait ran out (see EP_ERRBIT_TIMEOUT) */
} ep_status_t;

/* Bits OR-ed into the device error word. */
#define EP_ERRBIT_BAD_EXPERT 1 /* a topk_idx entry outside [-1, E): treated as masked */
#define EP_ERRBIT_CAPACITY 2   /* a slot >= recv_capacity_rows: that row was not written */
#define EP_ERRBIT_TIMEOUT 4    /* a bounded shared-memory pipeline wait ran out */
#define EP_ERRBIT_SCHED 8      /* a scheduled combine found its counters in use by another
                                  launch, or not zero at launch: tokens may be missing */

#define EP_MAX_RANKS 64
#define EP_MAX_TOPK 32
#define EP_MAX_EXPERTS 4096

/* Human-readable name of a status code (static storage; never NULL). */
const char* ep_status_string(ep_status_t status);

/*
 * Bytes of device scratch that ep_get_dispatch_layout needs for T tokens,
 * R ranks and E experts.  Returns 0 for invalid sizes.  The scratch holds
 * one 64-bit rank mask per token and per-block partial counts; its contents
 * need no initialisation and are dead after the call's kernels finish.
 */
size_t ep_workspace_bytes(int64_t num_tokens, int num_ranks, int num_experts);

/*
 * get_dispatch_layout + slot assignment ("Scope", Intranode:
 * get_dispatch_layout; the internode-combine commit: combine must use the
 * receiver-side prefix matrices, i.e. the slot order is fixed by prefix sums
 * over source rank and token order).
 *
 * In  (device): topk_idx [T, K] int64, row-major; -1 = masked slot.
 * Out (device), every element written:
 *   num_tokens_per_rank   [R, R] int32: [s][r] = tokens of source s sent to r
 *   num_tokens_per_expert [R, E] int32: [s][e] = slots (t,k) with src(t)=s, e_k = e
 *   is_token_in_rank      [T, R] uint8 (0/1; torch.bool storage)
 *   slot                  [T, R] int32: row of (t, r) in the receive buffer,
 *                         -1 if token t is not sent to rank r.  Rows are packed
 *                         destination-major: destination r owns rows
 *                         [recv_base[r], recv_base[r+1]), ordered by source
 *                         rank and then token index.
 *   recv_base             [R + 1] int32: exclusive prefix of rows per
 *                         destination; recv_base[R] = P.
 * err_word (device, nullable): EP_ERRBIT_BAD_EXPERT if some id is outside
 *   [-1, E) (the slot is then treated as masked).
 * workspace (device): at least ep_workspace_bytes(T, R, E) bytes, passed as
 *   workspace_bytes; a smaller value returns EP_ERR_CAPACITY.  Unused (may be
 *   NULL, with workspace_bytes 0) when ep_layout_auto_single_launch(T, R, E):
 *   such batches take the single-launch form described below.
 * T = 0 is valid (counts and recv_base are zeroed).
 * Same as ep_get_dispatch_layout_path(..., EP_LAYOUT_AUTO, stream).
 */
ep_status_t ep_get_dispatch_layout(const int64_t* topk_idx, int64_t num_tokens, int num_topk,
                                   int num_experts, int num_ranks, int32_t* num_tokens_per_rank,
                                   int32_t* num_tokens_per_expert, uint8_t* is_token_in_rank,
                                   int32_t* slot, int32_t* recv_base, int32_t* err_word,
                                   void* workspace, size_t workspace_bytes, ep_stream_t stream);

/*
 * Which kernels compute the layout.  Both forms give identical outputs.
 *
 * EP_LAYOUT_MULTI_LAUNCH: two or three launches spread over the whole GPU
 *   (counts per block of tokens, block offsets, slots), with scratch in the
 *   caller's workspace.  Any size.
 * EP_LAYOUT_SINGLE_LAUNCH: one launch of one thread-block cluster of up to
 *   16 CTAs (8 where the device does not schedule 16), which exchange their
 *   counts through distributed shared memory; no workspace.  For small
 *   batches only (ep_layout_single_launch_fits): T <= 16384 and
 *   R * E <= 16384.  At decode sizes the layout is bound by latency, and
 *   this form removes the round trips between kernels.  The pages run layout, count exchange (notify_dispatch,
 *   cached_notify) and data movement as separate kernels ("Scope",
 *   Internode HT); this fused form has no counterpart there.
 * EP_LAYOUT_AUTO: the single-launch form where it is the faster one
 *   (ep_layout_auto_single_launch: it fits and T <= 8192), else multi-launch.
 *   Should the device refuse the cluster launch (a partition with too few
 *   free SMs, say), AUTO runs the multi-launch form instead if a usable
 *   workspace was passed, and returns EP_ERR_CUDA if not.
 */
typedef enum {
  EP_LAYOUT_AUTO = 0,
  EP_LAYOUT_MULTI_LAUNCH = 1,
  EP_LAYOUT_SINGLE_LAUNCH = 2
} ep_layout_path_t;

/* 1 if the single-launch form applies to (T, R, E), else 0 (also for invalid sizes). */
int ep_layout_single_launch_fits(int64_t num_tokens, int num_ranks, int num_experts);

/* 1 if EP_LAYOUT_AUTO takes the single-launch form for (T, R, E), else 0. */
int ep_layout_auto_single_launch(int64_t num_tokens, int num_ranks, int num_experts);

/*
 * ep_get_dispatch_layout with an explicit choice of kernels (`path`, an
 * ep_layout_path_t).  Arguments and outputs as ep_get_dispatch_layout.
 * Returns EP_ERR_INVALID_ARG, with nothing enqueued, for an unknown path or
 * for EP_LAYOUT_SINGLE_LAUNCH when the batch does not fit it (T = 0
 * included).  The workspace is needed only when the multi-launch form runs.
 */
ep_status_t ep_get_dispatch_layout_path(const int64_t* topk_idx, int64_t num_tokens,
                                        int num_topk, int num_experts, int num_ranks,
                                        int32_t* num_tokens_per_rank,
                                        int32_t* num_tokens_per_expert,
                                        uint8_t* is_token_in_rank, int32_t* slot,
                                        int32_t* recv_base, int32_t* err_word, void* workspace,
                                        size_t workspace_bytes, int path, ep_stream_t stream);

/*
 * The same layout as ep_get_dispatch_layout, for callers that cannot
 * allocate device memory when they call it (the MSCCL++ EP pages have no counterpart to
 * this entry point).  Such callers include plugin or custom-op hosts that
 * hand the library only tensors they already own, C callers with no device
 * allocator of their own, and serving loops whose device-memory budget is
 * fixed at start-up (cudaMalloc may also stall every stream on the device).
 * The scratch comes from a fixed array of EP_NOALLOC_SCRATCH_BYTES inside the
 * library, which every GPU that loads the library holds until the process
 * exits; nothing is allocated or freed.
 *
 * Arguments, outputs and error word: as ep_get_dispatch_layout, without the
 * workspace.  It always runs the multi-launch form (EP_LAYOUT_MULTI_LAUNCH),
 * whatever the batch size; the outputs are the same as those of every other
 * form.  Returns EP_ERR_CAPACITY, with nothing enqueued, when
 * ep_workspace_bytes(T, R, E) exceeds EP_NOALLOC_SCRATCH_BYTES (about 8 bytes
 * per token plus a small per-block term: roughly 800k tokens at 256 experts).
 * The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call
 * before any stream capture.  All calls share the one array, so calls that
 * overlap on the GPU (two streams, or two threads enqueueing at once) race
 * and must be serialised by the caller.  The array needs no clearing: each
 * call writes every scratch word before reading it.
 */
#define EP_NOALLOC_SCRATCH_BYTES (8u << 20)
ep_status_t ep_get_dispatch_layout_noalloc(const int64_t* topk_idx, int64_t num_tokens,
                                           int num_topk, int num_experts, int num_ranks,
                                           int32_t* num_tokens_per_rank,
                                           int32_t* num_tokens_per_expert,
                                           uint8_t* is_token_in_rank, int32_t* slot,
                                           int32_t* recv_base, int32_t* err_word,
                                           ep_stream_t stream);

/*
 * Copies P = recv_base[R] (device) into *host_total_rows and synchronises
 * `stream`.  The only synchronising call; use it to size the receive buffer
 * exactly, or skip it and pass a worst-case capacity of
 * T * min(K, R) rows to ep_dispatch.
 */
ep_status_t ep_layout_total_rows(const int32_t* recv_base, int num_ranks, int32_t* host_total_rows,
                                 ep_stream_t stream);

/*
 * dispatch ("Scope", Intranode: intranode_dispatch; the low-latency port:
 * dispatch<kUseFP8,...>).  For every pair (t, r) with slot[t][r] >= 0:
 *   use_fp8 == 0:  recv_x[slot] = x[t]                      (bf16 bit copy)
 *   use_fp8 == 1:  for each block b of 128 channels,
 *                    amax  = max |x[t][b*128 .. b*128+127]|   (float32)
 *                    a     = max(amax, 1e-4f)
 *                    recv_scales[slot][b] = a / 448          (float32, rounded once)
 *                    recv_x[slot][i] = E4M3(x[t][i] * (448 / a)),
 *                    with 448/a rounded once, one float32 multiply, and the
 *                    E4M3 conversion rounding to nearest even and saturating
 *                    to +-448; dequantise as code * scale.
 *   recv_src_idx[slot]         = t
 *   recv_topk_idx[slot][k]     = e_k - r*E_l if rank(e_k) == r, else -1
 *   recv_topk_weights[slot][k] = w[t][k]     if rank(e_k) == r, else 0.0f
 * In (device): x [T, H] bf16; topk_idx [T, K] int64; topk_weights [T, K]
 *   float32; slot [T, R] int32 from ep_get_dispatch_layout.
 *   num_tokens_per_expert [R, E] int32 from ep_get_dispatch_layout (nullable;
 *   only read to fill num_recv_tokens_per_expert).
 * Out (device): recv_x [capacity, H] bf16, or [capacity, H] E4M3 bytes with
 *   recv_scales [capacity, H/128] float32 (FP8 only, else may be NULL);
 *   recv_src_idx [capacity] int32, recv_topk_idx [capacity, K] int64,
 *   recv_topk_weights [capacity, K] float32 (each nullable: skipped if NULL);
 *   num_recv_tokens_per_expert [R, E_l] int32 (nullable): rows each
 *   destination rank receives per local expert, summed over source ranks.
 *   Rows >= P are not touched.
 * recv_capacity_rows: rows the caller allocated; a pair whose slot is >= it
 *   is skipped and sets EP_ERRBIT_CAPACITY in err_word.  With 0 rows nothing
 *   is written, and recv_x / recv_scales may be NULL (a shard whose tokens
 *   all go nowhere has an empty send buffer).
 * T need not be a multiple of R here (the slots place the rows), so the
 * sharded form below dispatches one rank's own tokens with this call.
 */
ep_status_t ep_dispatch(const void* x, int hidden, const int64_t* topk_idx,
                        const float* topk_weights, int64_t num_tokens, int num_topk,
                        int num_experts, int num_ranks, const int32_t* slot,
                        const int32_t* num_tokens_per_expert, int64_t recv_capacity_rows,
                        int use_fp8, void* recv_x, float* recv_scales, int32_t* recv_src_idx,
                        int64_t* recv_topk_idx, float* recv_topk_weights,
                        int32_t* num_recv_tokens_per_expert, int32_t* err_word,
                        ep_stream_t stream);

/*
 * combine ("Scope", Intranode: intranode_combine; the bench-accounting
 * commit: combine moves one copy per dispatched (token, rank) row back to
 * its owner).  For every token t:
 *   out[t] = bf16_rne( sum over k with e_k != -1 of
 *                      w[t][k] * float(y[slot[t][rank(e_k)]]) )
 * accumulated in float32; a token whose slots are all masked gives +0.
 * A rank named by several slots contributes its row once per slot.
 * With topk_weights == NULL the combine is the unweighted rank sum of the
 * high-throughput kernels (the expert stage has applied the weights):
 *   out[t] = bf16_rne( sum over ranks r with slot[t][r] >= 0 of y[slot[t][r]] ),
 * each destination rank's row once.
 * In (device): y [rows, H] bf16 in dispatch's row layout (expert outputs,
 *   one row per (token, rank) pair), with rows >= P = recv_base[R] (every
 *   row a slot names; the call takes no row count, so this is not checked);
 *   topk_idx [T, K] int64; topk_weights [T, K] float32 (nullable, see
 *   above); slot [T, R] int32 from ep_get_dispatch_layout.
 * Out (device): out [T, H] bf16, every element written.
 * err_word (device, nullable): EP_ERRBIT_BAD_EXPERT for ids outside [-1, E)
 *   (skipped), EP_ERRBIT_TIMEOUT if a bounded pipeline wait ran out (the
 *   output is then incomplete).
 * y rows are staged through shared memory with 1-D bulk (TMA) copies; y and
 * out must not overlap.  T need not be a multiple of R here.
 */
ep_status_t ep_combine(const void* y, int hidden, const int64_t* topk_idx,
                       const float* topk_weights, int64_t num_tokens, int num_topk,
                       int num_experts, int num_ranks, const int32_t* slot, void* out,
                       int32_t* err_word, ep_stream_t stream);

/* ------------------------------------------------------------------------
 * Layout and dispatch in one launch, for small (decode-size) batches.
 *
 * The same outputs as ep_get_dispatch_layout followed by ep_dispatch, from
 * one kernel launch: the pages run layout, the count exchange that fixes
 * the receive offsets (notify_dispatch, cached_notify: "[Not ready] MSCCLPP
 * EP implementation", section "Scope", Internode HT) and the data movement
 * as separate kernels; on one GPU the exchange becomes a wait inside one
 * grid.  The first blocks of the grid to start (picked by an atomic ticket,
 * so that no block waits on one that has not started) compute the layout
 * and meet at a bounded barrier; every block loads its share of x at once
 * and waits, bounded, for the layout before it scatters.  At these sizes the
 * layout is bound by latency, and the fused launch hides the x loads behind
 * it and saves the launches between the kernels.
 *
 * Fits (ep_layout_dispatch_fused_fits): 1 <= T <= 16384 and at most 8192
 * ballots, R * R * ceil(T_r / 32) <= 8192 (one 32-bit ballot per
 * destination and group of 32 tokens, groups never straddling two source
 * ranks): the 4096-token decode batch at 32 ranks, or 16384 tokens at 8
 * ranks.  Other sizes return EP_ERR_INVALID_ARG with nothing enqueued.
 * Arguments: those of ep_get_dispatch_layout (its outputs, all required)
 *   and of ep_dispatch (slot is written here and read back by the scatter;
 *   num_recv_tokens_per_expert is computed here, nullable), plus:
 * workspace (device): ep_layout_dispatch_fused_workspace_bytes(T, R, E)
 *   bytes (about 8 * R * R * ceil(T_r / 32)); EP_ERR_CAPACITY if smaller.
 *   No initialisation needed.
 * sync (device, EP_FUSED_SYNC_WORDS 64-bit words, 8-byte aligned): the
 *   grid's counters (start ticket, barrier, layout done, blocks left) and
 *   release flags, spread over 256-byte lines.  The caller zeroes them once;
 *   every launch leaves them zero again when its last block exits,
 *   including a launch whose waits ran out.  Launches that can overlap on
 *   the GPU need separate states.
 * err_word: as ep_get_dispatch_layout and ep_dispatch, plus
 *   EP_ERRBIT_TIMEOUT if a bounded wait (1 s) ran out: the layout or its
 *   barrier did not complete, and no row was dispatched.
 * ------------------------------------------------------------------------ */
#define EP_FUSED_SYNC_WORDS 640

/* 1 if (T, R, E) fits the one-launch layout + dispatch, else 0. */
int ep_layout_dispatch_fused_fits(int64_t num_tokens, int num_ranks, int num_experts);

/* Bytes of workspace ep_layout_dispatch_fused needs (0 if it does not fit). */
size_t ep_layout_dispatch_fused_workspace_bytes(int64_t num_tokens, int num_ranks,
                                                int num_experts);

ep_status_t ep_layout_dispatch_fused(
    const void* x, int hidden, const int64_t* topk_idx, const float* topk_weights,
    int64_t num_tokens, int num_topk, int num_experts, int num_ranks,
    int32_t* num_tokens_per_rank, int32_t* num_tokens_per_expert, uint8_t* is_token_in_rank,
    int32_t* slot, int32_t* recv_base, int64_t recv_capacity_rows, int use_fp8, void* recv_x,
    float* recv_scales, int32_t* recv_src_idx, int64_t* recv_topk_idx, float* recv_topk_weights,
    int32_t* num_recv_tokens_per_expert, void* workspace, size_t workspace_bytes,
    uint64_t* sync, int32_t* err_word, ep_stream_t stream);

/*
 * Test hook for the bounded waits of ep_layout_dispatch_fused: the next
 * launch from this host thread leaves the first layout block's barrier
 * arrival out, so the barrier and the wait for the layout run out after
 * about 1 s each; the launch then reports EP_ERRBIT_TIMEOUT, dispatches
 * nothing, and still returns its state to zero.  One-shot; 0 cancels it.
 */
void ep_debug_set_fused_stall(int on);

/* ------------------------------------------------------------------------
 * Sharded form: one process and one GPU per rank ("[Not ready] MSCCLPP EP
 * implementation", section "Scope", Intranode: get_dispatch_layout on every
 * rank, then dispatch and combine over peer buffers; the internode
 * notify_dispatch commit: the count exchange that fixes the receiver-side
 * prefix matrices).  Rank s holds its own T tokens.  Per rank:
 *   1. ep_shard_layout: the rank's tokens as the one source of a layout
 *      with R destinations.  Its send buffer is packed destination-major in
 *      token order: destination r's rows are [send_base[r], send_base[r+1]).
 *   2. an all-gather of every rank's send_counts row gives counts [R, R]
 *      (counts[s][r] = tokens of rank s sent to rank r); ep_shard_offsets
 *      turns it into this rank's send and receive offsets.
 *   3. ep_dispatch with slot = send_slot (T need not be a multiple of R)
 *      fills the send buffer; an all-to-all-v moves run r to rank r, which
 *      stores the runs in source-rank order at its receive offsets.  Those
 *      are exactly the rows that destination r holds in the single-call
 *      layout (rows ordered by source rank, then token).  recv_src_idx then
 *      holds each row's token index within its source rank.
 *   4. combine: the reverse all-to-all-v brings every row back into the
 *      send buffer's layout, and ep_combine with slot = send_slot reduces it.
 * The collectives are the caller's (the Python package uses
 * torch.distributed); the library computes the layout, the offsets and the
 * rows.
 * ------------------------------------------------------------------------ */

/* Device scratch for ep_shard_layout (0 for invalid sizes). */
size_t ep_shard_workspace_bytes(int64_t num_tokens, int num_ranks, int num_experts);

/*
 * The layout of one rank's T tokens (any T >= 0) over R destinations.
 * In (device): topk_idx [T, K] int64.
 * Out (device), every element written:
 *   send_counts   [R] int32: tokens sent to each destination
 *   expert_counts [E] int32: slots naming each expert
 *   is_token_in_rank [T, R] uint8, send_slot [T, R] int32 (-1: not sent)
 *   send_base [R + 1] int32: exclusive prefix of send_counts
 * err_word, workspace (ep_shard_workspace_bytes), errors: as
 * ep_get_dispatch_layout.  Always the multi-launch kernels.
 */
ep_status_t ep_shard_layout(const int64_t* topk_idx, int64_t num_tokens, int num_topk,
                            int num_experts, int num_ranks, int32_t* send_counts,
                            int32_t* expert_counts, uint8_t* is_token_in_rank,
                            int32_t* send_slot, int32_t* send_base, int32_t* err_word,
                            void* workspace, size_t workspace_bytes, ep_stream_t stream);

/*
 * Host function (no GPU work).  counts (host) [R, R] int32: counts[s][r] =
 * tokens of rank s sent to rank r (every rank's send_counts, gathered).
 * Out (host): send_offsets [R + 1] int64, the exclusive prefix of
 * counts[rank][.] (this rank's runs in its send buffer); recv_offsets
 * [R + 1] int64, the exclusive prefix of counts[.][rank] (where the run
 * from each source rank lands in this rank's receive buffer;
 * recv_offsets[R] = rows received).  EP_ERR_INVALID_ARG for a negative
 * count or a rank outside [0, R).
 */
ep_status_t ep_shard_offsets(const int32_t* counts, int num_ranks, int rank,
                             int64_t* send_offsets, int64_t* recv_offsets);

/*
 * Host function (no GPU work).  expert_counts (host) [R, E] int32: every
 * rank's expert_counts row, gathered.  Out (host) [E/R] int32: the rows
 * this rank receives for each of its local experts (summed over sources),
 * the rank's row of ep_dispatch's num_recv_tokens_per_expert.
 */
ep_status_t ep_shard_recv_tokens_per_expert(const int32_t* expert_counts, int num_experts,
                                            int num_ranks, int rank, int32_t* out);

/* ------------------------------------------------------------------------
 * Low-latency (expert-major) layout: the receive layout of the low-latency
 * kernels ("[Not ready] MSCCLPP EP implementation", the low-latency port:
 * dispatch<kUseFP8,...> and combine over per-expert buffers indexed
 * [local_expert * num_ranks + dst_rank]).  Every unmasked top-k slot (t, k)
 * has its own row in the buffer of expert e = topk_idx[t][k]; expert e owns
 * rows [e*cap, (e+1)*cap) of one packed buffer of E*cap rows, packed by
 * source rank, then token, then k.
 * ------------------------------------------------------------------------ */

/* Device scratch for ep_ll_get_dispatch_layout (0 for invalid sizes). */
size_t ep_ll_workspace_bytes(int64_t num_tokens, int num_ranks, int num_experts);

/*
 * In (device): topk_idx [T, K] int64, -1 = masked.
 * expert_capacity: rows per expert (cap); cap * E < 2^31.  T is the largest
 *   count any expert can receive when each token names distinct experts.
 * Out (device):
 *   ll_slot [T, K] int32: row of slot (t, k), i.e.
 *     e*cap + ll_src_offset[e][src(t)]
 *     + #{(t', k') of src(t) before (t, k) in (token, k) order naming e};
 *     -1 for masked slots, ids outside [-1, E) (EP_ERRBIT_BAD_EXPERT) and
 *     positions >= cap (EP_ERRBIT_CAPACITY).
 *   ll_count [E] int32: slots naming each expert, over all sources
 *   ll_src_offset [E, R] int32 (nullable): first row of source s within
 *     expert e's rows (relative to e*cap).
 * workspace: ep_ll_workspace_bytes(T, R, E) bytes (EP_ERR_CAPACITY if less);
 *   unused (may be NULL) when ep_ll_layout_auto_single_launch(T, K, R, E).
 * Same as ep_ll_get_dispatch_layout_path(..., EP_LAYOUT_AUTO, stream).
 */
ep_status_t ep_ll_get_dispatch_layout(const int64_t* topk_idx, int64_t num_tokens, int num_topk,
                                      int num_experts, int num_ranks, int64_t expert_capacity,
                                      int32_t* ll_slot, int32_t* ll_count, int32_t* ll_src_offset,
                                      int32_t* err_word, void* workspace, size_t workspace_bytes,
                                      ep_stream_t stream);

/*
 * The expert-major layout's kernels, as for the rank-major layout
 * (ep_layout_path_t):
 *   EP_LAYOUT_MULTI_LAUNCH: three launches over the whole GPU (ranks within
 *     chunks of 16..128 tokens, a prefix over chunks per expert, rows), with
 *     scratch in the caller's workspace.  Any size.
 *   EP_LAYOUT_SINGLE_LAUNCH: one launch of one thread-block cluster of up to
 *     16 CTAs that exchange per-expert counts through distributed shared
 *     memory; no workspace.  Small batches only
 *     (ep_ll_layout_single_launch_fits): E <= 1024, and every warp of a
 *     cluster of 8 CTAs walks at most 2048 slots (roughly T * K <= 131072
 *     when R divides 64).
 *   EP_LAYOUT_AUTO: the single launch whenever it fits (measured faster
 *     at every size it takes); ep_ll_layout_auto_single_launch says which.
 *     As for the rank-major layout, AUTO falls back to the three launches
 *     if the device refuses the cluster and a usable workspace was passed.
 * Both give identical outputs.  EP_LAYOUT_SINGLE_LAUNCH on a batch that does
 * not fit (T = 0 included) returns EP_ERR_INVALID_ARG with nothing enqueued.
 */
int ep_ll_layout_single_launch_fits(int64_t num_tokens, int num_topk, int num_ranks,
                                    int num_experts);
int ep_ll_layout_auto_single_launch(int64_t num_tokens, int num_topk, int num_ranks,
                                    int num_experts);
ep_status_t ep_ll_get_dispatch_layout_path(const int64_t* topk_idx, int64_t num_tokens,
                                           int num_topk, int num_experts, int num_ranks,
                                           int64_t expert_capacity, int32_t* ll_slot,
                                           int32_t* ll_count, int32_t* ll_src_offset,
                                           int32_t* err_word, void* workspace,
                                           size_t workspace_bytes, int path, ep_stream_t stream);

/*
 * Low-latency dispatch: for every slot with ll_slot[t][k] >= 0, row
 * ll_slot[t][k] of recv_x receives token t, as a bf16 copy or (use_fp8) as
 * E4M3 codes with recv_scales per 128 channels, with the same rounding as
 * ep_dispatch; recv_src_idx[row] = t (nullable).  A token named by K experts
 * is written K times.
 * In (device): x [T, H] bf16, ll_slot [T, K].  Out (device): recv_x
 * [capacity, H] (bf16 or bytes), recv_scales [capacity, H/128] f32 (FP8),
 * recv_src_idx [capacity] int32.  Rows >= recv_capacity_rows are skipped
 * and set EP_ERRBIT_CAPACITY; with 0 rows recv_x / recv_scales may be NULL.
 */
ep_status_t ep_ll_dispatch(const void* x, int hidden, int64_t num_tokens, int num_topk,
                           const int32_t* ll_slot, int64_t recv_capacity_rows, int use_fp8,
                           void* recv_x, float* recv_scales, int32_t* recv_src_idx,
                           int32_t* err_word, ep_stream_t stream);

/*
 * Low-latency combine: out[t] = bf16_rne( sum over slots k with
 * ll_slot[t][k] >= 0 of w[t][k] * float(y[ll_slot[t][k]]) ), accumulated in
 * float32 (each expert's output row read once; with topk_weights == NULL
 * every slot weighs 1).  In (device): y [rows, H] bf16 in the expert-major
 * layout, with rows above every row ll_slot names (E * cap suffices; not
 * checked), topk_weights [T, K] f32 (nullable), ll_slot [T, K].  Out
 * (device): out [T, H] bf16, every element written.  Staging as ep_combine.
 */
ep_status_t ep_ll_combine(const void* y, int hidden, const float* topk_weights,
                          int64_t num_tokens, int num_topk, const int32_t* ll_slot, void* out,
                          int32_t* err_word, ep_stream_t stream);

/* ------------------------------------------------------------------------
 * Dynamically scheduled combine.  The combine grid is persistent, and its
 * blocks take the tokens in batches of a few.  Each block's first batch is
 * fixed.  ep_combine and ep_ll_combine hand out the rest statically (block b
 * takes every grid-th batch).  The _sched forms below hand out the rest on
 * demand from a counter in device memory, so a block that the memory system
 * serves faster takes more batches, and all blocks finish together.  On one
 * GB300 this took skewed routing (131072 tokens) from 1586 to 1550 us per
 * layout -> dispatch -> combine step, and Mixtral-shaped routing from 978 to
 * 945 us.  The outputs are identical: each token is summed in the same
 * order whichever block takes it.
 *
 * sched (device, EP_COMBINE_SCHED_WORDS 64-bit words, 8-byte aligned): the
 * counter state.  The caller zeroes it once after allocating it.  Every
 * launch leaves it zero again when its last block exits, including a launch
 * that ran out of a bounded wait.  So one state serves any number of
 * launches in order on one stream, and inside a CUDA graph.  Two combines
 * that can run at the same time (other streams, a graph replayed beside
 * eager calls) need separate states: a shared state would split the tokens
 * between them and leave both outputs incomplete.  A launch checks, as its
 * blocks leave, that it made exactly the claims a launch alone makes and
 * that no claim or exit came from elsewhere; if not (a shared state, or one
 * that was not zero at launch) it sets EP_ERRBIT_SCHED in err_word, and its
 * output may be missing tokens.  A shared state is not always caught (a
 * launch that runs entirely between the other's claims sees nothing amiss,
 * but then neither output is affected).  A NULL sched is the static
 * schedule of ep_combine.  A batch small enough that every block has only
 * its first batch is scheduled statically too, and leaves the state
 * untouched.  Other arguments and errors: as ep_combine and ep_ll_combine.
 * ------------------------------------------------------------------------ */
#define EP_COMBINE_SCHED_WORDS 2

ep_status_t ep_combine_sched(const void* y, int hidden, const int64_t* topk_idx,
                             const float* topk_weights, int64_t num_tokens, int num_topk,
                             int num_experts, int num_ranks, const int32_t* slot, void* out,
                             uint64_t* sched, int32_t* err_word, ep_stream_t stream);
ep_status_t ep_ll_combine_sched(const void* y, int hidden, const float* topk_weights,
                                int64_t num_tokens, int num_topk, const int32_t* ll_slot,
                                void* out, uint64_t* sched, int32_t* err_word,
                                ep_stream_t stream);

/*
 * Test hook for the bounded waits of the combine pipeline (ep_combine,
 * ep_ll_combine and their _sched forms).  The next combine launched from this host thread leaves
 * pipeline unit `unit` of CTA 0 unarmed, so the waits on it run out after
 * about 1 s.  The launch then reports EP_ERRBIT_TIMEOUT in the error word,
 * its output is incomplete, and it returns.  The hook is one-shot; -1
 * cancels it.  It faults, traps and hangs nothing, and exists only so that
 * tests can exercise the timeout path.
 */
void ep_debug_set_combine_stall(int unit);

/*
 * Test hook for the FP8 payload conversion (the pages give the FP8 cast only
 * by name, kUseFP8 in the low-latency port of "[Not ready] MSCCLPP EP
 * implementation"; this hook has no counterpart there).  out[i] receives the
 * E4M3 code that the FP8 dispatch's conversion (round to nearest even,
 * saturating to +-448) gives the float32 whose bit pattern is first + i, for
 * 0 <= i < n, so that a test can compare the oracle's encoder with the
 * device on every float32.  n % 4 == 0 and first + n <= 2^32, else
 * EP_ERR_INVALID_ARG; out: device, n bytes, 4-byte aligned.  Asynchronous
 * on `stream`.
 */
ep_status_t ep_debug_e4m3_range(uint32_t first, int64_t n, uint8_t* out, ep_stream_t stream);

/* ------------------------------------------------------------------------
 * The router: from logits to the topk_idx / topk_weights that the layouts,
 * the dispatch and the combine take, and its gradient.  (The pages start
 * from a finished topk_idx; these entry points have no counterpart there.)
 *
 * For token t with logits l[e], e < E:
 *   score  softmax: s[e] = exp(l[e] - max l) / sum exp(l - max l)
 *          sigmoid: s[e] = 1 / (1 + exp(-l[e]))
 *   key    c[e] = s[e] + bias[e] (bias: a balance term that steers the choice
 *          and stays out of the weights); without a bias c = s for sigmoid
 *          scores and c = l for softmax scores (the same order, no rounding)
 *   groups E/num_groups consecutive experts each; the topk_groups groups with
 *          the largest group scores are kept.  A group's score is the sum of
 *          its two largest keys (sigmoid) or its largest key (softmax).
 *   choice the num_topk largest keys of the kept groups, in descending order
 *   weight u_k = s[e_k]; renormalize: w_k = scale * u_k / sum_j u_j (0 where
 *          the sum is 0), else w_k = scale * u_k.  Renormalised softmax
 *          weights are computed as the softmax over the chosen logits.
 * Ties, of experts and of groups, go to the lowest index.  An expert whose
 * logit is -inf or NaN is never chosen and counts nowhere, also not in its
 * group's score (a group with none left scores -inf); one whose bias makes its
 * key -inf or NaN is never chosen either.  A slot for which no
 * expert is left gets idx -1 and weight 0, the masked slot of every other
 * call.  If the largest softmax logit is +inf, the experts at +inf share the
 * mass equally.  All arithmetic is float32.
 * ------------------------------------------------------------------------ */
typedef enum { EP_SCORE_SOFTMAX = 0, EP_SCORE_SIGMOID = 1 } ep_score_t;

/*
 * In (device): logits [T, E], float32 or (logits_bf16 != 0) bfloat16, rows
 *   row_stride elements apart (>= E), any alignment of the element type; bias
 *   [E] float32 (nullable).
 * score: an ep_score_t.  1 <= num_topk <= min(E, EP_MAX_TOPK); num_groups
 *   divides E and is at most 64, 1 <= topk_groups <= num_groups; 1 and 1: no
 *   groups.
 * Out (device), every element written: topk_idx [T, K] int64, topk_weights
 *   [T, K] float32.
 */
ep_status_t ep_route(const void* logits, int logits_bf16, int64_t row_stride, const float* bias,
                     int64_t num_tokens, int num_experts, int num_topk, int score, int num_groups,
                     int topk_groups, int renormalize, float scale, int64_t* topk_idx,
                     float* topk_weights, ep_stream_t stream);

/*
 * The gradient of the weights w of ep_route with respect to the logits, at a
 * fixed choice topk_idx (a choice has no gradient, so neither has the bias).
 * With du_k = scale * (dw_k - sum_j dw_j u_j / S) / S, S = sum_j u_j
 * (renormalize; 0 where S is 0) or du_k = scale * dw_k:
 *   sigmoid: dl[e] = sum_{k: e_k = e} du_k * u_k (1 - u_k), 0 elsewhere
 *   softmax: dl[e] = s[e] * (sum_{k: e_k = e} du_k - sum_j u_j du_j); with
 *            renormalised weights this is w'_k (scale dw_k - sum_j w'_j scale
 *            dw_j) on the chosen experts, w' = softmax over the chosen
 *            logits, and 0 elsewhere.
 * In (device): dweights [T, K] float32, logits as in ep_route, topk_idx
 *   [T, K] int64 (-1: masked; an id outside [-1, E) is taken as masked and
 *   sets EP_ERRBIT_BAD_EXPERT; an expert named twice sums its slots, k
 *   ascending).  A chosen expert whose logit is -inf or NaN gets 0.
 * Out (device): dlogits [T, E] contiguous, of the logits' type, every element
 *   written (rounded once from float32).  dlogits and logits must not overlap.
 */
ep_status_t ep_route_backward(const float* dweights, const void* logits, int logits_bf16,
                              int64_t row_stride, const int64_t* topk_idx, int64_t num_tokens,
                              int num_experts, int num_topk, int score, int renormalize,
                              float scale, void* dlogits, int32_t* err_word, ep_stream_t stream);

/* ------------------------------------------------------------------------
 * The gradient of the combine.  (That of the dispatch is the combine itself:
 * the unweighted rank sum for the rank-major layout, ep_ll_combine with NULL
 * weights for the expert-major one.)
 * For every row that token t's slots name:
 *   dy[row]          = bf16_rne( W * float(dout[t]) ), W = the sum, k
 *                      ascending, of the weights w[t][k] of the slots that
 *                      name the row (one slot in the expert-major layout,
 *                      every slot of that rank in the rank-major one)
 *   dweights[t][k]   = sum_h float(dout[t][h]) * float(y[row][h])   (float32;
 *                      0 for a masked slot)
 * In (device): dout [T, H] bf16; y [num_rows, H] bf16, topk_idx, topk_weights
 *   (required here) and slot as in ep_combine / ep_ll_combine.
 * Out (device): dy [num_rows, H] bf16: rows that no slot names are not
 *   touched; dweights [T, K] float32, every element written.  Either may be
 *   NULL (skipped; y may be NULL when dweights is).  dy must overlap neither
 *   y nor dout.
 * A row >= num_rows is skipped (its dweights are 0) and sets
 * EP_ERRBIT_CAPACITY; an id outside [-1, E) sets EP_ERRBIT_BAD_EXPERT.
 * ------------------------------------------------------------------------ */
ep_status_t ep_combine_backward(const void* dout, const void* y, int hidden, int64_t num_rows,
                                const int64_t* topk_idx, const float* topk_weights,
                                int64_t num_tokens, int num_topk, int num_experts, int num_ranks,
                                const int32_t* slot, void* dy, float* dweights, int32_t* err_word,
                                ep_stream_t stream);
ep_status_t ep_ll_combine_backward(const void* dout, const void* y, int hidden, int64_t num_rows,
                                   const float* topk_weights, int64_t num_tokens, int num_topk,
                                   const int32_t* ll_slot, void* dy, float* dweights,
                                   int32_t* err_word, ep_stream_t stream);

/* ------------------------------------------------------------------------
 * The experts' products with 4-bit weights, on the rows of the expert-major
 * layout (serving: quantised weights have no gradient).
 *
 * Expert e's rows are x[e*cap .. e*cap + n_e), n_e = min(ll_count[e], cap).
 * Its weights are W_e [N', I] with N' = N (act EP_ACT_NONE) or 2N
 * (EP_ACT_SWIGLU: rows [0, N) are the gate's, rows [N, 2N) the up
 * projection's), held as 4-bit codes q in [0, 16) with one scale and one
 * zero point per group of group_size consecutive input channels:
 *   W_e[n][i] = (q[e][n][i] - zero[e][n][i / group_size]) * scale[e][n][i / group_size]
 *   p[n]      = sum_i W_e[n][i] * x[row][i]                       (float32)
 *   none:   y[row][n] = bf16_rne(p[n])
 *   swiglu: y[row][n] = bf16_rne(p[n] / (1 + exp(-p[n])) * p[N + n])
 * In (device): x [E*cap, I] bf16, or (x_fp8 != 0) E4M3 codes with x_scales
 *   [E*cap, I/128] float32, as ep_ll_dispatch leaves them; ll_count [E] int32;
 *   q [E, N', I/2] bytes, channel i in the low (i even) or high (i odd) half of
 *   byte i/2; scales [E, N', I/group_size] bf16; zeros of the same shape, one
 *   byte each, of which the low four bits count (nullable: every zero point is 8).
 * group_size 32, 64 or 128, dividing I; x_fp8: I % 128 == 0; N % 8 == 0.
 * Out (device): y [E*cap, N] bf16; rows at or beyond n_e are not touched.  y and
 *   x must not overlap.
 * E * cap and E * N' below 2^31.
 * Rounding: q - zero is multiplied as the integer it is, which no type rounds;
 * a group's sum is scaled in float32, and the sums are float32 throughout.  For
 * E4M3 rows of an expert with more than 8 rows, q x and zero x are two products
 * of the same float32 sum, so a group whose weights are all 0 gives a rounding
 * error of that sum there, not always 0.  Experts with more than 8 rows are
 * added up in another order than those with fewer: results may differ in their
 * last bits between the two.  Infinities and NaN stay in their row of x.
 * err_word (nullable): EP_ERRBIT_TIMEOUT if a wait inside the kernel ran out
 *   (after about 1 s; rows of y are then missing).
 * ------------------------------------------------------------------------ */
typedef enum { EP_ACT_NONE = 0, EP_ACT_SWIGLU = 1 } ep_act_t;

ep_status_t ep_ll_experts_w4(const void* x, int x_fp8, const float* x_scales, int in_channels,
                             const int32_t* ll_count, int num_experts, int64_t expert_capacity,
                             const uint8_t* q, const void* scales, const uint8_t* zeros,
                             int group_size, int out_channels, int act, void* y,
                             int32_t* err_word, ep_stream_t stream);

/*
 * Test hook for the bounded waits of ep_ll_experts_w4: the next launch from this
 * host thread of its kernel for more than 8 rows an expert leaves step `step`
 * (128 channels; counted over the block's work) of its first block unloaded,
 * so the waits on it run out after about 1 s.  The launch then reports
 * EP_ERRBIT_TIMEOUT, the block's remaining results are missing, and it returns.
 * One-shot; -1 cancels it.
 */
void ep_debug_set_experts_stall(int step);

/* ------------------------------------------------------------------------
 * A whole mixture-of-experts layer for a few tokens, in two launches: what
 * ep_route, ep_ll_get_dispatch_layout, ep_ll_dispatch, ep_ll_experts_w4 (twice)
 * and ep_ll_combine compute one after the other.
 *
 *   e_k, w_k  the choice of ep_route for the logits' row, the same experts in every case, and its
 *             weights (sums of a token's weights may be added up in another order)
 *   h_k[n]  = w_k * silu(G_{e_k} x)[n] * (U_{e_k} x)[n]
 *   out     = bf16_rne( sum_k D_{e_k} h_k )
 *
 * G and U are rows [0, N) and [N, 2N) of the gate_up weights, D the down weights,
 * held as in ep_ll_experts_w4; the two may differ in their group sizes and in
 * having zero points.  A slot for which no expert is left contributes nothing;
 * a token without any gives zeros.  Codes are multiplied as the integers they
 * are and all sums are float32; h is kept in 16 bits of mantissa (two bf16), so only out is
 * rounded noticeably.  Infinities and NaN stay in their token.
 * In (device): x [T, H] bf16; logits, row_stride, bias, score, num_groups,
 *   topk_groups, renormalize, scale: as ep_route; gate_up_q [E, 2N, H/2],
 *   gate_up_scales [E, 2N, H/gate_up_group] bf16, gate_up_zeros of the same
 *   shape (nullable); down_q [E, H, N/2], down_scales [E, H, N/down_group],
 *   down_zeros (nullable).
 * Limits: T <= EP_LAYER_MAX_TOKENS, E <= EP_LAYER_MAX_EXPERTS, H a multiple of
 *   gate_up_group and N of down_group, H * N < 2^31; those of ep_route.
 * Out (device): topk_idx [T, K] int64, topk_weights [T, K] float32, out [T, H]
 *   bf16, every element written.  out may be x; nothing else may overlap.
 * workspace (device): ep_layer_w4_workspace_bytes(T, N, K) bytes, no
 *   initialisation needed (EP_ERR_CAPACITY if smaller).  Calls that can overlap on
 *   the GPU need workspaces of their own.
 * ------------------------------------------------------------------------ */
#define EP_LAYER_MAX_TOKENS 16
#define EP_LAYER_MAX_EXPERTS 512

/* Bytes of device scratch for ep_layer_w4 (0 for invalid sizes). */
size_t ep_layer_w4_workspace_bytes(int64_t num_tokens, int inter, int num_topk);

ep_status_t ep_layer_w4(const void* x, int hidden, int inter, int64_t num_tokens,
                        const void* logits, int logits_bf16, int64_t row_stride, const float* bias,
                        int num_experts, int num_topk, int score, int num_groups, int topk_groups,
                        int renormalize, float scale, const uint8_t* gate_up_q,
                        const void* gate_up_scales, const uint8_t* gate_up_zeros,
                        int gate_up_group, const uint8_t* down_q, const void* down_scales,
                        const uint8_t* down_zeros, int down_group, int64_t* topk_idx,
                        float* topk_weights, void* out, void* workspace, size_t workspace_bytes,
                        ep_stream_t stream);

/* ------------------------------------------------------------------------
 * What stands between two blocks: the norm after a block, its gate and
 * residual scale, the addition to the residual stream, and the norm before
 * the next block, in one pass.  For every token, with rms(v) = sqrt(mean(v^2) +
 * eps) over the H channels:
 *   n = y / rms(y) * post_weight       (y without a post_weight)
 *   z = x + scale * gate * n           (gate 1 for EP_GATE_NONE)
 *   h = z / rms(z) * pre_weight
 * y is the block's output per token (ll_slot NULL), or the rows of the
 * expert-major layout, which are combined first, as by ep_ll_combine but without
 * its rounding: y[t] = sum over slots k with ll_slot[t][k] >= 0 of w[t][k] * rows[ll_slot[t][k]].
 * h is made from z before its rounding.  All arithmetic is float32, and every
 * output is rounded once.  A row's sum of squares, of y or of z, has to stay below 2^128: a row
 * of one magnitude v reaches that at v = 2^64 / sqrt(H) (2^57 for H = 16384), and from there on
 * its 1 / rms counts as 0.
 * In (device): x [T, H] bf16, or (stream_f32 != 0) float32; y [T, H] or
 *   [num_rows, H] bf16 (NULL without ll_slot: no block's output, h = x / rms(x) *
 *   pre_weight); ll_slot [T, K] int32 and topk_weights [T, K] float32 (nullable: 1
 *   each) with num_rows, num_topk; gate by gate_kind: [H] (EP_GATE_CHANNEL), [T]
 *   (EP_GATE_TOKEN) or [T, H] (EP_GATE_FULL); post_weight, pre_weight [H] (nullable).
 *   gate and the weights are float32, or (weights_bf16 != 0) bfloat16.  eps > 0.
 * Out (device), every element written: z [T, H] of x's type (NULL if and only if there
 *   is no y), h [T, H] bf16 (NULL if and only if pre_weight is), combined [T, H] bf16
 *   (nullable; the combined rows, for the gradient).  z may be x; nothing else may overlap.
 * H % 8 == 0, H <= EP_NORM_MAX_HIDDEN.
 * err_word (nullable): EP_ERRBIT_CAPACITY for a slot >= num_rows (left out).
 * ------------------------------------------------------------------------ */
#define EP_NORM_MAX_HIDDEN 16384
typedef enum {
  EP_GATE_NONE = 0,
  EP_GATE_CHANNEL = 1,
  EP_GATE_TOKEN = 2,
  EP_GATE_FULL = 3
} ep_gate_t;

ep_status_t ep_block_norm(const void* x, int stream_f32, const void* y, int64_t num_rows,
                          const float* topk_weights, int num_topk, const int32_t* ll_slot,
                          int64_t num_tokens, int hidden, const void* gate, int gate_kind,
                          const void* post_weight, const void* pre_weight, int weights_bf16,
                          float scale, float eps, void* z, void* h, void* combined,
                          int32_t* err_word, ep_stream_t stream);

/*
 * The gradient of ep_block_norm, from those of z (dz, of the stream's type) and of h
 * (dh, bf16), at the stored z and y (with rows: the combined y; the gradient of the
 * combine itself is ep_ll_combine_backward).  With d = dh * pre_weight, r_z =
 * 1 / rms(z), r_y = 1 / rms(y):
 *   dx    = dz + r_z d - r_z^3 mean(z d) z
 *   dn    = scale * gate * dx
 *   dy    = r_y dn post_weight - r_y^3 mean(y dn post_weight) y   (dn without a post_weight)
 *   dpre  = sum_t dh z r_z,  dpost = sum_t dn y r_y
 *   dgate = scale * n * dx, summed over what the gate is shared by
 * Beside the sums of squares, a row's sums of the products z d, q dz, q d and q z with q = y *
 * post_weight * gate have to stay below 2^128.
 * Either of dz and dh may be NULL (zero; dh is NULL if and only if pre_weight is);
 * z may be NULL without dh, y without post_weight and gate.
 * Out (device): dx [T, H] of the stream's type; dy [T, H] bf16, dpost_weight and
 *   dpre_weight [H] float32 (each nullable); dgate (nullable): [H] or [T]
 *   float32, or [T, H] of the gate's type.  Sums over tokens are added in an order that the
 *   sizes and the GPU fix, so results repeat.  No output may overlap anything.
 * workspace (device): ep_block_norm_backward_workspace_bytes(T, H) bytes
 *   (EP_ERR_CAPACITY if smaller) where dpre_weight, dpost_weight or a channel's dgate
 *   is asked for, else unused.
 */
size_t ep_block_norm_backward_workspace_bytes(int64_t num_tokens, int hidden);

ep_status_t ep_block_norm_backward(const void* dz, const void* dh, const void* z, int stream_f32,
                                   const void* y, int64_t num_tokens, int hidden, const void* gate,
                                   int gate_kind, const void* post_weight, const void* pre_weight,
                                   int weights_bf16, float scale, float eps, void* dx, void* dy,
                                   void* dgate, float* dpost_weight, float* dpre_weight,
                                   void* workspace, size_t workspace_bytes, ep_stream_t stream);

/* ------------------------------------------------------------------------
 * The experts' gated activation on the rows of the expert-major layout, for
 * training: unlike ep_ll_experts_w4's it keeps what its gradient needs, in 8 bits.
 * For every slot (t, k) with row = ll_slot[t][k] >= 0, [g | u] = gate_up[row]:
 *   h[row]      = bf16_rne( w[t][k] * g / (1 + exp(-g)) * u )    (w NULL: 1 each)
 *   codes[row], scales[row] = g and u as E4M3 with one scale per 128 channels,
 *                 rounded as ep_dispatch rounds its rows (use_fp8); a block of 128
 *                 that holds an infinity or a NaN reads back as NaN throughout
 * All arithmetic is float32, and every output is rounded once (exp(-|g|) below 2^-126 counts as 0).
 * With the weights here, the combine takes none (topk_weights NULL), and the
 * gradient of the weights comes from these rows instead of the experts' outputs.
 * In (device): gate_up [num_rows, 2N] bf16; topk_weights [T, K] float32
 *   (nullable); ll_slot [T, K] int32, in which no row is named twice.
 * Out (device): h [num_rows, N] bf16; codes [num_rows, 2N] and scales [num_rows, 2N/128]
 *   float32 (both or neither).  Rows that no slot names are not touched.
 * N % 8 == 0, with codes N % 128 == 0.  Nothing may overlap.
 * err_word (nullable): EP_ERRBIT_CAPACITY for a slot >= num_rows (skipped).
 * ------------------------------------------------------------------------ */
ep_status_t ep_ll_swiglu(const void* gate_up, int inter, int64_t num_rows,
                         const float* topk_weights, int64_t num_tokens, int num_topk,
                         const int32_t* ll_slot, void* h, uint8_t* codes, float* scales,
                         int32_t* err_word, ep_stream_t stream);

/*
 * Its gradient, from the checkpoint (codes, scales; gate_up NULL) or from gate_up
 * itself (codes and scales NULL).  With s = 1 / (1 + exp(-g)):
 *   dgate_up[row] = [ w dh u s (1 + g (1 - s)) | w dh g s ]     (bf16, rounded once)
 *   dweights[t][k] = sum_n dh g s u     (float32; 0 for a slot without a row)
 * All arithmetic is float32, as above.
 * In (device): dh [num_rows, N] bf16; the rest as ep_ll_swiglu.
 * Out (device): dgate_up [num_rows, 2N] bf16: rows that no slot names are not
 *   touched; dweights [T, K] float32 (nullable), every element written.
 */
ep_status_t ep_ll_swiglu_backward(const void* dh, const void* gate_up, const uint8_t* codes,
                                  const float* scales, int inter, int64_t num_rows,
                                  const float* topk_weights, int64_t num_tokens, int num_topk,
                                  const int32_t* ll_slot, void* dgate_up, float* dweights,
                                  int32_t* err_word, ep_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EP_H_ */
