/*
 * Exact attention forward (bf16 and FP8, on device or host buffers), backward, paged-KV
 * decoding over bf16 and 8-bit caches, the cache's append and the partial-result merge of ring
 * attention for NVIDIA B200 (sm_100a): C ABI.
 *
 * Computes, for every batch b, query head h and query row i,
 *
 *     out[b,h,i,:] = sum_j softmax_j(scale * q[b,h,i,:] . k[b,g(h),j,:] + mask(i,j)) * v[b,g(h),j,:]
 *     lse[b,h,i]   = ln sum_{j visible} exp(scale * q[b,h,i,:] . k[b,g(h),j,:])
 *
 * which is the masked softmax attention of "Efficient attention: long context and
 * sub-quadratic variants" (stanleyjacob.dev), section "Implementation, twice"
 * (masked_attention: masked scores are -inf before the softmax, each row is
 * renormalised over its visible keys), computed tile by tile with an online
 * softmax so the N x N score matrix never reaches HBM (same page, section
 * "FlashAttention: exact attention, IO-aware").
 *
 * Masks (mask(i,j) = 0 where visible, -inf elsewhere):
 *   ATTN_MASK_FULL            every key;
 *   ATTN_MASK_CAUSAL          j <= i ("Efficient Attention: Flash Attention, Sliding
 *                             Window, Sparse", creativeworksofknowledge.com, section "Code":
 *                             is_causal=True);
 *   ATTN_MASK_SLIDING_WINDOW  i - window < j <= i (stanleyjacob.dev, section
 *                             "Sliding-window and local attention" and sliding_window_mask);
 *                             a window >= N is exactly causal and is run as causal.
 *                             With sinks (attn_fwd_options) the first keys stay visible too.
 * Head sharing (GQA/MQA): query head h reads key/value head g(h) = h / (Hq / Hkv)
 * ("Attention Mechanism Variants Beyond Self-Attention", tempatgunting.com, section
 * "Multi-Query and Grouped-Query Attention": repeat_interleave on the head axis).
 * The log-sum-exp output is not on those pages; it is the natural-log normaliser of
 * each row's softmax, written so a caller can merge or recompute partial results.
 */
#ifndef ATTN_B200_ATTN_H_
#define ATTN_B200_ATTN_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_MASK_FULL = 0,
  ATTN_MASK_CAUSAL = 1,
  ATTN_MASK_SLIDING_WINDOW = 2
} attn_mask_kind;

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_INVALID_ARG = 1,  /* null pointer, bad size, bad mask, window < 1, scale not finite or <= 0,
                                overlapping buffers */
  ATTN_ERR_UNSUPPORTED = 2,  /* head dimension other than 64 or 128, or no sm_100 device */
  ATTN_ERR_MISALIGNED = 3,   /* q, k, v or out not 16-byte aligned, lse not 4-byte aligned */
  ATTN_ERR_CUDA = 4,         /* a CUDA runtime / driver call failed (launch, tensor-map encode) */
  ATTN_ERR_TIMEOUT = 5,      /* a device-side wait gave up (reported by attn_debug_error) */
  ATTN_ERR_RANGE = 6         /* a V value that fp16 cannot hold (magnitude >= 2^16, or not finite) met
                                the default fp16 P V product (reported by attn_debug_error) */
} attn_status;

/*
 * attn_fwd: enqueue the forward on `stream` and return immediately.
 *
 *   q    device pointer, bf16, [B, Hq,  N, d], contiguous (d fastest), 16-byte aligned
 *   k    device pointer, bf16, [B, Hkv, N, d], contiguous, 16-byte aligned
 *   v    device pointer, bf16, [B, Hkv, N, d], contiguous, 16-byte aligned
 *   out  device pointer, bf16, [B, Hq,  N, d], contiguous, 16-byte aligned; fully overwritten
 *   lse  device pointer, fp32, [B, Hq,  N],    contiguous, 4-byte aligned; fully overwritten
 *   B, Hq, Hkv, N >= 1; Hq % Hkv == 0; d in {64, 128}
 *   scale      finite and > 0 (usually 1/sqrt(d)); multiplies q.k before the mask
 *   mask_kind  an attn_mask_kind
 *   window     >= 1 when mask_kind == ATTN_MASK_SLIDING_WINDOW, ignored otherwise
 *   stream     CUDA stream (0 = legacy default stream) of the current device, which
 *              must own all five buffers
 *
 * Ownership: the caller owns every buffer. The library allocates no device memory and
 * never synchronises; out and lse are written by the kernel when the stream reaches it.
 * out and lse must not overlap each other or the inputs (ATTN_ERR_INVALID_ARG).
 * Precision: scores and sums are fp32; the softmax weights P go to the tensor core as
 * fp16 (11 significant bits), with V converted to fp16 on chip, and out is rounded once
 * to bf16. V values must therefore have magnitude below 2^16 (every finite bf16 value
 * up to 65280 qualifies); a larger or non-finite V value makes the launch's result
 * undefined and is reported by attn_debug_error as ATTN_ERR_RANGE. attn_fwd_ex with
 * p_bf16 = 1 takes any V, with P rounded to bf16 instead (8 significant bits: out can
 * then be off by about one bf16 ulp of a value near 1 where one or two keys dominate).
 * Errors: every argument is checked before anything is enqueued; on error nothing is
 * launched and the status says why. ATTN_ERR_CUDA reports a failed launch. Device-side
 * waits are bounded (about 2 s); a wait that gives up makes the kernel stop early and
 * leave a code that attn_debug_error returns as ATTN_ERR_TIMEOUT.
 */
int attn_fwd(const void* q, const void* k, const void* v, void* out, float* lse,
             int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t d,
             float scale, int mask_kind, int64_t window, cudaStream_t stream);

/* Options for attn_fwd_ex (and the _ex forms of the other calls, which say which
   fields they read). Zero-initialise, then set what is needed. */
typedef struct {
  uint64_t wait_timeout_ns; /* bound of every device-side wait; 0 = default (2 s) */
  int inject_stall;         /* test hook: 1 = the loader issues no copies, so every consumer
                               wait runs out and the kernel exits with ATTN_ERR_TIMEOUT
                               pending in attn_debug_error; nothing faults or hangs */
  int grid_ctas;            /* number of persistent CTAs; 0 = one per SM */
  unsigned int* item_visits; /* test hook (forward): NULL, or a device array of
                               attn_fwd_num_work_items() counters, each incremented once
                               per visit of its work item (the caller zeroes it) */
  int p_bf16;               /* 1 = P and V go to the P V product as bf16 (any V value, coarser
                               P); 0 = fp16 (default; |V| below 2^16). bf16 inputs only */
  int out_fp32;             /* forward: 1 = out is fp32 [B, Hq, N, d] (16-byte aligned) and
                               receives O / l unrounded, for partial results that are merged
                               afterwards (attn_merge mode 2 or 3); 0 = bf16 out */
  int64_t key_offset;       /* forward, causal and window masks: query row i sits at key
                               position i + key_offset (>= 0), so it sees keys j <= i + key_offset
                               (and, with a window, j > i + key_offset - window), e.g. a query
                               block against an earlier key block in ring attention; rows that
                               see no key end with out 0 and lse -inf. 0 = the square masks */
  int bwd_deterministic;    /* backward, d = 128: 1 = the two-kernel path (query-tile dQ kernel,
                               key-tile dK/dV kernel; seven matmuls per pair, dq bitwise
                               reproducible, workspace 4 B Hq N bytes, 4-byte aligned);
                               0 = the fused key-tile kernel where Hq == Hkv (default) */
  int64_t sinks;            /* sliding window (forward, backward, decoding): the first `sinks` keys
                               stay visible to every row at or behind them, beside the row's window:
                               key j is visible if j <= i and (j > i - window or j < sinks), with i
                               the row's position (key_offset added). 0 = none; > 0 is refused with
                               the other masks, as is < 0. A decoding step looks up the pages that
                               hold sinks, and none between them and the window */
} attn_fwd_options;

/* attn_fwd with options (same arguments, same checks); opts may be NULL. */
int attn_fwd_ex(const void* q, const void* k, const void* v, void* out, float* lse,
                int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t d,
                float scale, int mask_kind, int64_t window, cudaStream_t stream,
                const attn_fwd_options* opts);

/*
 * attn_fwd_fp8: the same forward with E4M3 inputs. q, k, v hold 8-bit E4M3 codes (OCP
 * format: bias 7, no infinities, largest magnitude 448) in the layouts of attn_fwd, with
 * one scale per tensor: element value = E4M3(code) * q_scale (k_scale, v_scale). The
 * result is the exact attention of those values (scale multiplies their q.k), out bf16
 * and lse fp32 as attn_fwd. The pages name FP8 inputs as a feature of the production
 * kernel line ("Efficient Attention: Flash Attention, Sliding Window, Sparse",
 * creativeworksofknowledge.com, section "Flash Attention (exact, memory-efficient)").
 * Inside, q.k runs on E4M3 tensor-core products and P is rounded to E4M3 (times 2^8)
 * for the product with V; accumulation is fp32.
 *
 *   q, k, v      device pointers to uint8 codes, [B, Hq|Hkv, N, d], contiguous, 16-byte aligned
 *   q_scale, k_scale, v_scale   finite and > 0
 *   d            128 only (ATTN_ERR_UNSUPPORTED otherwise)
 *   everything else as attn_fwd
 */
int attn_fwd_fp8(const void* q, const void* k, const void* v, float q_scale, float k_scale, float v_scale,
                 void* out, float* lse, int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t d,
                 float scale, int mask_kind, int64_t window, cudaStream_t stream);
/* attn_fwd_fp8 with options (as attn_fwd_ex); opts may be NULL. */
int attn_fwd_fp8_ex(const void* q, const void* k, const void* v, float q_scale, float k_scale, float v_scale,
                    void* out, float* lse, int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t d,
                    float scale, int mask_kind, int64_t window, cudaStream_t stream,
                    const attn_fwd_options* opts);

/*
 * attn_fwd_host: attn_fwd on HOST buffers, with the copies overlapped with the work.
 * The (batch, key/value head) units are independent and a contiguous range of units is a
 * contiguous range of every tensor, so the job is cut into `chunks` ranges. Each range is
 * uploaded on a copy stream. Its forward runs on `stream` once it has arrived, and its out
 * and lse go back on a second copy stream once computed. Different chunks' uploads, kernels
 * and downloads therefore run at the same time.
 *
 *   hq, hk, hv    host pointers, layouts and types of attn_fwd's q, k, v (page-locked
 *                 memory lets the copies overlap; pageable memory works, more slowly)
 *   hout, hlse    host pointers, layouts of attn_fwd's out and lse; must not overlap the
 *                 host inputs or each other
 *   dq, dk, dv, dout, dlse   device staging buffers with attn_fwd's sizes, alignment and
 *                 overlap rules (owned by the caller; their contents are overwritten);
 *                 since the uploads write dq, dk and dv, these three must not overlap
 *                 one another either (ATTN_ERR_INVALID_ARG)
 *   B ... window  as attn_fwd
 *   chunks        number of ranges, >= 0; 0 = 8; more than B * Hkv means B * Hkv
 *   stream        CUDA stream of the current device
 *
 * Everything is enqueued and the call returns. hout and hlse are complete when `stream`
 * reaches the point after the call: `stream` waits for the last download. The call does
 * not block the host unless the host memory is pageable, in which case the runtime may
 * copy synchronously. The library keeps two copy streams per device, created on first
 * use, and allocates no memory. Errors: arguments are checked before anything is
 * enqueued, as in attn_fwd, and so is the device (ATTN_ERR_UNSUPPORTED unless sm_100).
 * If something fails part way, its status is returned: ATTN_ERR_CUDA for a copy, the
 * chunk's attn_fwd status for a launch. `stream` is still ordered after whatever had been
 * enqueued.
 */
int attn_fwd_host(const void* hq, const void* hk, const void* hv, void* hout, float* hlse,
                  void* dq, void* dk, void* dv, void* dout, float* dlse,
                  int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t d,
                  float scale, int mask_kind, int64_t window, int64_t chunks, cudaStream_t stream);
/* attn_fwd_host for the E4M3 inputs of attn_fwd_fp8 (same scales, same restrictions). */
int attn_fwd_fp8_host(const void* hq, const void* hk, const void* hv,
                      float q_scale, float k_scale, float v_scale, void* hout, float* hlse,
                      void* dq, void* dk, void* dv, void* dout, float* dlse,
                      int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t d,
                      float scale, int mask_kind, int64_t window, int64_t chunks, cudaStream_t stream);

/*
 * attn_merge: fold one partial attention result into an accumulator, the combining step of
 * ring attention ("Attention Mechanism Variants Beyond Self-Attention", tempatgunting.com,
 * section "Ring Attention for Very Long Sequences": each GPU holds a chunk of the sequence
 * and key/value blocks rotate around a ring). For each row, with partial (O_p, lse_p) over
 * one set of keys and accumulated (O_a, lse_a) over a disjoint set,
 *   lse = ln(e^lse_a + e^lse_p),  O = e^(lse_a - lse) O_a + e^(lse_p - lse) O_p,
 * the attention over the union (each partial O is normalised by its own softmax sum).
 *
 *   acc_out   device, fp32 [rows, d], 16-byte aligned; read (mode 1) and written
 *   acc_lse   device, fp32 [rows], natural log; read (mode 1) and written
 *   part_out  device, [rows, d] (attn_fwd's out for one block of keys): bf16, 8-byte aligned
 *             (modes 0, 1), or fp32, 16-byte aligned (modes 2, 3: attn_fwd_ex with out_fp32)
 *   part_lse  device, fp32 [rows] (attn_fwd's lse for the same block)
 *   out       device, bf16 [rows, d], 8-byte aligned, or NULL: when given, the merged rows are
 *             also written here rounded to bf16 (it may be part_out itself)
 *   rows      1 .. 2^33; d in {64, 128}
 *   mode      0: the accumulator is set to the partial; 1: the partial is merged into it;
 *             2, 3: the same with an fp32 partial (no bf16 rounding before the merge)
 * Errors as attn_fwd; nothing is allocated and nothing synchronises.
 */
int attn_merge(float* acc_out, float* acc_lse, const void* part_out, const float* part_lse, void* out,
               int64_t rows, int64_t d, int mode, cudaStream_t stream);
/* Human-readable name of an attn_status value (static string, never NULL). */
const char* attn_status_string(int status);

/*
 * attn_debug_error: synchronise `stream`, read and clear the device error word of the
 * current device. Returns ATTN_OK if no device wait gave up since the last call,
 * ATTN_ERR_TIMEOUT if one did (the raw code, which names the waiting role, goes to
 * *device_code when device_code is not NULL), ATTN_ERR_RANGE if a V value beyond the
 * fp16 range met the fp16 P V product, ATTN_ERR_CUDA if the synchronisation itself
 * failed. The error word is one per device, shared by every stream and every forward
 * launch on it (attn_fwd, attn_fwd_fp8, the host-buffer calls): it keeps the first code
 * any of them records until a call of this function clears it, and this function waits
 * only for `stream`. With launches on several streams, synchronise them all before
 * reading it, or a code may be seen (and cleared) by the call for another stream.
 */
int attn_debug_error(cudaStream_t stream, int* device_code);

/* Number of persistent work items a launch with these sizes schedules (host-only
   helper for tests and tools; returns -1 on invalid sizes). */
int64_t attn_fwd_num_work_items(int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t d,
                                int mask_kind, int64_t window);

/*
 * attn_bwd: enqueue the backward pass on `stream`: the gradients of sum(dout * out)
 * with respect to q, k and v for the forward above (same masks, head map and scale).
 * With S = scale q k^T (masked entries -inf) and P = exp(S - lse) per query row, the
 * chain rule gives dV = P^T dO, dP = dO V^T, dS = P (dP - D) with D_i = dO_i . O_i,
 * dQ = scale dS K and dK = scale dS^T Q; a KV head's dK, dV sum over the query heads
 * that read it. The pages name a recompute-based backward pass as part of the
 * production kernel line ("Efficient attention: long context and sub-quadratic
 * variants", stanleyjacob.dev, section "Against the real libraries"); P is recomputed
 * from lse, never stored.
 *
 *   q, k, v    as attn_fwd (bf16, contiguous, 16-byte aligned)
 *   out, lse   attn_fwd's outputs for these q, k, v, scale and mask (read only)
 *   dout       device pointer, bf16, [B, Hq, N, d], contiguous, 16-byte aligned
 *   dq         device pointer, bf16, [B, Hq,  N, d], 16-byte aligned; fully overwritten
 *   dk, dv     device pointers, bf16, [B, Hkv, N, d], 16-byte aligned; fully overwritten
 *   workspace  device pointer owned by the caller; attn_bwd_workspace_bytes(B, Hq, N) bytes,
 *              16-byte aligned, always suffice. The minimum: on the two-kernel path (d = 64,
 *              Hq != Hkv, or bwd_deterministic) 4 B Hq N bytes, 4-byte aligned, holding D
 *              (fp32 [B, Hq, N]); on the fused path the full size, 16-byte aligned: D, then (from
 *              the next 256-byte boundary) an fp32 [B, Hq, N, 128] dQ accumulator that the
 *              call zeroes and fills. Not to be reused until the stream has passed the call.
 *   B, Hq, Hkv, N, d, scale, mask_kind, window, stream: as attn_fwd
 *
 * Launches: D, then for d = 128 with Hq == Hkv a fused kernel that forms P and dS once
 * per (query, key) pair (one CTA per 128-key tile: dK, dV in TMEM; dQ's partial sums of
 * each tile added into the accumulator with fp32 global reductions) and a kernel rounding
 * dQ to bf16; otherwise (d = 64, grouped heads) a query-tile kernel for dQ and a key-tile
 * kernel for dK, dV. On the fused path the order of the fp32 additions into dQ varies
 * from run to run, so dq is reproducible only up to the rounding of those sums (dk and dv
 * are bitwise reproducible); attn_bwd_ex with bwd_deterministic = 1 takes the two-kernel
 * path there too.
 *
 * The library allocates nothing. Outputs and the workspace must not overlap each other
 * or the inputs (ATTN_ERR_INVALID_ARG). Errors and bounded waits as attn_fwd; a wait
 * that gives up leaves a code that attn_bwd_debug_error returns as ATTN_ERR_TIMEOUT.
 */
int attn_bwd(const void* q, const void* k, const void* v, const void* out, const float* lse,
             const void* dout, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
             int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t d,
             float scale, int mask_kind, int64_t window, cudaStream_t stream);

/* attn_bwd with options (wait bound and CTA count as for attn_fwd_ex, bwd_deterministic and
   sinks; the other fields are ignored); opts may be NULL. */
int attn_bwd_ex(const void* q, const void* k, const void* v, const void* out, const float* lse,
                const void* dout, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t d,
                float scale, int mask_kind, int64_t window, cudaStream_t stream,
                const attn_fwd_options* opts);

/* Workspace bytes attn_bwd needs for any supported d: 4 B Hq N rounded up to 256, plus
   4 B Hq N 128 (the d = 128 dQ accumulator); 0 for invalid sizes or a total beyond 2^61. */
size_t attn_bwd_workspace_bytes(int64_t B, int64_t Hq, int64_t N);

/* Workspace bytes attn_bwd_ex needs with the sliding window and sinks > 0, 16-byte aligned (0 for
   invalid sizes): attn_bwd_workspace_bytes (with Hq != Hkv 4 B Hq N bytes, all that those calls
   take) and room for the fp32 partial sums of the key tiles that hold sinks, whose queries are cut
   into parts. That room, the difference to the size with sinks = 0, lies behind what the call takes
   without sinks, rounded up to 256 bytes: 4 B Hq N bytes also with d = 64 or bwd_deterministic. A
   workspace too small for the path taken is refused. dk and dv stay bitwise reproducible: the parts are added in a fixed order. */
size_t attn_bwd_sink_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t d, int64_t window,
                                     int64_t sinks);

/* attn_debug_error for the backward kernels' error word (same contract). */
int attn_bwd_debug_error(cudaStream_t stream, int* device_code);
/*
 * attn_decode: enqueue one decoding step on `stream`: the Nq new tokens of each of B
 * sequences attend to that sequence's cached keys and values, which are stored in
 * fixed-size pages reached through a per-sequence page table ("Efficient attention:
 * long context and sub-quadratic variants", stanleyjacob.dev, section "FlashAttention:
 * exact attention, IO-aware", PagedAttention paragraph; "Efficient Attention",
 * giftedprocrastinator.com, section "What it does": the KV cache keeps past keys and
 * values so a new token does not recompute them). Nothing is approximated: the result is
 * the masked softmax attention of attn_fwd for the new tokens' rows.
 *
 * With L_b = seq_lens[b] cached positions (the new tokens included), new token t of
 * sequence b is at position L_b - Nq + t and sees cached positions j with
 *   ATTN_MASK_FULL            0 <= j < L_b;
 *   ATTN_MASK_CAUSAL          j <= L_b - Nq + t;
 *   ATTN_MASK_SLIDING_WINDOW  L_b - Nq + t - window < j <= L_b - Nq + t.
 * Position j of sequence b lives in physical page block_table[b][j / page_size], slot
 * j % page_size. Only pages holding positions from lo_b = max(0, L_b - Nq - window + 1)
 * (0 without a window) to L_b - 1 are looked up or read: under a sliding window a caller
 * may recycle older pages and leave their table entries stale (a rolling window buffer);
 * slots past L_b in the last page may hold anything.
 *
 *   q            device, bf16, [B, Hq, Nq, d], contiguous, 16-byte aligned
 *   k_cache      device, bf16, [num_pages, Hkv, page_size, d], contiguous, 16-byte aligned
 *   v_cache      device, bf16, same shape as k_cache
 *   block_table  device, int32, [B, max_pages_per_seq], 4-byte aligned
 *   seq_lens     device, int32, [B], 4-byte aligned; Nq <= seq_lens[b] <= max_pages_per_seq *
 *                page_size (violations are reported by attn_decode_debug_error as
 *                ATTN_ERR_INVALID_ARG and leave those rows zero with lse = -inf)
 *   out          device, bf16, [B, Hq, Nq, d], 16-byte aligned; fully overwritten
 *   lse          device, fp32, [B, Hq, Nq], 4-byte aligned; natural-log normaliser of each row
 *   workspace    device, 16-byte aligned, at least attn_decode_workspace_bytes(B, Hq, Nq, d,
 *                num_splits) bytes, owned by the caller. Its first 256 bytes hold the counter
 *                that hands work items to the SMs: they must be zero before the first call that
 *                uses the workspace, and every call leaves them zero again. The rest holds the
 *                splits' partial results until the merge launch of the same call has read them.
 *                Calls that share a workspace must not run concurrently.
 *   Hq % Hkv == 0; query head h reads KV head h / (Hq / Hkv); d in {64, 128};
 *   page_size in {16, 32, 64, 128, 256}
 *   num_splits   1..4096: each sequence's visible key range is cut into this many parts
 *                processed in parallel and merged by their log-sum-exp
 *                (attn_decode_num_splits suggests one)
 *   scale, mask_kind, window, stream: as attn_fwd
 *
 * Ownership: the caller owns every buffer; the library allocates nothing and never
 * synchronises. Outputs and the workspace must not overlap each other or the inputs
 * (ATTN_ERR_INVALID_ARG). A page-table entry outside [0, num_pages) that the step needs
 * is reported by attn_decode_debug_error as ATTN_ERR_INVALID_ARG (the step's result is
 * then undefined, but nothing outside the given buffers is read). Precision: scores, sums
 * and the split partials are fp32; P goes to the P V product rounded to bf16 (RNE), so,
 * unlike attn_fwd, a row dominated by a few keys can be off by about one bf16 ulp of out
 * (the step is bound by HBM reads, and an fp16 copy of V in shared memory would hold each
 * V slot of the load ring longer, costing 15-40 % of the bandwidth). Any bf16 V is taken.
 * Errors, bounded waits and ATTN_ERR_TIMEOUT as attn_fwd.
 */
int attn_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                const int32_t* seq_lens, void* out, float* lse, void* workspace, size_t workspace_bytes,
                int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t d,
                int64_t num_pages, int64_t page_size, int64_t max_pages_per_seq, int64_t num_splits,
                float scale, int mask_kind, int64_t window, cudaStream_t stream);
/* attn_decode with options (wait bound and CTA count as for attn_fwd_ex, and sinks; the
   other fields are ignored); opts may be NULL. */
int attn_decode_ex(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                   const int32_t* seq_lens, void* out, float* lse, void* workspace, size_t workspace_bytes,
                   int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t d,
                   int64_t num_pages, int64_t page_size, int64_t max_pages_per_seq, int64_t num_splits,
                   float scale, int mask_kind, int64_t window, cudaStream_t stream,
                   const attn_fwd_options* opts);
/* Workspace bytes attn_decode needs for num_splits (256 + the partial results when
   num_splits > 1; 0 on invalid sizes). */
size_t attn_decode_workspace_bytes(int64_t B, int64_t Hq, int64_t Nq, int64_t d, int64_t num_splits);
/* Suggested num_splits for a step whose longest sequence has max_seq_len cached positions,
   on the current device: one wave of work items when B * Hkv (times the query-row chunks)
   is below the SM count, otherwise splits of at most 64 128-key tiles; never a split
   shorter than four tiles; -1 on invalid sizes. Host-only. */
int64_t attn_decode_num_splits(int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t max_seq_len,
                               int mask_kind, int64_t window);
/* attn_debug_error for the decoding kernel's error word (one per device, shared like the
   forward's): ATTN_ERR_TIMEOUT for a wait that gave up, ATTN_ERR_INVALID_ARG for a bad
   sequence length or page-table entry. */
int attn_decode_debug_error(cudaStream_t stream, int* device_code);

/*
 * attn_decode_static: attn_decode without a caller workspace, for callers that cannot
 * allocate device memory. (The pages have no counterpart: this is a deployment variant
 * of the decoding step above, with the same result.)
 *
 * Who needs it: code that runs inside a host program which owns all device memory and
 * hands the code only its input and output buffers -- an inference-server plugin, an
 * embedded runtime with a fixed memory plan, a language binding without a device
 * allocator. There a cudaMalloc is either not permitted, breaks the owner's memory plan,
 * or synchronises the device at a moment the caller does not control.
 *
 * Instead of `workspace`, the call uses a scratch array that the library itself defines
 * in device memory: ATTN_DECODE_STATIC_SCRATCH_BYTES bytes, held by every GPU that loads
 * the library until the process exits. Nothing is allocated by the call: no cudaMalloc,
 * no cudaFree, no allocating library routine.
 *
 *   arguments    those of attn_decode without workspace and workspace_bytes, with the
 *                same meaning, layouts, checks and errors
 *   size limit   attn_decode_workspace_bytes(B, Hq, Nq, d, num_splits) must not exceed
 *                ATTN_DECODE_STATIC_SCRATCH_BYTES; a larger step is refused with
 *                ATTN_ERR_UNSUPPORTED before anything is enqueued (use fewer splits, a
 *                smaller batch, or attn_decode with a workspace)
 *
 * Set-up: the first call on a device, with that device current, looks up the device
 * address of the array (once per device); make that first call before any stream capture.
 * Every call then enqueues, on `stream`, a clear of the array's work counter followed by
 * the decoding launches. If attn_decode's argument checks then refuse the call, that
 * clear, which touches only the library's own array, may already be enqueued.
 * Every call on a device shares the one array, and the array keeps the last call's
 * partial results: calls that overlap on the GPU (other streams, other host threads)
 * race on it and give wrong results. Order them, e.g. on one stream.
 */
#define ATTN_DECODE_STATIC_SCRATCH_BYTES (8u * 1024u * 1024u)
int attn_decode_static(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                       const int32_t* seq_lens, void* out, float* lse,
                       int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t d,
                       int64_t num_pages, int64_t page_size, int64_t max_pages_per_seq, int64_t num_splits,
                       float scale, int mask_kind, int64_t window, cudaStream_t stream);

/*
 * attn_kv_append: enqueue the write side of the paged cache on `stream`: the keys and values
 * of new tokens go into their sequences' pages, the keys rotated by their positions on the
 * way; the queries of the same tokens are rotated too and written where attn_decode (or
 * attn_decode_kv8) reads them. (The pages name the cache and its pages, see attn_decode;
 * how the cache is filled is not on them.)
 *
 * Rotation (rotary positions): with x the token's position and f_i = inv_freq[i], the pair
 * (a, b) number i of a head's row becomes (a cos(x f_i) - b sin(x f_i), b cos(x f_i) + a sin(x f_i)).
 * Pair i is elements (i, i + rot_dim / 2), or (2i, 2i + 1) with `interleaved`; elements from
 * rot_dim on are copied. Angles are formed in fp64, the rotation is fp32, rounded once.
 *
 * Tokens are rows of q, k and v, sequence after sequence. With cu_tokens NULL every one of
 * the B sequences has T / B rows; otherwise sequence b has rows cu_tokens[b] .. cu_tokens[b + 1]
 * - 1 (none is fine), and rows from cu_tokens[B] on are not read. seq_lens counts the new
 * tokens in, as in attn_decode: with n_b new tokens, they take positions seq_lens[b] - n_b ..
 * seq_lens[b] - 1. Only the table entries of the pages they fall into are read, only their
 * slots are written: every other slot of the cache keeps its bytes.
 *
 * 8-bit cache (scale_block != 0): slots hold E4M3 codes, and k_scale, v_scale
 * [num_pages, Hkv, page_size / scale_block] hold one scale for each block of scale_block
 * slots of a head: value = E4M3(code) * scale. A scale is the smallest power of two s >= 2^-40
 * with amax <= 448 s over the block's new tokens (finite values; infinities become +-448 s,
 * NaN stays NaN), and a code is x / s rounded to nearest even. A block that held tokens of the
 * sequence before this call keeps its scale where its new tokens fit (amax <= 448 s);
 * otherwise it takes theirs, and its older codes are rounded again under it (which changes
 * their values only where they turn subnormal). (Values from 448 * 2^60 on, some 5e20, get scales that
 * attn_decode_kv8 no longer takes.)
 *
 * Fields of the argument block (zero-initialise, then set what is needed):
 *   k, v          device, bf16, T rows of [Hkv, d]; k_stride, v_stride elements from row to row
 *                 (at least Hkv * d, a multiple of 8), 16-byte aligned: views of one projection's
 *                 output will do
 *   q, q_stride   device, bf16, T rows of [Hq, d], likewise; NULL: no queries
 *   q_out         device, bf16, 16-byte aligned: [B, Hq, T / B, d] without cu_tokens, [T, Hq, d]
 *                 with it; NULL exactly where q is
 *   k_cache, v_cache  device, bf16 or E4M3 codes, [num_pages, Hkv, page_size, d], 16-byte aligned
 *   k_scale, v_scale  device, fp32, as above; NULL exactly where scale_block is 0
 *   block_table   device, int32, [B, max_pages_per_seq]
 *   seq_lens      device, int32, [B]; n_b <= seq_lens[b] <= max_pages_per_seq * page_size, or 0 (idle)
 *   cu_tokens     device, int32, [B + 1], or NULL (T % B == 0)
 *   positions     device, int32, [T]: the rotation's positions; NULL: the cache's positions
 *   inv_freq      device, fp32, [rot_dim / 2]; NULL exactly where rot_dim is 0 (no rotation)
 *   rot_dim       0 .. d, a multiple of 16;  d in {64, 128};  page_size in {16, 32, 64, 128, 256}
 *   scale_block   0 (bf16 cache) or a power of two <= page_size
 *
 * Without cu_tokens seq_lens[b] == 0 marks an idle slot of a padded batch, as in attn_decode_kv8: its
 * rows of q, k and v and its table are not read, nothing is cached, its rows of q_out are zeros,
 * no error. (With cu_tokens an idle slot has no rows.)
 *
 * A sequence whose length or row range is unusable is skipped, as are the cache rows of a page
 * entry outside [0, num_pages); both are reported by attn_kv_append_debug_error as
 * ATTN_ERR_INVALID_ARG. Two sequences of one call must not name the same page for new tokens.
 * What is written must not overlap anything else (ATTN_ERR_INVALID_ARG). One launch; nothing
 * is allocated and nothing synchronises; the result does not depend on any order of execution.
 */
typedef struct {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;
  void* q_out;
  void* k_cache;
  void* v_cache;
  float* k_scale;
  float* v_scale;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* cu_tokens;
  const int32_t* positions;
  const float* inv_freq;
  int64_t B, T, Hq, Hkv, d, rot_dim, num_pages, page_size, max_pages_per_seq, scale_block;
  int interleaved;
} attn_kv_append_args;
int attn_kv_append(const attn_kv_append_args* args, cudaStream_t stream);
/* attn_debug_error for the append's error word (one per device, shared like the forward's):
   ATTN_ERR_INVALID_ARG for an unusable sequence or page-table entry. */
int attn_kv_append_debug_error(cudaStream_t stream, int* device_code);

/*
 * attn_decode_kv8: attn_decode over a cache held in 8 bits (as attn_kv_append writes it, or
 * any E4M3 codes with scales). Cached values are E4M3(code) * scale, one scale for each block
 * of scale_block slots of a page and head; the result is the exact masked softmax attention
 * of those values for the bf16 queries. Half the bytes of the bf16 cache are read.
 *
 *   q, block_table, seq_lens, out, lse, num_splits, scale, window, stream: as attn_decode, and
 *                     seq_lens[b] == 0 marks an idle slot of a padded batch: out 0, lse -inf,
 *                     nothing of its table read, no error
 *   k_cache, v_cache  device, E4M3 codes, [num_pages, Hkv, page_size, d], contiguous, 16-byte aligned
 *   k_scale, v_scale  device, fp32, [num_pages, Hkv, page_size / scale_block], contiguous, 4-byte
 *                     aligned; finite. V scales are meant to lie in [2^-40, 2^60]: one outside is
 *                     taken as the nearest bound
 *   scale_block       a power of two, at most page_size
 *   mask_kind         as attn_decode
 *   sinks             with ATTN_MASK_SLIDING_WINDOW: the first `sinks` positions stay visible
 *                     (j < sinks, j <= the row's position) beside the window; 0 = none. Pages
 *                     between the sinks and the oldest window position are neither looked up nor
 *                     read. Must be 0 with the other masks
 *   workspace         device, 16-byte aligned, attn_decode_kv8_workspace_bytes(B, Hq, Hkv, Nq, d,
 *                     num_splits) bytes, with the contract of attn_decode's (first 256 bytes zero
 *                     before the first call and after each; not shared by concurrent calls)
 *   opts              wait bound and CTA count as for attn_fwd_ex; inject_stall = n > 0: the loaders of a
 *                     CTA stop before its n-th tile of 128 positions (test hook: waits run out and the call
 *                     ends with ATTN_ERR_TIMEOUT pending, its outputs undefined); may be NULL
 *
 * Precision: the products take the codes exactly; a bf16 query row is split into two E4M3
 * terms (exact to 2^-17 of the row's largest element); scores, statistics and sums are fp32;
 * the weights that the product with V takes, w = softmax weight * V scale, are sums of three
 * E5M2 numbers: off by at most (2^-9 + 2^-11) w + 2^-29 M, with M the row's largest w (bf16's
 * rounding is 2^-8 w; a w below 2^-29 M is lost there, and only there: the weights' sum has it).
 * Ownership, checks, overlap rules, bounded waits and errors as attn_decode.
 */
int attn_decode_kv8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                    const float* v_scale, const int32_t* block_table, const int32_t* seq_lens, void* out, float* lse,
                    void* workspace, size_t workspace_bytes, int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq,
                    int64_t d, int64_t num_pages, int64_t page_size, int64_t max_pages_per_seq, int64_t scale_block,
                    int64_t num_splits, float scale, int mask_kind, int64_t window, int64_t sinks,
                    cudaStream_t stream, const attn_fwd_options* opts);
/* Workspace bytes attn_decode_kv8 needs (0 on invalid sizes). */
size_t attn_decode_kv8_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t d, int64_t num_splits);
/* Suggested num_splits, as attn_decode_num_splits (-1 on invalid sizes). Host-only. */
int64_t attn_decode_kv8_num_splits(int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t max_seq_len, int mask_kind,
                                   int64_t window, int64_t sinks);
/* attn_decode_debug_error for the 8-bit decoding kernel's error word. */
int attn_decode_kv8_debug_error(cudaStream_t stream, int* device_code);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_B200_ATTN_H_ */
