/*
 * sb.h -- C ABI of libsb: the LM-head contraction logits = H·Wᵀ over a vocabulary split
 * into k contiguous lane shards, fused on one GPU (sm_103a) with the consumer-surface
 * projection, so that only the surface the consumer asked for leaves the kernel.
 *
 * Source of the operation -- "SemBridge: Compiling Consumer Observations into
 * Cross-Stack Communication Plans" (Chen, Zhu, Lin):
 *   - Section 5.2 (Data, Result, and Control Paths): the tail output head materialises
 *     full logits; a complete-logits or log-probability request slices them by TP lane
 *     and rebuilds the full value; a token-only request applies the deterministic
 *     sampler to the same tensor and sends int32 IDs.
 *   - Section 2.2 (Consumer Surfaces and Delivery Obligations): the consumer surfaces are
 *     complete logits, log-probabilities, token IDs or another registered projection.
 *   - Section 3.1 (Boundary Contract): the registered projection operator names its
 *     input/output types and deterministic tie-breaking (here: the lowest global
 *     vocabulary index wins a tie).
 *   - Figure 1: full-logit transfer and source projection expose the same token; they
 *     differ only in where argmax runs.  Here argmax runs inside the GEMM epilogue.
 *   - Section 5.2 also notes the transport reserves no persistent device-buffer pool;
 *     likewise this library allocates no device memory: the caller owns every buffer.
 *
 * Conventions for every entry point:
 *   - Pointers named "device" must point to device memory of the current CUDA device
 *     and be 16-byte aligned; sizes are element counts unless named *_bytes.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default stream).
 *     All device work is enqueued asynchronously on it; nothing synchronises.
 *   - The return value is an sb_status.  It covers argument validation and launch
 *     errors only; when it is not SB_OK nothing was enqueued.  Errors found on the
 *     device (a bounded wait that ran out) are recorded in the workspace status word
 *     and read with sb_last_device_status() after the caller synchronises.
 *   - There is no CPU fallback: a device that is not sm_103 returns SB_ERR_UNSUPPORTED.
 *   - Calls that share a workspace must not overlap on the GPU (they would race on it).
 *   - The calls enqueue kernels only (no host synchronisation), so they can be captured in
 *     a CUDA graph; arguments are checked and tensor maps encoded at capture time.  Every
 *     replay then carries the captured call's launch epoch, so after replays
 *     sb_last_device_status reports the worst device status since the capture.
 */
#ifndef SB_H
#define SB_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Consumer surface (Section 2.2).  Every surface produces the token; the surface
 * decides which other outputs are mandatory and whether logits are written. */
typedef enum sb_surface {
    SB_TOKEN = 0,        /* deterministic argmax token (int32, lowest index on ties)      */
    SB_TOKEN_LOGPROB = 1,/* token + its natural-log log-probability over the full vocab   */
    SB_FULL_LOGITS = 2,  /* token + bf16 logits [M, V] in shard-to-full (global) layout    */
    SB_GUMBEL_TOKEN = 3, /* counter-based Gumbel-max sample from softmax(z / T) + log-prob */
    SB_TOPK_LOGPROB = 4  /* token + the K most likely tokens and their log-probabilities   */
} sb_surface;

/* Largest K of the SB_TOPK_LOGPROB surface. */
#define SB_MAX_TOPK 16

/* Layout flag OR'ed into the `surface` argument of the calls that read W (sb_lmhead_project,
 * sb_lmhead_records, sb_lmhead_project_from_host, sb_host_step_create,
 * sb_lmhead_project_static_scratch): W points to the packed copy written by
 * sb_pack_weights for the same V, d and k instead of the row-major [V, d] matrix.  The
 * results are bit for bit those of the row-major call (the same operands reach the same
 * MMAs); only the memory layout of W, and so how fast it streams, differs.
 * sb_workspace_bytes ignores the flag; the other calls reject it. */
#define SB_W_PACKED 0x100

typedef enum sb_status {
    SB_OK = 0,
    SB_ERR_INVALID_ARG = 1,          /* a size, enum, pointer or temperature is out of range */
    SB_ERR_UNSUPPORTED = 2,          /* the current device is not an sm_103 GPU               */
    SB_ERR_ALIGNMENT = 3,            /* a pointer is not 16-byte aligned, or d % 8 != 0       */
    SB_ERR_WORKSPACE_TOO_SMALL = 4,  /* workspace_bytes < sb_workspace_bytes(...)             */
    SB_ERR_CUDA = 5,                 /* a CUDA runtime or driver call failed                  */
    SB_ERR_DEVICE_TIMEOUT = 6        /* device side: a bounded wait gave up (after sync)      */
} sb_status;

/*
 * Output buffers of one projection call.  All pointers are device pointers owned by the
 * caller; NULL means "not requested".  Every surface fills every non-NULL output.
 *   token           int32 [M]      required for every surface.
 *   token_logprob   float [M]      log p(token); required for SB_TOKEN_LOGPROB and
 *                                  SB_GUMBEL_TOKEN.  For SB_GUMBEL_TOKEN the distribution
 *                                  is softmax(z / T), the one sampled from.
 *   lse             float [M]      natural-log logsumexp of z (of z / T for SB_GUMBEL_TOKEN).
 *   logits_bf16     uint16 [M*V]   bf16 bit patterns of z, row-major [M][V], column = the
 *                                  global vocabulary index (lane shard s holds columns
 *                                  [s*V/k, (s+1)*V/k)); required iff SB_FULL_LOGITS and
 *                                  written only then.
 *   target_ids      int32 [M]      optional scoring targets, each in [0, V).  Values out of
 *                                  range are found on the device: sb_last_device_status
 *                                  then reports SB_ERR_INVALID_ARG and the outputs are
 *                                  undefined.
 *   target_logprob  float [M]      log p(target_ids[r]); required iff target_ids != NULL.
 *   workspace       bytes          scratch of at least sb_workspace_bytes(M, V, k, surface)
 *                                  bytes, 256-byte aligned; holds the per-tile records, the
 *                                  target logits and the device status word.  Its contents
 *                                  need no initialisation.
 *   topk_ids        int32 [M*K]    SB_TOPK_LOGPROB: per row the K columns with the largest
 *                                  logits, largest first, equal logits by ascending column.
 *   topk_logprob    float [M*K]    SB_TOPK_LOGPROB: their log-probabilities z_j - lse.
 *   topk            K              SB_TOPK_LOGPROB: 1 <= K <= min(SB_MAX_TOPK, V); ignored by
 *                                  the other surfaces (as are the two arrays above).
 */
typedef struct sb_outputs {
    int32_t *token;
    float *token_logprob;
    float *lse;
    uint16_t *logits_bf16;
    const int32_t *target_ids;
    float *target_logprob;
    void *workspace;
    size_t workspace_bytes;
    int32_t *topk_ids;
    float *topk_logprob;
    int32_t topk;
} sb_outputs;

/*
 * Workspace layout (byte offsets from `workspace`; n = M * k * T with T =
 * sb_tiles_per_shard(M, V, k); each array starts on a 256-byte boundary, in this order):
 *   [0, 256)      header: uint32 epoch of the last launch, uint32 (internal use),
 *                 uint64 status word = (epoch << 32) | sb_status of that launch
 *   float   m[n]     per-tile record: max of y over the tile's columns
 *   int32   idx[n]   lowest global column attaining m
 *   float   s[n]     sum over the tile of exp(y - m)
 *   float   gkey[n]  SB_GUMBEL_TOKEN only: max of y + g over the tile
 *   int32   gidx[n]  SB_GUMBEL_TOKEN only: lowest column attaining gkey
 *   float   gz[n]    SB_GUMBEL_TOKEN only: z at gidx
 *   float   tkv[n][K] SB_TOPK_LOGPROB only: the tile's K largest logits, largest first
 *   int32   tki[n][K] SB_TOPK_LOGPROB only: their columns (INT32_MAX marks an empty slot)
 *   float   tz[M]    z at target_ids[r] (written only when targets are given)
 * Record (r, s, t) sits at index (r * k + s) * T + t and covers the global columns
 * [s*S + 128t, min(s*S + 128(t+1), (s+1)*S)) with S = V/k and T = ceil(S / 128).  y is z,
 * or z * (1/T) for SB_GUMBEL_TOKEN with 1/T rounded to fp32 on the host; g is the Gumbel
 * noise of sb_lmhead_project.
 */

/* Bytes of workspace one call needs (for SB_TOPK_LOGPROB: with K = SB_MAX_TOPK, enough for
 * every K); 0 if the arguments are invalid. */
size_t sb_workspace_bytes(int64_t M, int64_t V, int32_t k, int32_t surface);

/*
 * The packed layout of W for the calls with SB_W_PACKED: every (128-row tile, 64-column K
 * block) box the kernels read is one contiguous 16 KB block, so each box is one linear
 * stream of HBM reads instead of 128 rows of 128 bytes, 2d bytes apart.  With S = V/k,
 * T128 = ceil(S / 128) tiles per shard and KB = ceil(d / 64) K blocks, element (r, c) of W
 * (row r of shard s = r / S, i = (r - s*S) mod 128 in tile t = (r - s*S) / 128; column c in
 * K block kb = c / 64 at j = c mod 64) is bf16 number
 *     (((s * T128 + t) * KB + kb) * 128 + i) * 64 + j
 * of the packed buffer; the rows past a shard's end in its last tile and the columns past d
 * in the last K block are zero.  A weight is packed once (it is a model parameter) and then
 * read by every call.
 */
/* Bytes of the packed copy of a [V, d] W for k lane shards: k * T128 * KB * 16384; 0 if the
 * arguments are invalid (the same shape rules as sb_lmhead_project, d % 8 == 0). */
size_t sb_packed_weight_bytes(int64_t V, int64_t d, int32_t k);
/* Writes the packed copy of the row-major W [V, d] (device, bf16, 16-byte aligned) into
 * W_packed (device, 16-byte aligned, `bytes` >= sb_packed_weight_bytes), enqueued on
 * `stream`.  SB_ERR_WORKSPACE_TOO_SMALL if `bytes` is short, SB_ERR_ALIGNMENT for a
 * misaligned pointer or d % 8 != 0. */
int32_t sb_pack_weights(const void *W, int64_t V, int64_t d, int32_t k, void *W_packed,
                        size_t bytes, void *stream);

/* Records per (row, lane shard): T = ceil((V / k) / 128), one per 128 vocabulary columns;
 * -1 if the arguments are invalid.  (M is accepted for symmetry and does not change T.) */
int32_t sb_tiles_per_shard(int64_t M, int64_t V, int32_t k);

/*
 * One projection call: logits z = H·Wᵀ (fp32 accumulation on the tensor cores, no bias,
 * scale or soft-cap), projected per Section 5.2 onto `surface`, in two kernels enqueued on
 * `stream` -- the fused GEMM + record epilogue, then the record combine
 * (sb_combine_shard_records) -- with no host synchronisation.
 *   H          device bf16 [M, d] row-major (K-major), 16-byte aligned.
 *   W          device bf16 [V, d] row-major (the output-head weight), 16-byte aligned; or,
 *              with SB_W_PACKED in `surface`, its packed copy (sb_pack_weights, same k).
 *   M, d, V    M >= 1, d >= 8 with d % 8 == 0, V >= 1.
 *   k          number of contiguous lane shards, 1 <= k <= 1024 and V % k == 0.
 *   surface    an sb_surface, optionally OR'ed with SB_W_PACKED.
 *   temperature  SB_GUMBEL_TOKEN: finite and > 0 (the key is z * (1/T) + g); ignored
 *              otherwise.
 *   seed       SB_GUMBEL_TOKEN: the SplitMix64 stream seed.  Column j of row r draws the
 *              output at stream index n = r*V + j, i.e. the SplitMix64 finaliser of
 *              seed + (n + 1) * 0x9E3779B97F4A7C15; u = (x >> 40) * 2^-24 and
 *              g = -log(-log u) in fp32 to within 2e-6 absolute (u = 0 gives g = -inf).
 *              Ignored otherwise.
 *   out        outputs and workspace (see sb_outputs); read on the host during the call.
 * The GEMM is a programmatic dependent launch that starts loading W before the preceding
 * kernel in the stream has finished, so W must not be written by a kernel that can still be
 * running then (one that signals its dependents early); H, the targets and the workspace are
 * read only after that kernel has finished.
 * Returns SB_OK, or an error with nothing enqueued.
 */
int32_t sb_lmhead_project(const void *H, const void *W, int64_t M, int64_t d, int64_t V,
                          int32_t k, int32_t surface, float temperature, uint64_t seed,
                          const sb_outputs *out, void *stream);

/*
 * The first kernel of sb_lmhead_project alone: the fused GEMM + record epilogue, which
 * writes the per-tile records (and the target logits) into out->workspace and, for
 * SB_FULL_LOGITS, the bf16 logits; token, log-prob and lse outputs are left unwritten.
 * Same arguments, validation and return values as sb_lmhead_project.  It is the step a
 * vocabulary-sharded caller runs before exchanging records (Section 5.2: each TP lane
 * projects its own shard) and then finishing with sb_combine_shard_records.
 */
int32_t sb_lmhead_records(const void *H, const void *W, int64_t M, int64_t d, int64_t V,
                          int32_t k, int32_t surface, float temperature, uint64_t seed,
                          const sb_outputs *out, void *stream);

/*
 * sb_lmhead_project for a caller whose hidden states are in host memory and who wants the
 * token surface back in host memory ("SemBridge", Section 5.2: the consumer observes the
 * projected surface, never the logits).  Enqueues on stream, in order: H_host into H_dev,
 * the projection of sb_lmhead_project on H_dev, and the token (and, when
 * token_logprob_host is not NULL, the chosen log-probability) into the host buffers; the
 * device outputs in out are written as well.
 * Host buffers the device can address (pinned memory from cudaHostAlloc or
 * cudaHostRegister, mapped under unified addressing) are moved by the kernels themselves:
 * a copy kernel reads H_host and the combine writes the host results directly, with no
 * copy-engine operations.  Other host memory (pageable) is moved with cudaMemcpyAsync
 * (synchronous with respect to the host for pageable memory).
 *   H_host              host bf16 [M, d].
 *   H_dev               device staging buffer of M * d bf16, 16-byte aligned; overwritten
 *                       once the previous kernel in the stream has finished.
 *   out                 device outputs and workspace as for sb_lmhead_project.
 *   token_host          host int32 [M] (required); token_logprob_host host float [M] or NULL
 *                       (then out->token_logprob may be NULL).
 * On the copy path, when out->token_logprob directly follows out->token (M int32) and
 * token_logprob_host directly follows token_host, both come back in one copy.  The caller
 * synchronises stream before reading the host outputs.  Every argument is checked before
 * anything is enqueued; returns an sb_status.
 */
int32_t sb_lmhead_project_from_host(const void *H_host, void *H_dev, const void *W, int64_t M,
                                    int64_t d, int64_t V, int32_t k, int32_t surface,
                                    float temperature, uint64_t seed, const sb_outputs *out,
                                    int32_t *token_host, float *token_logprob_host,
                                    void *stream);

/*
 * The host-buffer call of a serving loop, captured once: sb_host_step_create checks the
 * arguments as sb_lmhead_project_from_host does and records that call (the copy kernel
 * reading H_host, the projection, the combine storing into the host buffers) into a CUDA
 * graph; sb_host_step_launch enqueues one replay on `stream` (one graph launch, about a
 * quarter of the host-side time of the plain call); sb_host_step_destroy releases it.
 * Every buffer is bound at creation: each replay reads the current contents of H_host and
 * overwrites token_host / token_logprob_host and the device outputs of `out`.
 *   H_host, token_host, token_logprob_host  host memory the device can address (pinned:
 *              cudaHostAlloc / cudaHostRegister under unified addressing); other host memory
 *              gives SB_ERR_UNSUPPORTED (use sb_lmhead_project_from_host).
 *   step       receives the handle (NULL on any error).
 * Replays reuse the launch epoch of the creation, so sb_last_device_status reports the worst
 * device status since then.  Returns an sb_status; creation enqueues nothing on any stream.
 */
typedef struct sb_host_step sb_host_step;
int32_t sb_host_step_create(const void *H_host, void *H_dev, const void *W, int64_t M,
                            int64_t d, int64_t V, int32_t k, int32_t surface,
                            float temperature, uint64_t seed, const sb_outputs *out,
                            int32_t *token_host, float *token_logprob_host,
                            sb_host_step **step);
int32_t sb_host_step_launch(sb_host_step *step, void *stream);
void sb_host_step_destroy(sb_host_step *step);

/*
 * The record combine alone (the second kernel of sb_lmhead_project): reads the per-tile
 * records of `workspace` (layout above; tiles_per_shard = T) and writes token,
 * token_logprob, lse and target_logprob of `out` (those that are non-NULL).  Per row it
 * merges the T records of each shard in a fixed tree (shard-local completion), then the k
 * shard results in ascending shard order (the cross-shard merge that replaces "AllGather
 * the logits, then argmax" of Section 5.2).  The merge of two records keeps the larger
 * max, the lower index on an equal max, and rescales the exp-sums to the new max; the
 * fixed order makes the output bits a function of the record bits alone.
 *   temperature  as for sb_lmhead_project (used by SB_GUMBEL_TOKEN and the target
 *              log-prob only).
 *   out->logits_bf16 is ignored; out->workspace must equal `workspace`.
 */
int32_t sb_combine_shard_records(const void *workspace, int64_t M, int32_t k,
                                 int32_t tiles_per_shard, int32_t surface, float temperature,
                                 const sb_outputs *out, void *stream);

/*
 * sb_lmhead_project without a caller-supplied workspace (the SemBridge paper has no
 * counterpart; this entry point exists for callers that cannot allocate device memory).
 * Some callers cannot call cudaMalloc: a plug-in inside a host engine that owns the whole
 * device-memory pool, code on a latency-critical path where cudaMalloc's implicit device
 * synchronisation is not allowed, or a foreign-function caller that links only this
 * library.  This call takes its scratch from an 8 MiB array compiled into the library
 * (every GPU that loads libsb holds it until the process exits) and allocates nothing.
 *   Arguments, outputs and return values are those of sb_lmhead_project, except that
 *   out->workspace and out->workspace_bytes are ignored.  A problem whose
 *   sb_workspace_bytes(M, V, k, surface) exceeds 8 MiB (8388608 bytes) is rejected with
 *   SB_ERR_WORKSPACE_TOO_SMALL before anything is enqueued.
 *   The first call on each device looks up the array's device address (with that device
 *   current); make that first call before any stream capture.
 *   Every call on a device shares the one array and leaves its records there; nothing in
 *   it needs clearing between calls, but calls that overlap on the GPU (different streams,
 *   or host threads without ordering) race on it and give undefined results.
 *   The device status word also lives in the array, out of the caller's reach: read it with
 *   sb_static_scratch_last_status() (not sb_last_device_status) after synchronising.  Both
 *   errors found on the device land there: a bounded wait that ran out
 *   (SB_ERR_DEVICE_TIMEOUT) and a scoring target outside [0, V) (SB_ERR_INVALID_ARG).
 */
int32_t sb_lmhead_project_static_scratch(const void *H, const void *W, int64_t M, int64_t d,
                                         int64_t V, int32_t k, int32_t surface,
                                         float temperature, uint64_t seed,
                                         const sb_outputs *out, void *stream);

/*
 * The device status of the last sb_lmhead_project_static_scratch call on the current device
 * (no paper counterpart): SB_OK, SB_ERR_DEVICE_TIMEOUT or SB_ERR_INVALID_ARG, as
 * sb_last_device_status reports for a caller's workspace; SB_ERR_CUDA if the array cannot be
 * read.  Synchronises with the device (a blocking device-to-host copy of 16 bytes into host
 * stack memory; allocates nothing).  Call it after the static-scratch call has completed and
 * before the next one is enqueued.
 */
int32_t sb_static_scratch_last_status(void);

/* Test hook: the two functions of the record merge, as the combine kernels evaluate them,
 * on count entries of device arrays (enqueued on stream): op 0 gives y[i] = e^x[i] for
 * x <= 0 (the hardware base-2 exponential of x * log2(e), the product rounded to fp32);
 * op 1 gives y[i] = ln x[i].  With these two, a host restatement of the merge order in
 * fp32 reproduces sb_combine_shard_records bit for bit. */
int32_t sb_debug_combine_math(int32_t op, const float *x, float *y, int64_t count,
                              void *stream);

/* Test hook: g[i] = the Gumbel noise the projection kernels derive from the 24-bit
 * uniform bits[i] & 0xFFFFFF (u = bits * 2^-24), for count entries of device arrays,
 * enqueued on stream. */
int32_t sb_debug_gumbel_from_bits(const uint32_t *bits, float *g, int64_t count, void *stream);

/*
 * Shard payloads: what each vocabulary lane would send to the others instead of its logit
 * slice (Figure 1 and Section 5.2: full-logit transfer ships V logit elements in k frames,
 * source projection ships the per-lane projection).  A lane's payload is its shard-local
 * completion: per row one record (m, idx, s) = (max logit, lowest global column attaining
 * it, sum of exp(z - m)) -- 12 bytes; the Gumbel surface adds (gkey, gidx, gz) -- 24 bytes.
 * The top-K surface has no payload form.
 * Layout: lane-major, record (lane s, row r) at byte (s * M + r) * record_bytes; fields are
 * float32 / int32 in that order.  Merging the k payloads in ascending lane order gives the
 * same bits as sb_combine_shard_records on the same records.
 */

/* k * M * record_bytes for the surfaces above; 0 for invalid arguments or SB_TOPK_LOGPROB. */
size_t sb_payload_bytes(int64_t M, int32_t k, int32_t surface);

/*
 * Shard-local completion of the k lanes' records in `workspace` (as left by
 * sb_lmhead_records for M, k and T = tiles_per_shard) into `payload` (device, 4-byte
 * aligned, sb_payload_bytes(M, k, surface) bytes), adding col_offset (>= 0) to every column
 * so that a caller holding only a slice of W (for example one device of a
 * vocabulary-sharded head) produces global columns.  Enqueued on stream.
 */
int32_t sb_pack_shard_records(const void *workspace, int64_t M, int32_t k,
                              int32_t tiles_per_shard, int32_t surface, int64_t col_offset,
                              void *payload, void *stream);

/*
 * Cross-lane merge of k lane payloads (device, lane-major as above): writes out->token and,
 * where non-NULL, out->token_logprob and out->lse (target log-probs are not carried by the
 * payload; out->workspace is not used).  temperature as for sb_lmhead_project.
 */
int32_t sb_merge_shard_payload(const void *payload, int64_t M, int32_t k, int32_t surface,
                               float temperature, const sb_outputs *out, void *stream);

/*
 * Row-parallel partial completion ("SemBridge", Section 6.4 and Table 3: in a row-parallel
 * MLP down projection each tensor-parallel lane owns a slice of the reduction dimension and
 * produces an incomplete full-width partial; the partials must be summed -- the completion
 * obligation of Section 3.5 -- before a consumer observes the value).
 *   Y[m][n] = sum over lanes l (ascending) of P_l[m][n],
 *   P_l[m][n] = sum over lane l's reduction columns of X[m][i] * W[n][i].
 *   X          device bf16 [M, K] row-major (activations), 16-byte aligned; 1 <= M <= 256.
 *   W          device bf16 [N, K] row-major (weights), 16-byte aligned; N >= 1.
 *   K          a multiple of 64 * lanes (each lane's slice is whole 64-column blocks).
 *   lanes      >= 1.
 *   Y          device [M, N] row-major: fp32 when y_bf16 == 0, else bf16 (round to nearest).
 *   workspace  device, 256-byte aligned, >= sb_partial_workspace_bytes(M, N, K, lanes):
 *              header (read by sb_last_device_status) and fp32 partials; no
 *              initialisation.  One call at a time per workspace.
 * The (128-feature tile, 64-column K block) work is split evenly over the SMs; each SM cuts
 * its share at lane boundaries and accumulates every piece in fp32 on the tensor cores.  A
 * second kernel (a programmatic dependent of the first) sums each tile's pieces in
 * ascending K order (lane 0's first), so the result bits do not depend on scheduling.  Two
 * kernels are enqueued on stream; returns SB_OK or an error with nothing enqueued.
 * The first kernel is a programmatic dependent launch: it starts loading W before the
 * preceding kernel in the stream has finished, so W must not be written by a kernel that
 * can still be running then (one that signals its dependents early); X and the workspace
 * are read only after that kernel has finished.
 * sb_partial_workspace_bytes depends on the shape and on the SM count of the current
 * device; it returns 0 for an invalid shape or when no CUDA device is usable.
 */
size_t sb_partial_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t lanes);
int32_t sb_partial_completion(const void *X, const void *W, int64_t M, int64_t N, int64_t K,
                              int32_t lanes, void *Y, int32_t y_bf16, void *workspace,
                              size_t workspace_bytes, void *stream);

/*
 * The decision before the path ("SemBridge", Section 8.2, Equation (7)): between the
 * checker-accepted plans, project at the source (plan s) rather than transfer the complete
 * logits (plan r) when the transfer saved exceeds the local cost added:
 *   (bytes_ref - bytes_proj) / link_bytes_per_s + frame_startup_s * (frames_ref - frames_proj)
 *       > local_proj_s - local_ref_s.
 * Bytes and frames are those crossing the link per step; the local costs are the two plans'
 * on-device times (for example this library's sb_lmhead_project time for the projected
 * surface and for SB_FULL_LOGITS).  *margin_s (may be NULL) receives left minus right side.
 * Returns 1 (project), 0 (transfer complete logits), or -1 for a non-positive or non-finite
 * bandwidth or a negative or non-finite byte, frame or startup argument.  Host only.
 */
int32_t sb_select_source_projection(double bytes_ref, double bytes_proj, double frames_ref,
                                    double frames_proj, double link_bytes_per_s,
                                    double frame_startup_s, double local_proj_s,
                                    double local_ref_s, double *margin_s);

/*
 * Training the head: the cross entropy of the rows' targets and its gradients (no paper
 * counterpart; the logits are those of sb_lmhead_project, and like there no logits are kept).
 *   lse_r  = log sum_j exp(z_rj),   z = H·Wᵀ
 *   loss_r = lse_r - z_r,target(r) + z_loss * lse_r^2
 * and 0, without a gradient, for rows whose target equals ignore_index (their row of dH is 0,
 * and they add nothing to dW, whatever their row of H holds).
 */
typedef enum sb_reduction {
    SB_REDUCE_NONE = 0, /* every row's own loss, [M]                                     */
    SB_REDUCE_SUM = 1,  /* their sum, [1]                                                */
    SB_REDUCE_MEAN = 2  /* the sum over the count of rows not ignored (0 where none is)  */
} sb_reduction;

/* Bytes of workspace of the forward call; 0 if the arguments are invalid. */
size_t sb_cross_entropy_workspace_bytes(int64_t M, int64_t d, int64_t V);

/*
 * The losses: the record GEMM of sb_lmhead_records, then one kernel over the records.
 *   H, W, M, d, V   as for sb_lmhead_project (row-major W); M = 0 is allowed (a batch without
 *               tokens: the sum and the mean are 0), and H, targets and lse may then be NULL.
 *   targets     device int32 [M]: in [0, V), or ignore_index (any value, also one inside the
 *               vocabulary, which then never counts as a target).  Another value gives the
 *               row's loss as NaN, and sb_last_device_status reports SB_ERR_INVALID_ARG.
 *   reduction   an sb_reduction;  z_loss: finite.
 *   loss        device float [M] (SB_REDUCE_NONE) or [1].
 *   lse         device float [M]: every row's logsumexp, also the ignored ones'; the backward
 *               call reads it.
 *   workspace   device, 256-byte aligned, >= sb_cross_entropy_workspace_bytes(M, d, V); no
 *               initialisation.  Its header is read by sb_last_device_status.
 * Two kernels on `stream`.  W may be written by the kernel before (an optimizer step): unlike
 * sb_lmhead_project, this call loads nothing before that kernel has finished.
 */
int32_t sb_cross_entropy_forward(const void *H, const void *W, const int32_t *targets, int64_t M,
                                 int64_t d, int64_t V, int32_t ignore_index, int32_t reduction,
                                 float z_loss, float *loss, float *lse, void *workspace,
                                 size_t workspace_bytes, void *stream);

/* Bytes of workspace of the backward call, which depend on the SM count of the current device
 * (the dH reduction may be split over the SMs): 0 for invalid arguments or without a device.
 * with_dH, with_dW: whether that gradient is asked for (at least one). */
size_t sb_cross_entropy_backward_workspace_bytes(int64_t M, int64_t d, int64_t V, int64_t piece,
                                                 int32_t with_dH, int32_t with_dW);

/*
 * The gradients, in pieces of the vocabulary: for each piece the logits are formed again and
 * G = dL/dz of the piece is written in bf16 (up to 32 rows: in two bf16 parts) to the
 * workspace, then dH += G·W and dW = Gᵀ·H in one launch.  Accumulation is fp32; dH and dW are
 * rounded to bf16 once.  Every sum has a fixed order, so equal calls give equal bits.
 * A target's entry, p - 1, is formed from lse and an fp32 logit: it is off by the roundings of
 * lse (2^-23 of it), however near 1 p is.
 *   H, W, targets, M, d, V, ignore_index, reduction, z_loss   as in the forward call.
 *   lse         device float [M], from the forward call.
 *   grad        device float: the incoming gradient, [M] for SB_REDUCE_NONE, else [1]; NULL
 *               stands for ones.  Read on the device when the kernels run.  One that is not
 *               finite shows in dW and in its rows of dH; ignored rows stay 0.
 *   piece       vocabulary columns per piece, rounded up to a multiple of 256; 0 leaves the
 *               choice to the library (at most 256 MB for the piece of G).
 *   dH, dW      device bf16 [M, d] and [V, d], 16-byte aligned, overwritten; either may be NULL
 *               (a frozen head, or a first layer), and its product is then not formed.
 *   workspace   device, 256-byte aligned, of at least
 *               sb_cross_entropy_backward_workspace_bytes(M, d, V, piece, dH, dW) bytes.
 * A target outside [0, V) that is not ignore_index contributes no "- 1" term; the forward call
 * reports it.  M = 0 writes dW = 0.
 */
int32_t sb_cross_entropy_backward(const void *H, const void *W, const int32_t *targets,
                                  const float *lse, const float *grad, int64_t M, int64_t d,
                                  int64_t V, int32_t ignore_index, int32_t reduction,
                                  float z_loss, int64_t piece, void *dH, void *dW,
                                  void *workspace, size_t workspace_bytes, void *stream);

/* Storage type of an array that may be bf16 or fp32. */
typedef enum sb_type { SB_BF16 = 0, SB_F32 = 1 } sb_type;

/* The gate of sb_residual_norm_*. */
typedef enum sb_gate {
    SB_GATE_NONE = 0,    /* factor 1                                                     */
    SB_GATE_CHANNEL = 1, /* one vector [d] for all rows, of the weights' type            */
    SB_GATE_TOKEN = 2    /* bf16 [M, d], one value per row and channel                   */
} sb_gate;

/*
 * The end of a transformer block, and what the output head reads after the last one (no paper
 * counterpart).  With n(x; w) = w * x / sqrt(mean(x^2) + eps) over a row:
 *   h_out = scale * h + gate * n(y; post),     x = n(h_out; pre).
 *   h           device [M, d] of stream_type (an sb_type): the residual stream.
 *   y           device bf16 [M, d]: the block's output.
 *   pre         device [d] of weight_type (an sb_type): the next block's (or the head's) norm.
 *   post        device [d] of weight_type, or NULL: no norm after the block, n(y; post) is y.
 *   gate        as gate_kind (an sb_gate) says; ignored for SB_GATE_NONE.
 *   M, d        M >= 0 rows; 1 <= d <= 16384.  Every array is contiguous; 16-byte aligned
 *               arrays with d a multiple of 8 (or 4) are read in wide loads, others value by
 *               value.
 *   scale, eps  finite; eps >= 0 (a row of zeros with eps = 0 gives NaN).
 *   h_out       device [M, d] of stream_type; may be h itself.
 *   x           device bf16 [M, d]; may be y itself.  Formed from h_out before its rounding.
 * One kernel on `stream`; no workspace.
 */
int32_t sb_residual_norm_forward(const void *h, const void *y, const void *pre, const void *post,
                                 const void *gate, int32_t gate_kind, int64_t M, int64_t d,
                                 int32_t stream_type, int32_t weight_type, float scale, float eps,
                                 void *h_out, void *x, void *stream);

/* Bytes of workspace of the backward call, which depend on the SM count of the current device;
 * 0 for invalid arguments or without a device. */
size_t sb_residual_norm_workspace_bytes(int64_t M, int64_t d);

/*
 * Its gradients.  h is here the forward call's h_out as it was stored; y, pre, post, gate,
 * gate_kind, the types, scale and eps as there.
 *   dx          device bf16 [M, d]: the gradient of x.
 *   dh          device [M, d] of stream_type: the gradient of h_out from its other readers, or
 *               NULL where there is none (the last block).
 *   dh_out      device [M, d] of stream_type: the gradient of the forward call's h; may be dh.
 *   dy          device bf16 [M, d]; may be dx.
 *   dpre, dpost device [d] of weight_type (dpost only with post), summed over the rows in fp32
 *               in a fixed order: equal calls give equal bits.
 *   dgate       like gate (NULL for SB_GATE_NONE); summed over the rows for SB_GATE_CHANNEL.
 *   workspace   device, 16-byte aligned, >= sb_residual_norm_workspace_bytes(M, d); no
 *               initialisation.
 * Two kernels on `stream`.  M = 0 writes zeros to dpre, dpost and the gate vector's gradient.
 */
int32_t sb_residual_norm_backward(const void *dx, const void *dh, const void *h, const void *y,
                                  const void *pre, const void *post, const void *gate,
                                  int32_t gate_kind, int64_t M, int64_t d, int32_t stream_type,
                                  int32_t weight_type, float scale, float eps, void *dh_out,
                                  void *dy, void *dpre, void *dpost, void *dgate, void *workspace,
                                  size_t workspace_bytes, void *stream);

/*
 * An AdamW step over many tensors at once (no paper counterpart).  Per value, with g the
 * gradient times *grad_scale and t the step:
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2,
 *   w = (1 - lr weight_decay) w - lr / (1 - beta1^t) * m / (sqrt(v / (1 - beta2^t)) + eps),
 * all in fp32; what the moments keep is rounded operation by operation, the quotient is within
 * 2^-20.  w is `master` where there is one (then param
 * receives its rounding to bf16), else param.  The moments are held
 *   state_bits = 32: in fp32;
 *   state_bits = 8: as E4M3 codes (the 8-bit floating-point type with 4 exponent and 3 mantissa
 *     bits, largest value 448) in blocks of 256 consecutive values with one fp32 scale each (top /
 *     448 with the largest magnitude top; the codes are those of value * (1 / top * 448); a block
 *     whose top is below 2^-100 is stored as zeros).
 *     exp_avg_sq then holds sqrt(v), whose range of exponents is half of v's, and a root that is
 *     not zero is never stored as zero, so that no small v turns into a division by eps alone.
 *     The step itself uses m and v before they are stored.
 */
typedef struct sb_adamw_tensor {
    void *param;        /* device [n] of param_type                                          */
    const void *grad;   /* device [n] of grad_type                                           */
    float *master;      /* device fp32 [n], for a bf16 param; NULL: param is the weight      */
    void *exp_avg;      /* device [n]: fp32, or E4M3 codes (one byte each)                   */
    void *exp_avg_sq;   /* device [n]: fp32, or E4M3 codes of the root                       */
    float *scale;       /* state_bits = 8: device fp32 [ceil(n / 256)], of exp_avg           */
    float *scale_sq;    /* state_bits = 8: device fp32 [ceil(n / 256)], of exp_avg_sq        */
    int64_t n;          /* values; 0 is allowed (the tensor is skipped)                      */
    double weight_decay;
    int32_t param_type, grad_type; /* sb_type                                                */
} sb_adamw_tensor;

/*
 *   tensors     host array of `count` (>= 0) descriptors, read during the call.  Arrays of
 *               different tensors must not overlap.  Tensors whose arrays are all 16-byte
 *               aligned are read in wide loads, others value by value.
 *   lr          >= 0; 0 <= beta1, beta2 < 1; eps >= 0; weight_decay >= 0; all finite.
 *   step        t, >= 1.
 *   grad_scale  device float [1] (an inverse loss scale, a clipping factor), read when the
 *               kernels run; NULL: 1.
 * One kernel per 384 tensors on `stream`; no workspace.  The kernels signal no dependents early,
 * which is what sb_lmhead_project asks of a kernel that writes its W.  Step number and rate are
 * host values: a captured call repeats its step's bias correction at every replay.
 */
int32_t sb_adamw_step(const sb_adamw_tensor *tensors, int64_t count, double lr, double beta1,
                      double beta2, double eps, int64_t step, int32_t state_bits,
                      const float *grad_scale, void *stream);

/*
 * The other end of the model (no paper counterpart): the tokens' rows of the vocabulary matrix,
 *   out[t] = scale * W[ids[t]],
 * and the gradient of that lookup.  W may be the output head's (a tied embedding).
 *   ids         device int32 [M]: in [0, V), or ignore_index (any value, also one inside the
 *               vocabulary): padding, whose row of out is 0 and which adds nothing to dW.  Another
 *               value gives a row of NaN, and adds nothing to dW; nothing outside W is read.
 *   W           device [V, d] of weight_type (an sb_type), row-major.
 *   M, d, V     M >= 0 tokens (M <= 2^31 - 65536); 1 <= d <= 2^22; 1 <= V < 2^31 - 1.  16-byte
 *               aligned arrays are read in wide loads, by the gradient where d is a multiple of 8 (or
 *               4), others value by value.
 *   scale       finite.
 *   out         device [M, d] of out_type, rounded once; not over W's or ids' memory.
 * One kernel on `stream`; no workspace.
 */
int32_t sb_embedding_forward(const int32_t *ids, const void *W, int64_t M, int64_t d, int64_t V,
                             int32_t ignore_index, float scale, int32_t weight_type,
                             int32_t out_type, void *out, void *stream);

/* Bytes of workspace of the backward call; 0 if the arguments are invalid. */
size_t sb_embedding_backward_workspace_bytes(int64_t M, int64_t d);

/*
 * Its gradient: with S[v] = scale * (sum of dout[t] over the t with ids[t] = v), in fp32 and in a
 * fixed order (equal calls give equal bits),
 *   add = 0:  dW = S, all of it written (zeros for the rows that no token has);
 *   add = 1:  dW = dW + S in the rows that a token has, rounded once; the others are not touched.
 *             That is how a tied embedding's gradient joins the head's (sb_cross_entropy_backward).
 *   dout        device [M, d] of grad_type (an sb_type).
 *   dW          device [V, d] of weight_type; not over ids' or dout's memory.
 *   workspace   device, 256-byte aligned, >= sb_embedding_backward_workspace_bytes(M, d); no
 *               initialisation; not over the other arrays' memory.
 * Up to four kernels on `stream` (one more for every factor of 8 that M is above 65,536).
 */
int32_t sb_embedding_backward(const int32_t *ids, const void *dout, int64_t M, int64_t d, int64_t V,
                              int32_t ignore_index, float scale, int32_t grad_type,
                              int32_t weight_type, int32_t add, void *dW, void *workspace,
                              size_t workspace_bytes, void *stream);

/*
 * Dropout whose mask is a function of a seed (no paper counterpart):
 *   out[i] = residual[i] + (element i is kept ? x[i] * 65536 / (65536 - t) : 0),   t = round(65536 p).
 * Element i is kept where 16-bit field i mod 4 (0: the lowest bits) of draw i / 4 of the SplitMix64
 * stream of the seed is >= t; draw n is the finaliser of seed + (n + 1) * 0x9E3779B97F4A7C15, as
 * for sb_lmhead_project.  No mask is stored: the gradient of x is the same call, without residual,
 * on the gradient of out.  Different layers and steps need different seeds.
 *   x           device [n] of x_type (an sb_type).
 *   residual    device [n] of out_type, or NULL: 0.
 *   n           >= 0.  16-byte aligned arrays are read in wide loads, others value by value.
 *   p           0 <= p <= 1; p = 1 drops everything.
 *   seed_offset device uint64 [1], added to seed when the kernel runs (a step counter, so that the
 *               replays of a captured call differ), or NULL: 0.
 *   out         device [n] of out_type; may be x (of the same type) or residual, but not lie over a part
 *               of them.
 * One kernel on `stream`.
 */
int32_t sb_dropout(const void *x, const void *residual, int64_t n, int32_t x_type, int32_t out_type,
                   float p, uint64_t seed, const uint64_t *seed_offset, void *out, void *stream);

/*
 * The end of a block with dropout and a layer norm (no paper counterpart): over each row,
 *   h_out = h + dropout(y),
 *   x = (h_out - mean) / sqrt(variance + eps) * weight + bias,
 * with mean and variance of h_out (variance: of the centred values, over d).  Element (r, c) of y
 * is dropped as element r * d + c of sb_dropout is.
 *   h           device [M, d] of stream_type (an sb_type): the residual stream.
 *   y           device bf16 [M, d]: the block's output, or NULL: h_out is h and is not written.
 *   weight, bias  device [d] of weight_type (an sb_type); bias may be NULL.
 *   M, d, eps, alignment   as for sb_residual_norm_forward (with one value to a row x is bias; a row of
 *               equal values has no answer with eps = 0: NaN, or what the mean's rounding leaves).
 *   p, seed, seed_offset   as for sb_dropout; without y not used.
 *   h_out       device [M, d] of stream_type; may be h itself.
 *   x           device bf16 [M, d]; may be y itself.  Formed from h_out before its rounding.
 * No other output may share memory with an input or another output.  One kernel on `stream`; no
 * workspace.
 */
int32_t sb_layer_norm_forward(const void *h, const void *y, const void *weight, const void *bias,
                              int64_t M, int64_t d, int32_t stream_type, int32_t weight_type,
                              float p, uint64_t seed, const uint64_t *seed_offset, float eps,
                              void *h_out, void *x, void *stream);

/* Bytes of workspace of the backward call, which depend on the SM count of the current device;
 * 0 for invalid arguments or without a device. */
size_t sb_layer_norm_workspace_bytes(int64_t M, int64_t d);

/*
 * Its gradients.  h is here the forward call's h_out as it was stored; weight, the types, p, seed,
 * seed_offset (with the value that it had then) and eps as there.
 *   dx          device bf16 [M, d]: the gradient of x.
 *   dh          device [M, d] of stream_type: the gradient of h_out from its other readers, or
 *               NULL where there is none.
 *   dh_out      device [M, d] of stream_type: the gradient of the forward call's h; may be dh.
 *   dy          device bf16 [M, d], the gradient of y, or NULL (there was none); may be dx.
 *   dweight, dbias  device [d] of weight_type (dbias or NULL), summed over the rows in fp32 in a
 *               fixed order: equal calls give equal bits.
 *   workspace   device, 16-byte aligned, >= sb_layer_norm_workspace_bytes(M, d); no initialisation.
 * No other output (nor the workspace) may share memory with an input or another output.  Two kernels
 * on `stream`.  M = 0 writes zeros to dweight and dbias.
 */
int32_t sb_layer_norm_backward(const void *dx, const void *dh, const void *h, const void *weight,
                               int64_t M, int64_t d, int32_t stream_type, int32_t weight_type,
                               float p, uint64_t seed, const uint64_t *seed_offset, float eps,
                               void *dh_out, void *dy, void *dweight, void *dbias, void *workspace,
                               size_t workspace_bytes, void *stream);

/*
 * Verification of drafted tokens against the head's distribution (no paper counterpart): what
 * follows SB_FULL_LOGITS when a small model has proposed the next tokens of each request.
 *
 * Request b has the rows starts[b] .. starts[b+1] - 1 of the logits, one more than drafts: the
 * target's logits behind each draft's predecessor, and behind the last draft.  With p the softmax
 * of a row's logits / T and q that of the draft's (1 at the drafted token and 0 elsewhere where the
 * drafts have no logits), the draft x of row r stays if
 *   uniforms[r] < p(x) / q(x)
 * and all drafts before it stay.  The first one that does not is replaced by a sample of
 * max(p - q, 0) (of p, where that is nowhere positive); where all stay the last row adds a sample
 * of its p.  The tokens are then distributed as samples of the target's own.  The sample of row r
 * is the column with the largest w_j / -log u_rj (the lowest of equal ones) with the 24-bit uniform
 * u of sb_lmhead_project at index r*V + j of the seed's stream.  u = 0 gives a score of 0, which wins
 * only where no other column has a weight (in fp32).  Where all stay that is SB_GUMBEL_TOKEN's choice
 * for the same logits; sb_lmhead_project races on its fp32 logits, SB_FULL_LOGITS has them rounded to
 * bf16 (2^-8 of a logit, over T), so that keys nearer than that may change places.
 *   logits      device [R, V] of logits_type (an sb_type).  -inf is a column without probability.
 *   draft_logits  device [draft_rows, V] of that type: a row for every draft, one request's behind
 *               the other's, without gaps; draft_rows = -1 and NULL: the drafts have none.
 *   drafts      device int32 [R]: in row r the token drafted for it; a request's last one is not
 *               read.  One outside [0, V) does not stay, its sample is of p, and
 *               sb_last_device_status reports SB_ERR_INVALID_ARG.
 *   starts      device int32 [B + 1], ascending, 0 <= starts[0], starts[B] <= R.  A request may have
 *               no rows, and rows in front of starts[0] belong to none (nor do they have draft rows).
 *               One whose rows are not between starts[0] and starts[B], or not inside R (or its
 *               drafts' not inside draft_rows) gets accepted -1 and nothing else, not in its rows
 *               either, and the status reports SB_ERR_INVALID_ARG.
 *   uniforms    device float [R], each in [0, 1); a request's last one is not read.
 *   lse, draft_lse  device float [R] and [draft_rows]: the rows' logsumexp of logits / T where the
 *               caller has it (T = 1: that of sb_lmhead_project), each or NULL: formed here.
 *              Given ones are taken as they are: log p is off by what they are, of which fp32's
 *              rounding alone is 2^-24 max|z| / T.  At temperatures where that counts leave them out.
 *              (sb_lmhead_project's is that of its fp32 logits: for bf16 ones the row's p then sum to 1
 *              but for what their roundings leave, 2^-8 max|z| at most and far less on average.)
 *   R, B, V     R, draft_rows < 2^24; B <= 2^24; 1 <= V < 2^31 - 65536.
 *   temperature finite, >= 1e-30; 1 / T is rounded to fp32.
 *   token       device int32 [R]: from starts[b] on the drafts that stay and the sample behind them,
 *               and -1 in all other rows, those in front of the first request and behind the last
 *               one among them.
 *   accepted    device int32 [B]: how many drafts of the request stay.
 *   token_logprob  device float [R], or NULL: log p(token); 0 where there is no token.
 *   workspace   device, 256-byte aligned, >= sb_verify_workspace_bytes(R, draft_rows, V); no
 *               initialisation.  Its header is read by sb_last_device_status.
 * token may be drafts itself.  No other output (nor the workspace) may share memory with an input or
 * another output.  A sampled row without any finite logit answers -1 with log-prob NaN.  Up to two
 * kernels on `stream`, three for more than 2048 requests with draft_logits.  Equal calls give equal bits.
 */
size_t sb_verify_workspace_bytes(int64_t R, int64_t draft_rows, int64_t V);
int32_t sb_verify_drafts(const void *logits, const void *draft_logits, const int32_t *drafts,
                         const int32_t *starts, const float *uniforms, const float *lse,
                         const float *draft_lse, int64_t R, int64_t draft_rows, int64_t B,
                         int64_t V, int32_t logits_type, float temperature, uint64_t seed,
                         int32_t *token, int32_t *accepted, float *token_logprob, void *workspace,
                         size_t workspace_bytes, void *stream);

/*
 * The same with a seed that moves on: seed_offset, device uint64 [1] (NULL: 0), is added to seed when
 * the kernels run.  A captured call repeats its seed at every replay, and with it the draws of every
 * row; a decoding loop that replays a step counts seed_offset up (and fills in new uniforms).
 */
int32_t sb_verify_drafts_at(const void *logits, const void *draft_logits, const int32_t *drafts,
                            const int32_t *starts, const float *uniforms, const float *lse,
                            const float *draft_lse, int64_t R, int64_t draft_rows, int64_t B,
                            int64_t V, int32_t logits_type, float temperature, uint64_t seed,
                            const uint64_t *seed_offset, int32_t *token, int32_t *accepted,
                            float *token_logprob, void *workspace, size_t workspace_bytes,
                            void *stream);

/*
 * The same for greedy decoding, where SB_TOKEN has given each row's own choice: a draft stays while
 * it is that choice, and the choice of the row behind the last one that stays follows.
 *   target      device int32 [R]: the rows' tokens; drafts, starts, token and accepted as above
 *               (starts that are out of range give accepted -1; there is no status word).  token may
 *               also be target itself.
 * One kernel on `stream`; no workspace.
 */
int32_t sb_verify_greedy(const int32_t *target, const int32_t *drafts, const int32_t *starts,
                         int64_t R, int64_t B, int32_t *token, int32_t *accepted, void *stream);

/* Device status of the last call that used out->workspace: SB_OK, SB_ERR_DEVICE_TIMEOUT
 * (a bounded wait gave up) or SB_ERR_INVALID_ARG (a scoring target outside [0, V); when
 * both happen the timeout is reported).  Synchronous: copies the header to the host (call
 * it after synchronising the stream).  Returns SB_ERR_CUDA if the copy fails. */
int32_t sb_last_device_status(const sb_outputs *out);

/* Static description of a status code; never NULL. */
const char *sb_status_string(int32_t status);

/* Number of SMs and compute capability (major * 10 + minor) of the current device, as the
 * library sees them; -1 without a usable device. */
int32_t sb_device_info(int32_t *num_sms, int32_t *cc);

/* Test hook for the device watchdog.  stall_epilogue != 0 makes the epilogue warps of
 * later sb_lmhead_project calls wait on a barrier that nothing ever arrives at, so their
 * bounded wait runs out and the call reports SB_ERR_DEVICE_TIMEOUT through
 * sb_last_device_status (the outputs are then undefined).  wait_limit_ns (> 0) is the
 * time limit of every device-side wait (default 2 s).  Process-wide; not for production.
 * Returns SB_ERR_INVALID_ARG for wait_limit_ns == 0. */
int32_t sb_debug_configure(int32_t stall_epilogue, uint64_t wait_limit_ns);

/* Test hook: how many tensor maps of row-major matrices this process has encoded (calls with the
 * operands of an earlier one find theirs and encode none). */
uint64_t sb_debug_map_encodes(void);

#ifdef __cplusplus
}
#endif

#endif /* SB_H */
