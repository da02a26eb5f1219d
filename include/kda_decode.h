/*
 * kda_decode.h -- C ABI of the MI355X (gfx950) KDA recurrent decode library.
 *
 * The operation (Kimi Delta Attention decode, one launch):
 *   for each request r, head h, and each of the request's rows t in order,
 *   with the state S of (r, h) held in fp32 between rows:
 *     qn = q / sqrt(|q|^2 + 1e-6),  kn = k / sqrt(|k|^2 + 1e-6)
 *     a  = exp(g)  (per key channel),  beta = 1 / (1 + exp(-b))
 *     S' = diag(a) S;  u = v - S'^T kn;  S = S' + beta kn u^T
 *     o  = scale * S^T qn
 *     state_at(r, t) <- S   (fp32 as is, or fp16 rounded to nearest even)
 *   The first row's initial state is read from state_at(r, 0).
 *
 * Passages this follows (page title, then section):
 *  - ROCm/ATOM PR #2945 (gfx950 mono K1 takes an fp16 KDA state pool),
 *    Summary and Changes: the pool's dtype is a build constant of the
 *    kernel; each loaded state is widened to fp32, the recurrence runs in
 *    fp32, each stored state is rounded to fp16 to nearest even; one address
 *    function, state_at, serves the request's initial state and every
 *    token's snapshot slot; a pool of the other dtype is refused (it would
 *    be read at the wrong element size); bf16 is refused, not reinterpreted.
 *    Limitations: k is unit after normalisation, beta in (0, 1), decay <= 1.
 *  - ROCm/ATOM PR #2130 "perf(kimi-k3): make the KDA temporal state dtype
 *    configurable", What: a [12, 128, 128] state per layer streams through
 *    HBM every decode token (state-bandwidth bound); q and k are
 *    L2-normalised in-kernel; the recurrence accumulates in fp32 whatever
 *    the pool stores.  Copilot review: the initial state must be validated
 *    early instead of being dereferenced when absent.
 *
 * Conventions for every function:
 *  - Return value: KDA_OK (0) or a kda_status code; kda_strerror() names it.
 *    Functions returning a size or offset return a negative kda_status on
 *    error instead.
 *  - Arguments are validated on the host before any HIP call; a refused call
 *    changes nothing and launches nothing.
 *  - The caller owns every buffer.  The library allocates no memory, never
 *    synchronises, and enqueues its work on the caller's stream (a
 *    hipStream_t passed as void*, NULL = the null stream).  A device fault
 *    surfaces at the caller's next synchronisation.
 */
#ifndef KDA_DECODE_H
#define KDA_DECODE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_ABI_VERSION 11  /* 11: kda_launch_opts.g_raw, later the kda_kv_* functions and those for trees of drafted tokens (new symbols only); 10: kda_rows_probe tile shapes; 9: kda_decode_step_conv_noalloc; 8: kda_decode_step_conv_ws; 7: kda_rows_probe; 6: kda_bw_probe and kda_tile_probe; 5: KDA_ROWS_MATRIX */

/* Head dimensions this build supports (the Kimi-K3 KDA layer shape). */
#define KDA_HEAD_K 128
#define KDA_HEAD_V 128
/* Rows (tokens) one request may chain in one launch: 1 + up to 7 drafts. */
#define KDA_MAX_ROWS 8

/* Nodes of one request's tree of drafted tokens. */
#define KDA_MAX_NODES 64

/* Element type of a state pool (or of the tensors of the kda_kv_* functions). */
typedef enum kda_dtype {
  KDA_F32 = 0,
  KDA_F16 = 1,
  KDA_BF16 = 2 /* refused for state pools; a type of the kda_kv_* functions' tensors
                  and of kda_verify_drafts' probabilities */
} kda_dtype;

typedef enum kda_status {
  KDA_OK = 0,
  KDA_ERR_NULL = 1,           /* a required pointer is NULL */
  KDA_ERR_DTYPE_REFUSED = 2,  /* bf16 or an unknown dtype */
  KDA_ERR_DTYPE_MISMATCH = 3, /* state_dtype differs from the pool's dtype */
  KDA_ERR_SHAPE = 4,          /* K or V != 128, H outside [1, 65535], n_slots < 1;
                                 or a key/value cache's shape */
  KDA_ERR_ROWS = 5,           /* rows per request outside [1, KDA_MAX_ROWS], or a
                                 tree's outside [0, KDA_MAX_NODES] */
  KDA_ERR_SLOT = 6,           /* slot id out of range or repeated, or more
                                 rows than slots */
  KDA_ERR_ALIGN = 7,          /* a device pointer is not 16-byte aligned */
  KDA_ERR_ARG = 8,            /* other bad argument (negative count, index
                                 out of range, non-finite scale) */
  KDA_ERR_LAUNCH = 9          /* the HIP runtime reported a launch error */
} kda_status;

/*
 * A state pool: device memory holding [n_slots, H, K, V] elements of dtype,
 * row-major with V fastest, i.e. slot s, head h, key row i, value column j
 * lives at element ((s * H + h) * K + i) * V + j.  base must be 16-byte
 * aligned.  The caller allocates, owns and frees it.
 */
typedef struct kda_pool {
  void* base;
  int32_t n_slots;
  int32_t H;
  int32_t K;
  int32_t V;
  kda_dtype dtype;
} kda_pool;

/*
 * kda_decode_step -- one decode launch over n_req requests of
 * n_rows_per_slot rows each (R = n_req * n_rows_per_slot rows in all).
 *
 *  pool        the state pool (dtype F32 or F16), updated in place.
 *  slot_ids    device int32 [R]: row t of request r uses slot
 *              slot_ids[r * n_rows_per_slot + t] (see kda_state_at).  The
 *              ids of one launch must be distinct and in [0, n_slots):
 *              kda_validate checks a host copy.  On the device, a request
 *              with any id out of range is skipped: its out rows are set to
 *              NaN and no state is read or written.  Repeated ids are not
 *              detected on the device and give an unspecified result.
 *  q, k, g     device fp32 [R, H, 128]; v: device fp32 [R, H, 128];
 *  b           device fp32 [R, H]; rows of one request are adjacent.
 *              g is the log-decay (a = exp(g)); callers keep g <= 0.
 *  out         device fp32 [R, H, 128], written.
 *  state_dtype the dtype the caller built for; must equal pool->dtype.
 *  scale       read-out scale, usually 1/sqrt(128).  Must be finite.
 *  stream      hipStream_t as void*, NULL for the null stream.
 *
 * All device pointers must be 16-byte aligned (slot_ids and b: 4-byte).
 * n_req == 0 is a valid no-op, and then only the pool must be non-NULL.
 * Checks run in the order: pool NULL, DTYPE_REFUSED, DTYPE_MISMATCH,
 * SHAPE, ROWS, ARG (counts), SLOT, then the row buffers' NULL, ARG (scale,
 * opts), ALIGN.  Errors: KDA_ERR_NULL, KDA_ERR_DTYPE_REFUSED,
 * KDA_ERR_DTYPE_MISMATCH, KDA_ERR_SHAPE, KDA_ERR_ROWS, KDA_ERR_SLOT (more
 * rows than slots), KDA_ERR_ALIGN, KDA_ERR_ARG, KDA_ERR_LAUNCH.
 */
int kda_decode_step(const kda_pool* pool, const int32_t* slot_ids,
                    const float* q, const float* k, const float* v,
                    const float* g, const float* b, float* out, int32_t n_req,
                    int32_t n_rows_per_slot, kda_dtype state_dtype,
                    float scale, void* stream);

/*
 * Chained-row layouts (kda_launch_opts.rows_layout; chained rows only).
 *  KDA_ROWS_K_SPLIT  each wave of a workgroup holds a slice of the 128 key
 *                    rows for all of the tile's bv columns; every row's
 *                    partial column sums over K meet in LDS behind a barrier.
 *  KDA_ROWS_WAVE_K   each wave holds all 128 key rows of bv / waves_per_tile
 *                    columns (2 or 4 lanes per 16-byte row piece): a
 *                    row's column sums over K stay inside the wave (DPP and
 *                    permlane exchanges), and the waves of a workgroup run
 *                    their chains with no barrier between rows.
 *  KDA_ROWS_MATRIX   the request's rows as one block: all 2 n column sums
 *                    of the initial state (w0_t = S0^T (gamma_t kn_t) and
 *                    p0_t = S0^T (gamma_t qn_t), gamma_t the decays of rows
 *                    0..t multiplied) in one fp32 matrix-core product per
 *                    wave, the n x n couplings of the rows, a triangular
 *                    solve per column, then element-wise snapshots streamed
 *                    as whole rows.  Fixed shape: 64 columns over 4 waves
 *                    (bv and waves_per_tile must be 0 or 64 and 4).
 */
#define KDA_ROWS_DEFAULT 0
#define KDA_ROWS_K_SPLIT 1
#define KDA_ROWS_WAVE_K 2
#define KDA_ROWS_MATRIX 3

/*
 * Launch options of kda_decode_step_ex.  Zero-initialise for the library's
 * defaults; each non-zero field overrides one choice.
 *  waves_per_tile  wavefronts per workgroup: 1, 2, 4, 8.  K-split layout and
 *                  single rows: the waves split one tile's 128 key rows.
 *  bv              value columns per workgroup.  K-split layout and single
 *                  rows: 32, 64 or 128 for fp32 pools (8, 16, 32 lanes per
 *                  tile row), 64 or 128 for fp16.  Whole-K layout: waves x
 *                  lanes x columns per lane (4 fp32, 8 fp16) with 2 or 4
 *                  lanes and 2, 4 or 8 waves, at most 128.
 *  block_rows      chained rows only: 0 (default) runs a request's rows
 *                  one after the other (two column sums over K and a
 *                  cross-lane reduction per row); non-zero takes them as one
 *                  block (all 2 n column sums of the initial state in one
 *                  pass, an n x n triangular solve, then element-wise
 *                  snapshots).  Both compute the same chain and round
 *                  differently; on MI355X the block form measured slower at
 *                  8 rows (its n x n coupling sums cost more than the
 *                  per-row reductions they replace).  The block form uses
 *                  the K-split layout (with KDA_ROWS_WAVE_K it is refused)
 *                  and, for fp16 pools, at least 2 waves (one wave's 128
 *                  state values and 8 x 8 x 3 column sums per lane do not
 *                  fit in the register file: refused).
 *  rows_layout     chained rows only: KDA_ROWS_DEFAULT, KDA_ROWS_K_SPLIT,
 *                  KDA_ROWS_WAVE_K or KDA_ROWS_MATRIX (a block form
 *                  whatever block_rows says); ignored for one row.  The
 *                  default, with units = requests x heads: for fp16 pools
 *                  the matrix-core block form for 3 rows or more up to 240
 *                  units, else the whole-K layout up to 48 units and the K
 *                  split beyond; when bv or waves_per_tile is set, the
 *                  whole-K layout (bv 64 over 4 waves unless set).  For
 *                  fp32 pools the matrix-core block form for 6 rows or
 *                  more up to 48 units with no bv or waves option, else the
 *                  K split (bv 64 over 8 waves).  block_rows alone selects
 *                  the K-split block form.
 * Supported K-split combinations keep 2..32 key rows per lane (rows per
 * lane = 2 * lanes per row / waves).  The shape changes the order of the
 * fp32 column sums over K (so results may differ in the last bits), never
 * the operation; fixing it fixes every result bit for given inputs.
 */
typedef struct kda_launch_opts {
  int32_t waves_per_tile;
  int32_t bv;
  int32_t block_rows;
  int32_t rows_layout;
  int32_t g_raw;  /* fused convolution entries only (0 elsewhere): see kda_decode_step_conv */
} kda_launch_opts;

/*
 * kda_decode_step_ex -- kda_decode_step with a separate initial-state slot
 * per request and launch options.
 *
 *  init_slot_ids  NULL, or device int32 [n_req]: request r reads its initial
 *                 state from slot init_slot_ids[r] instead of its row-0 slot
 *                 slot_ids[r * n_rows_per_slot].  This is how a speculative
 *                 step resumes from the snapshot of its last accepted token,
 *                 and how a checkpointed state is loaded (ROCm/ATOM PR #2945,
 *                 Changes: one address function serves the initial state,
 *                 every token's snapshot slot, and the checkpoint load and
 *                 flush).  An initial slot may be one of its own request's
 *                 snapshot slots (it is read before any store) but must not
 *                 be written by another request of the launch; kda_validate
 *                 checks a host copy.  With one row per request and
 *                 init_slot_ids[r] != slot_ids[r], the update is out of
 *                 place (ping-pong between two slots).
 *  opts           NULL for the defaults (see kda_launch_opts): for tests
 *                 that must hold the summation order fixed across launches
 *                 and for tuning sweeps.
 * Additional errors: KDA_ERR_ARG for a shape that is not supported; a request
 * whose initial slot is out of range is skipped on the device like one with
 * a bad snapshot slot (out rows NaN, nothing stored).
 */
int kda_decode_step_ex(const kda_pool* pool, const int32_t* slot_ids,
                       const int32_t* init_slot_ids,
                       const float* q, const float* k, const float* v,
                       const float* g, const float* b, float* out,
                       int32_t n_req, int32_t n_rows_per_slot,
                       kda_dtype state_dtype, float scale,
                       const kda_launch_opts* opts, void* stream);

/*
 * A short-convolution history pool: device memory holding [n_slots, 3, C]
 * bfloat16 values, C = 3 * H * 128 channels ordered (q | k | v) x H x 128,
 * entry 0 the oldest of the last 3 raw inputs of each channel.  Slot s of
 * the conv pool belongs with slot s of the state pool (one slot id addresses
 * both).  2 bytes x 3 entries x 4608 channels = 27,648 bytes per slot per
 * layer at H = 12: the part of the pages' per-slot memory that does not
 * follow the state dtype (ROCm/ATOM PR #2130, Memory).  base 16-byte aligned.
 */
typedef struct kda_conv_pool {
  void* base;
  int32_t n_slots;
  int32_t H;
} kda_conv_pool;

/*
 * kda_decode_step_conv -- the decode step with the short causal convolution
 * fused in front (q, k and v each pass a 4-tap depthwise causal convolution,
 * then SiLU; ROCm/ATOM PR #2894, the two-node trial: a 3-entry history is
 * read, then the old entries and the step's inputs are written back).
 *
 *  conv        the history pool (n_slots and H equal to the state pool's).
 *  x           device fp32 [R, 3, H, 128]: the raw q, k, v inputs (before
 *              the convolution) of every row.
 *  conv_w      device fp32 [3, H, 128, 4]: per-channel taps, tap 3 on the
 *              newest input.  No bias.
 *  g, b, out, slot_ids, init_slot_ids, n_req, n_rows_per_slot,
 *  state_dtype, scale, opts, stream: as in kda_decode_step_ex.
 * For row t of request r: q, k, v = silu(sum_j w_j win[t + j]) over the
 * window win = (history of the initial slot, raw rows 0..t of the request),
 * then the decode update.  Row t's snapshot slot receives both the state and
 * the history after row t (its last 3 raw inputs, rounded to bfloat16 to
 * nearest even); rows of one launch use their fp32 inputs directly.
 * Launch shapes: whole heads only (opts->bv 0 or 128), since a head's
 * history at the initial slot is read and may be rewritten in place by one
 * workgroup.  Chained rows take the matrix-core block form (KDA_ROWS_MATRIX:
 * 16 waves, two 64-column halves of 8; waves_per_tile 8: two halves of 4)
 * when rows_layout asks for it, or by default for 3 rows or more up to 192
 * (fp16) or 48 (fp32) requests x heads unless waves_per_tile or block_rows
 * is set; otherwise the K-split kernel with 2, 4 or 8 waves.  One row per
 * request: the single-row kernel over whole heads, by default 4 waves for
 * fp16 pools, and for fp32 pools 2 waves below 384 requests x heads and 4
 * from there.
 * KDA_ROWS_WAVE_K is refused; rows_layout is ignored for one row.
 * opts->g_raw: 0 (default), g is the log-decay as in kda_decode_step; 1, g
 * holds the raw gate x of each key channel and the step takes the
 * log-decay g = -softplus(x) = -log(1 + e^x), computing the decay as
 * 1 / (1 + e^x), so the gate is fused into the front end beside the
 * convolution.  Other values are refused, as is g_raw != 0 on the entries
 * without the convolution.
 * Errors: as kda_decode_step_ex, plus KDA_ERR_NULL for a missing conv pool,
 * x or conv_w, KDA_ERR_SHAPE if the pools' n_slots or H differ.
 */
int kda_decode_step_conv(const kda_pool* pool, const kda_conv_pool* conv,
                         const int32_t* slot_ids, const int32_t* init_slot_ids,
                         const float* x, const float* conv_w, const float* g,
                         const float* b, float* out, int32_t n_req,
                         int32_t n_rows_per_slot, kda_dtype state_dtype,
                         float scale, const kda_launch_opts* opts, void* stream);

/*
 * kda_decode_step_conv_ws -- kda_decode_step_conv with pair counters, which
 * let chained rows in the matrix-core block form split each head into two
 * 64-column workgroups of 8 waves (twice the workgroups: with fewer heads
 * than compute units, a unit's store throughput bounds the whole-head form).
 * Both halves read the initial slot's q and k history; the row whose slot
 * is the initial slot may overwrite it only after both have read it, so each
 * half adds 1 to the counter of its (request, head) once its reads are done,
 * and the half that finds an odd count writes that row's q and k history.
 * No workgroup waits for another.
 *
 *  pair_counts    NULL (then exactly kda_decode_step_conv), or device
 *                 uint32 [n_pair_counts], n_pair_counts >= n_req * H,
 *                 4-byte aligned: counter r * H + h serves request r, head
 *                 h.  Owned by the caller.  Every entry must be even
 *                 (zero-fill once) before the first call; each call adds 0
 *                 or 2 to an entry, so entries stay even and one buffer
 *                 serves any number of calls in sequence.  Calls that may run
 *                 at the same time (other streams, concurrent graphs) need
 *                 buffers of their own.
 *  n_pair_counts  entries of pair_counts (0 with NULL).
 *  opts           as kda_decode_step_conv, plus bv 64: the halves, which
 *                 need pair_counts.  With pair_counts, chained rows take
 *                 the halves when rows_layout is KDA_ROWS_MATRIX or by
 *                 default for fp16 up to 96 requests x heads, or 240 with
 *                 6 rows or more, and for fp32 up to 48, or 96 with 4 rows
 *                 or more, unless waves_per_tile or block_rows is set;
 *                 bv 128 keeps whole heads; beyond, the
 *                 defaults of kda_decode_step_conv.
 * Errors: as kda_decode_step_conv, plus KDA_ERR_NULL for NULL pair_counts
 * with n_pair_counts != 0, KDA_ERR_ARG for n_pair_counts < 0 or, with
 * counters given, n_pair_counts < n_req * H, or bv 64 without counters,
 * KDA_ERR_ALIGN for misaligned counters.
 */
int kda_decode_step_conv_ws(const kda_pool* pool, const kda_conv_pool* conv,
                            const int32_t* slot_ids, const int32_t* init_slot_ids,
                            const float* x, const float* conv_w, const float* g,
                            const float* b, float* out, int32_t n_req,
                            int32_t n_rows_per_slot, kda_dtype state_dtype,
                            float scale, uint32_t* pair_counts,
                            int32_t n_pair_counts, const kda_launch_opts* opts,
                            void* stream);

/*
 * kda_decode_step_conv_noalloc -- kda_decode_step_conv_ws for callers that
 * cannot allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc): the pair counters live in a
 * static device array of KDA_NOALLOC_MAX_PAIRS entries inside the library,
 * one per GPU it runs on, held until the process ends.  The call allocates
 * nothing; its first call on a device looks the array's address up on that
 * device (the stream's device, or the current one for the null stream).
 * Arguments and launch shapes as kda_decode_step_conv_ws with counters given.
 * Every call on a GPU shares that GPU's counters: calls that overlap on one
 * GPU race (results of chained rows in halves are then undefined), calls in
 * sequence do not.  Nothing needs clearing between calls: the counters stay
 * even.
 * Errors: as kda_decode_step_conv_ws, plus KDA_ERR_ARG when n_req * H exceeds
 * KDA_NOALLOC_MAX_PAIRS (checked before any device work), KDA_ERR_LAUNCH if
 * the counters' address cannot be found on the device.
 */
#define KDA_NOALLOC_MAX_PAIRS 4096
int kda_decode_step_conv_noalloc(const kda_pool* pool, const kda_conv_pool* conv,
                                 const int32_t* slot_ids, const int32_t* init_slot_ids,
                                 const float* x, const float* conv_w, const float* g,
                                 const float* b, float* out, int32_t n_req,
                                 int32_t n_rows_per_slot, kda_dtype state_dtype,
                                 float scale, const kda_launch_opts* opts, void* stream);

/*
 * kda_validate -- host-side check of a launch's arguments and slot tables
 * (ROCm/ATOM PR #2945, Changes: the step checks the pool's dtype against
 * the build; anything but fp32 or fp16 is refused).  slot_ids_host is a
 * HOST copy of the slot table [n_req * n_rows]; every id must lie in
 * [0, n_slots) and appear once.  init_slot_ids_host is NULL or a host copy
 * of the initial slots [n_req]: each in range and not among another
 * request's snapshot slots.  Touches no device memory.  Returns KDA_OK or
 * the first error found, in the order: NULL, DTYPE_REFUSED, DTYPE_MISMATCH,
 * SHAPE, ROWS, ARG, SLOT.
 */
int kda_validate(const kda_pool* pool, const int32_t* slot_ids_host,
                 const int32_t* init_slot_ids_host, int32_t n_req,
                 int32_t n_rows, kda_dtype state_dtype);

/*
 * kda_state_copy -- copy whole slots of a pool: for i in [0, n), the
 * [H, K, V] block of slot dst_slot_ids[i] becomes that of src_slot_ids[i]
 * (every head).  The ReplaySSM-style checkpoint flush (a chosen snapshot
 * into a checkpoint slot) and load (back into a working slot) through the
 * same slot addressing as the decode (ROCm/ATOM PR #2945, Changes).
 * src_slot_ids, dst_slot_ids: device int32 [n].  dst ids must be distinct
 * and no dst may be another pair's src (caller contract).  A pair with an
 * id out of range is skipped on the device.  Bytes are copied as they are:
 * the pool keeps its dtype.  Errors: KDA_ERR_NULL, KDA_ERR_DTYPE_REFUSED,
 * KDA_ERR_DTYPE_MISMATCH, KDA_ERR_SHAPE, KDA_ERR_ARG (n < 0 or n > 65535),
 * KDA_ERR_ALIGN, KDA_ERR_LAUNCH.  n == 0 is a no-op.
 */
int kda_state_copy(const kda_pool* pool, const int32_t* src_slot_ids,
                   const int32_t* dst_slot_ids, int32_t n, kda_dtype state_dtype,
                   void* stream);

/*
 * kda_state_at -- element offset, from pool->base, of the [H, K, V] block
 * that row `row` of request `req` reads or writes (ROCm/ATOM PR #2945,
 * Changes: one address function for the initial state and every token's
 * snapshot slot).  Head h's [K, V] state follows at + h * K * V.  Row 0's
 * block is also the request's initial state.  slot_ids_host is a host copy
 * of the slot table.  Returns a negative kda_status on error.
 */
int64_t kda_state_at(const kda_pool* pool, const int32_t* slot_ids_host,
                     int32_t n_rows, int32_t req, int32_t row);

/*
 * kda_pool_bytes -- bytes of a pool of n_slots slots of [H, K, V] elements
 * of dtype: every size derives from the one dtype decision (ROCm/ATOM PR
 * #2130, What and Memory).  Returns 0 for a refused dtype or a bad size.
 */
size_t kda_pool_bytes(int32_t n_slots, int32_t H, int32_t K, int32_t V,
                      kda_dtype dtype);

/*
 * kda_tile_bv -- value columns per state tile that single-row launches use
 * by default once they are large enough to be bound by bandwidth (more than
 * 128 requests x heads for fp32, 96 for fp16): 128 for fp32 pools (whole
 * 512-byte state rows per wave instruction, K over 2 waves), 64 for fp16
 * (whole 128-byte lines, one wave per tile).  Smaller single-row launches
 * take narrower tiles or more waves by default (kda_describe_launch reports
 * the shape of any launch).  Other widths (32 fp32 / 64 fp16 columns is the V-block cap of
 * the pages' portable kernel, ROCm/ATOM PR #2130, Copilot review) remain
 * available through kda_launch_opts.  Returns a negative kda_status for a
 * refused dtype.
 */
int32_t kda_tile_bv(kda_dtype dtype);

/*
 * kda_prefill -- chunked prefill: whole prompts through the same recurrence
 * as kda_decode_step (ROCm/ATOM PR #2130, What and Depends on: every path,
 * prefill included, reads and writes the state in the pool's dtype while
 * the recurrence runs in fp32; the prefill kernel takes its initial state
 * from the pool, fp16 included).
 *
 * Sequence s owns tokens cu_seqlens[s] .. cu_seqlens[s + 1] - 1.  Its state
 * starts from slot init_slot_ids[s] (widened exactly), every token t is
 * applied in order, out[t] receives scale * S_t^T qn_t, and only the final
 * state is stored, to slot dst_slot_ids[s] (NULL: back to init_slot_ids[s];
 * fp16 pools round to nearest even).  An empty sequence copies its state.
 *
 *  pool           device pool [n_slots, H, 128, 128] of state_dtype.
 *  init_slot_ids  device int32 [n_seq].
 *  dst_slot_ids   NULL or device int32 [n_seq]: distinct, and none is
 *                 another sequence's initial slot (kda_prefill_validate
 *                 checks host copies).
 *  cu_seqlens     device int32 [n_seq + 1], non-decreasing, cu_seqlens[0]
 *                 >= 0, cu_seqlens[n_seq] <= n_tokens.
 *  q, k, g        device fp32 [n_tokens, H, 128], 16-byte aligned; v, out
 *                 device fp32 [n_tokens, H, 128]; b device fp32 [n_tokens, H].
 *  n_seq          sequences (<= n_slots); n_tokens: rows of the token arrays.
 *  opts           NULL or kda_prefill_opts (chunk: 0 = default 32, or 32/64
 *                 tokens per chunk; the chunk changes the rounding order,
 *                 never the operation).
 * The chunked form (per-channel cumulative decay, a unit lower-triangular
 * solve per chunk, matrix-core products) equals the token-by-token
 * recurrence up to rounding.  Device-side, a sequence whose table entries
 * are out of range is skipped (nothing written for it).
 * Errors: as kda_decode_step (KDA_ERR_SLOT: n_seq > n_slots; KDA_ERR_SHAPE
 * also for H > 16384, which keeps byte offsets within a chunk below 2^31),
 * KDA_ERR_ARG (bad chunk, n_tokens < 0, n_seq * H > INT32_MAX, non-finite
 * scale).  Asynchronous on stream.
 */
typedef struct kda_prefill_opts {
  int32_t chunk;
} kda_prefill_opts;

int kda_prefill(const kda_pool* pool, const int32_t* init_slot_ids,
                const int32_t* dst_slot_ids, const int32_t* cu_seqlens, const float* q,
                const float* k, const float* v, const float* g, const float* b, float* out,
                int32_t n_seq, int64_t n_tokens, kda_dtype state_dtype, float scale,
                const kda_prefill_opts* opts, void* stream);

/*
 * kda_prefill_validate -- host-side check of a prefill's tables (host
 * copies): KDA_ERR_NULL, KDA_ERR_ARG (cu_seqlens not non-decreasing from
 * >= 0 to <= n_tokens), KDA_ERR_SLOT (an id out of range, two sequences
 * storing to one slot, or a destination that is another sequence's initial
 * slot), plus the pool checks of kda_validate.  CPU only.
 */
int kda_prefill_validate(const kda_pool* pool, const int32_t* init_slot_ids_host,
                         const int32_t* dst_slot_ids_host, const int32_t* cu_seqlens_host,
                         int32_t n_seq, int64_t n_tokens, kda_dtype state_dtype);

/* ------------------------------------------------------------------------
 * The paged 4-bit key/value cache: what the softmax-attention layers of a
 * hybrid model keep beside the KDA layers' states, for grouped or single query
 * heads.  (The blocks that an fp16 state pool makes room for in ROCm/ATOM
 * PR #2945, Performance, are a latent cache's, another kind.)
 *
 * Format: OCP microscaling MXFP4.  A value is an E2M1 number (0, 0.5, 1, 1.5,
 * 2, 3, 4, 6 and their negatives; the code's high bit is the sign) times
 * 2^(e - 127), with one exponent byte e for 32 channels.  For 32 numbers x,
 *   e = clamp(floor(log2 max|x|) - 2 + 127, 2, 252)
 *   code = x / 2^(e - 127) rounded to nearest, ties to even, at most 6.
 * Exponents 2..252 make every value a normal (or zero) bf16.  4.25 bits a
 * value: 136 bytes for a token's key and value of 128 channels.
 */

/*
 * A cache: device memory holding [n_pages, H] blocks of page_tokens tokens.
 * A block is P * (D + D / 16) bytes (P = page_tokens):
 *   key codes       [P][D / 2]    channels 2i (low half) and 2i + 1 of a byte
 *   value codes     [P][D / 2]
 *   key exponents   [P][D / 32]
 *   value exponents [D / 32][P]
 * page_tokens: 16, 32, 64, 128 or 256; D: 64 or 128; H in [1, 4096]; base
 * 16-byte aligned.  The caller allocates, owns and frees it; it need not be
 * cleared.
 */
typedef struct kda_kv_pool {
  void* base;
  int32_t n_pages;
  int32_t page_tokens;
  int32_t H;
  int32_t D;
} kda_kv_pool;

/* Bytes of a cache; 0 for a shape that is not supported. */
size_t kda_kv_pool_bytes(int32_t n_pages, int32_t page_tokens, int32_t H, int32_t D);

/*
 * The tables every kda_kv_* launch takes (device memory):
 *  page_table  int32 [n_seq, max_pages]: sequence s keeps position p on page
 *              page_table[s][p / page_tokens], at token p % page_tokens.
 *              Entries behind a sequence's last token may hold anything (they
 *              may be read, never used).  max_pages >= 1, and max_pages *
 *              page_tokens <= 2^31 - 4096.
 *  cu_seqlens  int32 [n_seq + 1], non-decreasing: sequence s owns tokens
 *              cu_seqlens[s] .. cu_seqlens[s + 1] - 1 of the launch (none, one,
 *              chained rows or a prompt).  A sequence whose entries are
 *              out of range is skipped; entries that descend may take others
 *              with them (memory outside the tables and tensors is never
 *              touched).  Tokens before the first or behind
 *              the last sequence are left as they were.
 *  cache_lens  int32 [n_seq]: tokens sequence s had before this launch: its
 *              i-th token of the launch is at position cache_lens[s] + i.  The
 *              append and the attention of a step take the same tables.
 *  n_tokens    rows of the token tensors (< 2^31).
 * Token tensors are [n_tokens, heads, D] of `dtype` (KDA_F32, KDA_F16 or
 * KDA_BF16) with D contiguous channels, heads next to each other, and
 * `..._stride` elements from one token to the next (at least heads * D, a
 * multiple of 16 bytes), so that slices of one joint projection can be passed
 * as they lie.  All device pointers 16-byte aligned (the tables: 4-byte).
 * Nothing is allocated or synchronised; launches are captured into graphs as
 * they are.  Calls on different streams may overlap as long as they do not
 * write the same pages, outputs or workspaces, or read pages being written.  A
 * launch of more than 4 million workgroups is KDA_ERR_ARG.
 * Checks run in the order: pool NULL, SHAPE (pool), ARG (counts, max_pages),
 * DTYPE_REFUSED, SHAPE (heads, rot_dim) and ARG (the other numbers), then, for
 * n_seq and n_tokens > 0 (either 0 is a valid no-op), NULL, ARG (strides),
 * ALIGN, the workspace.  KDA_ERR_LAUNCH as everywhere.
 */

/*
 * kda_kv_append -- stores a step's new keys and values, turning keys (and
 * queries) by their positions on the way.
 *
 *  k, v      [n_tokens, H, D]; q: NULL, or [n_tokens, q_heads, D].
 *  q_out     the turned queries, [n_tokens, q_heads, D] without gaps, of
 *            dtype; may be q itself where q has no gaps either.  Not
 *            touched with q_heads == 0.
 *  cos, sin  device fp32 [n_positions, rot_dim / 2], row p for position p; the
 *            first rot_dim channels (a multiple of 16, 0 for no rotation) of
 *            every key and query are turned: pair (a, b) of table column c
 *            becomes (a cos - b sin, b cos + a sin), where (a, b) are channels
 *            (c, c + rot_dim / 2), or with interleaved = 1 (2c, 2c + 1).
 * Queries are turned in fp32 and rounded once; keys are turned and rounded
 * in fp64, so a code next to a rounding border is the definition's.
 * A key or value row (one token, one cached head) that holds a NaN or an
 * infinity poisons that token for that head: its key exponents become 255 (its
 * key reads back as NaN) and its value zeros; rows that see the token get NaN
 * from the attention in that head's outputs, other rows are not changed.
 * A token whose position has no valid page, or lies behind the tables, is not
 * stored, and its q_out rows are NaN.  Two tokens of one launch must not have
 * the same place (kda_kv_validate checks host copies).
 */
int kda_kv_append(const kda_kv_pool* kv, const int32_t* page_table, int32_t max_pages,
                  const int32_t* cu_seqlens, const int32_t* cache_lens, const void* k, const void* v,
                  int64_t k_stride, int64_t v_stride, const void* q, int64_t q_stride, void* q_out,
                  const float* cos, const float* sin, int32_t n_positions, int32_t rot_dim,
                  int32_t interleaved, int32_t n_seq, int64_t n_tokens, int32_t q_heads,
                  kda_dtype dtype, void* stream);

/*
 * kda_kv_read -- the values the cache holds: token i of sequence s gets those
 * of position first[s] + i (moving a prefix to another cache, inspection).
 * k_out, v_out: [n_tokens, H, D] of dtype with strides as above; one of them
 * may be NULL.  Exact in fp32 and bf16; fp16 rounds to nearest even (values
 * from 65520 are infinite there, below 2^-24 zero or rounded).  Tokens without
 * a valid page read as NaN.
 */
int kda_kv_read(const kda_kv_pool* kv, const int32_t* page_table, int32_t max_pages,
                const int32_t* cu_seqlens, const int32_t* first, void* k_out, void* v_out,
                int64_t k_stride, int64_t v_stride, int32_t n_seq, int64_t n_tokens, kda_dtype dtype,
                void* stream);

/*
 * kda_kv_attend -- attention of a launch's rows over the cache, causal: the
 * row at position p sees the sequence's positions 0..p (its own included: the
 * step's tokens are appended first).  Query head i reads cached head
 * i / (q_heads / H).
 *   out = sum_t softmax_t(scale * q . k_t) v_t
 *  q               [n_tokens, q_heads, D]; out: the same without gaps; may be q
 *                  itself where q has no gaps either.
 *  max_rows        the longest sequence's rows in this launch, max_kv_len its
 *                  tokens including them (0: all that max_pages covers).  They
 *                  choose the kernel and lay out its launch; longer sequences
 *                  are taken as well, more slowly.
 *  q_heads         a multiple of H, at most 65535; n_tokens * q_heads / H < 2^29.
 *                  (0..65535 for kda_kv_append.)
 *  scale           finite.
 *  workspace       kda_kv_attend_workspace() bytes for the same arguments (may
 *                  be NULL for 0), 16-byte aligned, free for use again once
 *                  the launch has run.  Calls that may overlap need their own.
 * Cached values enter the matrix cores as they are.  So does q, as 3 (fp32), 2
 * (fp16) or 1 bf16 numbers that add up to it; scores, weights, their sums and the
 * output's sums are fp32, and weights are rounded to nearest, by at most 2^-16 of
 * themselves, where outputs have 16 bits.  Prompts of 16-bit types (more than 64 rows of a
 * sequence and cached head) are multiplied in fp16 where the exponents they meet
 * allow it (104..140, and 2, which zeros have): weights are then rounded to 11
 * bits, in both sums alike, and a bf16 query, divided by its row's power of two, is off by at most
 * 2^-25 of the row's largest channel.  From the first other exponent on, a tile's
 * tokens are multiplied as above (up to 1.6 times the time for a whole prompt).
 * The order of the sums depends on the launch's sizes, not on timing: equal calls
 * give equal bits.
 * Scores are fp32 numbers: a row whose largest score is infinite, of either sign,
 * is NaN (a score that passes the largest fp32 when multiplied by scale, or by a
 * query with an infinity; where q . k alone passes it, bf16 prompts, which take
 * the row's power of two out first, may still hold it).
 * Rows are computed in tiles of up to 128, and where a row's sums are rounded may
 * depend on what its tile's other rows see; nothing else of a row does.
 * A row that sees a poisoned token or a page that does not exist is NaN in
 * that head; the rows of a sequence with a negative length or one that
 * max_pages cannot hold are NaN.  Errors: KDA_ERR_NULL and KDA_ERR_ARG also for
 * a workspace that is missing or too small.
 */
int kda_kv_attend(const kda_kv_pool* kv, const int32_t* page_table, int32_t max_pages,
                  const int32_t* cu_seqlens, const int32_t* cache_lens, const void* q, int64_t q_stride,
                  void* out, int32_t n_seq, int64_t n_tokens, int32_t max_rows, int64_t max_kv_len,
                  int32_t q_heads, kda_dtype dtype, float scale, void* workspace, size_t workspace_bytes,
                  void* stream);

/* Bytes of workspace kda_kv_attend needs for these arguments (0: none, or
 * arguments it refuses). */
size_t kda_kv_attend_workspace(const kda_kv_pool* kv, int32_t max_pages, int32_t n_seq, int64_t n_tokens,
                               int32_t max_rows, int64_t max_kv_len, int32_t q_heads, kda_dtype dtype);

/*
 * kda_kv_validate -- host-side check of a step's tables (host copies): ARG for
 * cu_seqlens that descend or leave [0, n_tokens], a negative length or one
 * that max_pages cannot hold; SLOT for a page that is out of range, or one that
 * takes new tokens and appears twice among the pages in use (pages before a
 * sequence's first new token may be shared).  ARG also when host memory does not
 * hold a list of the written pages.  CPU only.
 */
int kda_kv_validate(const kda_kv_pool* kv, const int32_t* page_table_host, int32_t max_pages,
                    const int32_t* cu_seqlens_host, const int32_t* cache_lens_host, int32_t n_seq,
                    int64_t n_tokens);

/* ------------------------------------------------------------------------
 * Trees of drafted tokens.  A speculative step may offer a target model more
 * than one continuation: the drafted tokens of a request form a tree, each
 * node a token that follows its parent's.  (The pages' own drafts are chains,
 * 1 + 7 rows a request, ROCm/ATOM PR #2945, Method; kda_decode_step takes
 * those, with a snapshot for each row.)  One step over a tree is
 *   kda_kv_append_at, kda_kv_attend_tree   in every softmax-attention layer
 *   kda_decode_tree                        in every KDA layer
 *   kda_verify_drafts                      once, on the target's probabilities
 *   kda_kv_keep, kda_decode_path           the accepted path enters the caches
 *                                          and the states
 * A short convolution in front of a KDA layer is the caller's: a node's window
 * holds its path's inputs, and the accepted path's go into the history.
 * (kda_decode_step_conv has both for chains.)
 *
 * The tables (device int32):
 *  cu_seqlens  [n_req + 1], non-decreasing: request r owns nodes
 *              cu_seqlens[r] .. cu_seqlens[r + 1] - 1 of the launch, up to
 *              KDA_MAX_NODES of them (none: nothing is done for it).  A request
 *              whose entries are out of range is skipped.
 *  parents     [n_tokens]: the parent of the request's node i, counted from the
 *              request's first node: -1 (the node follows the context) or a
 *              node before it, 0 .. i - 1.  Node 0 has -1.  (A chain: i - 1.)
 *  path        [n_req, max_path], path_lens [n_req]: the accepted nodes, from
 *              the root down, as kda_verify_drafts writes them; entries behind
 *              a path's length may hold anything.  max_path in
 *              [1, KDA_MAX_NODES].
 * Rows of nodes before the first or behind the last request are left as they
 * were.  Nothing is allocated or synchronised; launches are captured into
 * graphs as they are.  Calls on different streams may overlap as long as none
 * writes what another one reads or writes.
 */

/*
 * kda_tree_validate -- host-side check of a step's tables (host copies): ARG
 * for cu_seqlens that descend or leave [0, n_tokens], and for a parent that is
 * neither -1 nor before its node; ROWS for a request of more than
 * KDA_MAX_NODES nodes.  CPU only.
 */
int kda_tree_validate(const int32_t* cu_seqlens_host, const int32_t* parents_host, int32_t n_req,
                      int64_t n_tokens);

/*
 * kda_kv_append_at -- kda_kv_append with the positions that keys and queries are
 * turned by given apart from their places.  positions: NULL (then exactly
 * kda_kv_append), or device int32 [n_tokens], 4-byte aligned: token t is turned
 * by row positions[t] of cos and sin and stored at cache_lens[s] + i as ever.
 * A tree's node stands at the context's length plus its depth.  A position
 * outside [0, n_positions) is treated like a token without a page: not stored,
 * its q_out rows NaN.  With rot_dim 0 positions are not read.
 */
int kda_kv_append_at(const kda_kv_pool* kv, const int32_t* page_table, int32_t max_pages,
                     const int32_t* cu_seqlens, const int32_t* cache_lens, const void* k, const void* v,
                     int64_t k_stride, int64_t v_stride, const void* q, int64_t q_stride, void* q_out,
                     const float* cos, const float* sin, const int32_t* positions, int32_t n_positions,
                     int32_t rot_dim, int32_t interleaved, int32_t n_seq, int64_t n_tokens, int32_t q_heads,
                     kda_dtype dtype, void* stream);

/*
 * kda_kv_attend_tree -- kda_kv_attend for a tree's nodes: node i of sequence s,
 * cached at position cache_lens[s] + i, sees the cache_lens[s] tokens of the
 * context, the nodes on its path and itself.  Everything else is
 * kda_kv_attend's; workspace: kda_kv_attend_tree_workspace() bytes for the same
 * arguments.  So is the precision, more than 64 rows of a sequence and cached head
 * (max_rows * q_heads / H) counting as a prompt, but for fp16 weights, which then keep
 * 22 bits, not 11 (down to 2^-32 of the largest).
 *  parents   device int32 [n_tokens], 4-byte aligned (see above).
 *  max_rows  at most KDA_MAX_NODES (else KDA_ERR_ROWS, checked with the counts).
 * The rows of a sequence of more than KDA_MAX_NODES nodes, or with a parent
 * that does not lie before its node, are NaN.
 */
int kda_kv_attend_tree(const kda_kv_pool* kv, const int32_t* page_table, int32_t max_pages,
                       const int32_t* cu_seqlens, const int32_t* cache_lens, const int32_t* parents,
                       const void* q, int64_t q_stride, void* out, int32_t n_seq, int64_t n_tokens,
                       int32_t max_rows, int64_t max_kv_len, int32_t q_heads, kda_dtype dtype, float scale,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace kda_kv_attend_tree needs for these arguments (0: none, or
 * arguments it refuses). */
size_t kda_kv_attend_tree_workspace(const kda_kv_pool* kv, int32_t max_pages, int32_t n_seq, int64_t n_tokens,
                                    int32_t max_rows, int64_t max_kv_len, int32_t q_heads, kda_dtype dtype);

/*
 * kda_kv_keep -- moves the cache entries of accepted nodes together: node
 * path[s][e], cached at position cache_lens[s] + path[s][e], to position
 * cache_lens[s] + e, for every e < path_lens[s], bytes as they are.  The caller
 * then counts path_lens[s] more tokens in cache_lens[s].
 *  path must ascend (a path from the root down does); a path that does not,
 *  that names a node the sequence does not have, or whose length is outside
 *  [0, max_path], leaves its sequence as it was.
 * A token whose source has no page becomes a poisoned one (it reads back as
 * NaN); one whose destination has none is not moved.  Checks as kda_kv_read's,
 * with ROWS (max_path) behind the counts.
 */
int kda_kv_keep(const kda_kv_pool* kv, const int32_t* page_table, int32_t max_pages,
                const int32_t* cu_seqlens, const int32_t* cache_lens, const int32_t* path, int32_t max_path,
                const int32_t* path_lens, int32_t n_seq, int64_t n_tokens, void* stream);

/*
 * kda_decode_tree -- the recurrence of kda_decode_step over trees: a node starts
 * from its parent's state (the roots from slot init_slot_ids[r], widened
 * exactly), is updated by its own q, k, v, g, b, and out receives its read-out.
 * All states between are fp32 and none is stored: the pool is only read, so a
 * rejected branch leaves nothing to undo.
 *  init_slot_ids  device int32 [n_req], may repeat; a request whose slot is
 *                 out of range has NaN rows.
 *  q, k, g, v     device fp32 [n_tokens, H, 128]; b device fp32 [n_tokens, H];
 *  out            device fp32 [n_tokens, H, 128], apart from every input.
 *  max_nodes      the most nodes of a request, in [0, KDA_MAX_NODES]: it chooses
 *                 the kernel.  A request with more nodes has NaN rows, as has one
 *                 with a parent that does not lie before its node.
 * g <= 0 as everywhere: decays multiply along a path, from the node up.
 * Checks run in the order: pool NULL, DTYPE_REFUSED, DTYPE_MISMATCH, SHAPE (also
 * H > 16384), ARG (counts), ROWS (max_nodes), then, for n_req and n_tokens > 0
 * (either 0 is a valid no-op), NULL, ARG (scale, launch size), ALIGN.
 */
int kda_decode_tree(const kda_pool* pool, const int32_t* init_slot_ids, const int32_t* cu_seqlens,
                    const int32_t* parents, const float* q, const float* k, const float* v,
                    const float* g, const float* b, float* out, int32_t n_req, int64_t n_tokens,
                    int32_t max_nodes, kda_dtype state_dtype, float scale, void* stream);

/*
 * kda_decode_path -- the accepted nodes' updates applied in turn: the state of
 * slot init_slot_ids[r] takes the k, v, g, b rows of nodes path[r][0],
 * path[r][1], .. and is stored to slot dst_slot_ids[r] (NULL: back to
 * init_slot_ids[r]; fp16 pools round to nearest even, once).  A path of length
 * 0 copies the state.  dst_slot_ids: distinct, and none is another request's
 * initial slot (kda_prefill_validate checks host copies).  A request with a slot
 * out of range, a length outside [0, max_path], or a path entry that is not one
 * of its nodes, is skipped: nothing is stored for it.
 * Checks as kda_decode_tree's (ROWS: max_path outside [1, KDA_MAX_NODES]; SLOT:
 * n_req > n_slots, behind it), but only n_req 0 is a no-op; k, v, g and b may be
 * NULL with n_tokens 0.
 */
int kda_decode_path(const kda_pool* pool, const int32_t* init_slot_ids, const int32_t* dst_slot_ids,
                    const int32_t* cu_seqlens, const int32_t* path, int32_t max_path,
                    const int32_t* path_lens, const float* k, const float* v, const float* g,
                    const float* b, int32_t n_req, int64_t n_tokens, kda_dtype state_dtype, void* stream);

/*
 * kda_verify_drafts -- which drafted tokens are kept, and the token that follows
 * them, so that every token is distributed as the target's probabilities say
 * (rejection sampling from given random numbers).
 *
 * A request's walk starts at node 0, which is certain, with weights f = the
 * target's row of node 0 and M = 1.  Its nodes 1, 2, .. are looked at in turn;
 * node i is tried if its parent is the last accepted node.  With x =
 * tokens[i], u = accept_rand[i] and q the draft's row of that parent:
 *   accepted if u q(x) M < f(x): then f = target's row of node i, M = 1;
 *   else f <- max(f - M q, 0), M <- sum f.
 * (q: the distribution that each child of that node was drawn from.)  Without
 * a draft, for children that are chosen and not drawn (the draft's likeliest):
 *   accepted if u M < f(x); else M <- M - f(x), f(x) <- 0.
 * Last, the following token is the smallest x with f(x) > 0 and f(0) + .. + f(x)
 * > sample_rand[r] * (sum f); the last with f(x) > 0 if rounding leaves none;
 * drawn from the target's row itself if sum f is 0.
 * All of it in fp64 on the stored probabilities, so that a draw next to a
 * border is the definition's; an entry that is not above 0 (NaN among them)
 * counts as 0, and a token outside [0, vocab) has probability 0.
 *
 *  target       device [n_tokens, vocab] of dtype (KDA_F32, KDA_F16 or KDA_BF16),
 *               target_stride (>= vocab) elements from row to row: row i is the
 *               distribution behind node i.  Not rescaled: acceptance takes the
 *               rows as normalised.
 *  draft        NULL, or the same of the draft (draft_stride not read with NULL).
 *  tokens       device int32 [n_tokens]; node 0's is not read.
 *  accept_rand  device fp32 [n_tokens], in [0, 1); sample_rand fp32 [n_req].
 *  path         int32 [n_req, max_path], out: node 0 and the accepted nodes, then
 *               -1.  A path that fills max_path ends there, and its last node's
 *               children are not tried.
 *  path_lens    int32 [n_req], out: at least 1; 0 for a request without nodes,
 *               or one that is skipped (its path -1), whose tree is bad, or which
 *               has more than KDA_MAX_NODES nodes.
 *  next_tokens  int32 [n_req], out: the following token; -1 for a request of
 *               length 0, and where the last row has no weight or an infinite one.
 *  workspace    kda_verify_workspace() bytes (may be NULL for 0), 8-byte aligned,
 *               free for use again once the launch has run.
 * Probabilities and rows may have any alignment of their type.  Equal calls give
 * equal results.  Checks run in the order: DTYPE_REFUSED, ARG (counts, vocab < 1),
 * ROWS (max_path), then, for n_req > 0 (0 is a valid no-op; n_tokens 0 leaves
 * lengths of 0), NULL, ARG (strides), ALIGN, the workspace (NULL, ARG).
 */
int kda_verify_drafts(const void* target, int64_t target_stride, const void* draft, int64_t draft_stride,
                      const int32_t* cu_seqlens, const int32_t* parents, const int32_t* tokens,
                      const float* accept_rand, const float* sample_rand, int32_t* path, int32_t max_path,
                      int32_t* path_lens, int32_t* next_tokens, int32_t n_req, int64_t n_tokens,
                      int32_t vocab, kda_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace kda_verify_drafts needs (0: none, or arguments it refuses). */
size_t kda_verify_workspace(int32_t n_req, int64_t n_tokens, int32_t vocab, int32_t max_path, kda_dtype dtype);

/* Launch shape kda_decode_step uses for a given problem (host only). */
typedef struct kda_launch_desc {
  int32_t bv;              /* value columns per workgroup */
  int32_t waves_per_tile;  /* wavefronts per workgroup */
  int32_t threads;         /* threads per workgroup */
  int32_t tiles;           /* n_req * H * (V / bv) */
  int32_t blocks;          /* workgroups launched */
  int32_t lds_bytes;       /* static LDS per workgroup */
  const char* kernel;      /* kernel symbol family name */
  int32_t rows_layout;     /* KDA_ROWS_K_SPLIT, _WAVE_K or _MATRIX (one row: K_SPLIT) */
} kda_launch_desc;

/* Fills *desc for (n_req, n_rows, H, dtype) under opts (NULL = defaults).
 * Errors: KDA_ERR_NULL, KDA_ERR_DTYPE_REFUSED, KDA_ERR_SHAPE (H < 1),
 * KDA_ERR_ROWS, KDA_ERR_ARG. */
int kda_describe_launch(int32_t n_req, int32_t n_rows, int32_t H,
                        kda_dtype dtype, const kda_launch_opts* opts,
                        kda_launch_desc* desc);

/*
 * kda_tile_of_block -- the tile a workgroup processes.  Workgroups are
 * handed to the 8 XCDs of the chip round-robin; this maps them so that the
 * workgroups one XCD runs hold consecutive tiles (the tiles of one
 * (request, head) share that XCD's L2 for q, k, g).  A bijection of
 * [0, n_blocks).  Returns -1 for block out of range.
 */
int32_t kda_tile_of_block(int32_t block, int32_t n_blocks);

/*
 * kda_copy_probe -- measurement helper: copies `bytes` (a multiple of 16)
 * from src to dst with a plain streaming kernel of the same load/store
 * width as the decode kernel, on `stream`.  Used to calibrate achievable
 * bandwidth and hardware byte counters.  Both pointers 16-byte aligned.
 */
int kda_copy_probe(void* dst, const void* src, size_t bytes, void* stream);

/*
 * kda_bw_probe -- measurement helper: a streaming kernel over `bytes` (a
 * multiple of 16) on `stream`, to set the decode's bandwidth against what the
 * GPU reaches on plain traffic (ROCm/ATOM PR #2130, What: the production
 * kernel is quoted at 71-90% of "achievable" bandwidth, which the pages leave
 * undefined).
 *  mode                KDA_PROBE_COPY: read src, write dst; KDA_PROBE_READ:
 *                      read src only (dst must be a 16-byte device buffer it
 *                      never writes in practice); KDA_PROBE_WRITE: write dst
 *                      only (src may be NULL).
 *  vectors_per_thread  1, 2 or 4 16-byte vectors per thread, all loads
 *                      issued before the first store; consecutive threads
 *                      on consecutive vectors.
 *  nontemporal         non-zero: loads and stores carry the nontemporal
 *                      hint, as the decode's state traffic does.
 * Both pointers 16-byte aligned; src and dst hold at least `bytes` (dst 16
 * bytes for KDA_PROBE_READ).  Errors: KDA_ERR_NULL, KDA_ERR_ALIGN,
 * KDA_ERR_ARG (mode, vectors_per_thread, bytes), KDA_ERR_LAUNCH.
 */
#define KDA_PROBE_COPY 0
#define KDA_PROBE_READ 1
#define KDA_PROBE_WRITE 2
int kda_bw_probe(void* dst, const void* src, size_t bytes, int32_t mode,
                 int32_t vectors_per_thread, int32_t nontemporal, void* stream);

/*
 * kda_tile_probe -- measurement helper: the memory traffic of a single-row
 * decode launch over n_req requests with the arithmetic taken out.  Same grid
 * and block-to-tile map as kda_decode_step at its default shape for launches
 * bound by bandwidth (kda_tile_bv columns; fp32 2 waves, fp16 1 wave), same
 * slot id load, lane layout and 16-byte nontemporal loads; each tile is
 * written back unchanged, in place, to slot_ids[r].  slot_ids: device int32
 * [n_req]; an id out of range skips its request.  Errors: as kda_state_copy
 * for the pool; KDA_ERR_ARG (n_req outside [0, n_slots]).
 */
int kda_tile_probe(const kda_pool* pool, const int32_t* slot_ids, int32_t n_req,
                   kda_dtype state_dtype, void* stream);

/*
 * kda_rows_probe -- measurement helper: the memory traffic of a chained-row
 * launch in the matrix-core block form (KDA_ROWS_MATRIX at its default 8
 * waves: 64-column halves, K over the waves) with the arithmetic taken out.
 * Same grid, block-to-tile map, slot id loads, lane layout and nontemporal
 * loads and stores as kda_decode_step there; each request's initial state
 * (init_slot_ids[r], or slot_ids[r * n_rows] if init_slot_ids is NULL) is
 * written unchanged to each of its rows' slots slot_ids[r * n_rows + t].
 *  slot_ids       device int32 [n_req * n_rows]; init_slot_ids: NULL or
 *                 device int32 [n_req].  A request with an id out of range
 *                 is skipped.
 *  tile_cols, waves  the workgroup's value columns and waves: 0, 0 or 64, 8
 *                 (the block form), 32 or 128 over 8 waves (narrower and
 *                 wider tiles, each lane still 4 columns of a row), or 128
 *                 over 16 waves (two 64-column halves of 8, the fused
 *                 convolution's whole-head form).
 * Errors: as kda_tile_probe; KDA_ERR_ROWS (n_rows outside [1,
 * KDA_MAX_ROWS]); KDA_ERR_ARG (n_req < 0, n_req * n_rows > n_slots, or
 * another tile shape).
 */
int kda_rows_probe(const kda_pool* pool, const int32_t* slot_ids, const int32_t* init_slot_ids,
                   int32_t n_req, int32_t n_rows, int32_t tile_cols, int32_t waves,
                   kda_dtype state_dtype, void* stream);

/* Message for a kda_status code (static string, never NULL). */
const char* kda_strerror(int code);

/* KDA_ABI_VERSION of the built library. */
int kda_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_DECODE_H */
