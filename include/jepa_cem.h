/*
 * jepa_cem.h -- C ABI of the GB300 (sm_103a) CEM planner over an action-conditioned
 * JEPA world-model predictor.
 *
 * What it computes follows "Real-time inference for JEPA world-model architectures
 * with Ray", section "Where the sixteen seconds actually goes": in each of R rounds a
 * planning step samples N action sequences from a Gaussian, predicts with the world
 * model where each one leads, measures how far each predicted embedding lies from the
 * goal embedding and refits the Gaussian to the K closest; the caller receives only
 * the first action of the closest sequence of the last round. Section "Measured on 8x A100" adds that the
 * predictor attends only to current and earlier frames (so keys and values cached between
 * rollout steps stay exact), that it
 * runs in bf16 with flash attention, and that the same seed gives the same plan
 * however the candidates are batched.
 *
 * Conventions for every entry point:
 *   - Tensors are dense, row-major, float32 unless stated. Shapes use
 *     B problems, N candidates, H horizon steps, A action dim, S state dim,
 *     P patch tokens per frame, E embedding dim.
 *   - Pointers marked "dev" are device pointers on the context's device. Pointers
 *     marked "dev|host" may be device memory or host memory (pinned or pageable);
 *     the library copies them with cudaMemcpyAsync(cudaMemcpyDefault).
 *   - The caller owns every buffer it passes; the context owns weights, workspaces
 *     and captured CUDA graphs. Nothing passed in is retained after the call returns
 *     except through the stream's pending work.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream). Work is enqueued
 *     asynchronously; outputs are valid once the stream has been synchronised.
 *   - Every call returns a jepa_status and never aborts the process. After an error
 *     the output contents are unspecified; the context stays usable and
 *     jepa_last_error() describes the failure. A context must not be used from two
 *     host threads at once.
 */
#ifndef JEPA_CEM_H_
#define JEPA_CEM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  JEPA_OK = 0,
  JEPA_ERR_INVALID_ARG = 1,  /* NULL pointer, non-positive size, K > N, ... */
  JEPA_ERR_SHAPE = 2,        /* shape outside what the context was created for */
  JEPA_ERR_NOT_LOADED = 3,   /* weights not loaded yet */
  JEPA_ERR_OOM = 4,          /* device allocation failed */
  JEPA_ERR_CUDA = 5,         /* a CUDA runtime/driver call failed */
  JEPA_ERR_TIMEOUT = 6,      /* a bounded device-side wait gave up (kernel returned early) */
  JEPA_ERR_UNSUPPORTED = 7   /* device is not sm_103 / feature not built */
} jepa_status;

/* FP8: the bf16 path with the GEMMs fed by a LayerNorm (QKV, MLP up, projection to E) on
 * fp8 e4m3 operands (kind::f8f6f4): weights with one scale per output channel, the
 * LayerNorm output with one scale per row; everything else as in BF16. (The planning
 * page's "Further Optimization", D, and the Realtime-VLA notes, 9.1, name 8-bit
 * quantisation of the predictor as the way to shrink its compute.) */
typedef enum { JEPA_FP32 = 0, JEPA_BF16 = 1, JEPA_FP8 = 2 } jepa_precision;

/* MLP of each layer. GELU: u = GELU(W_1 h + b_1). GATED (the Realtime-VLA notes, section 4.2
 * "Fusing Gated Linear Layers": FC1(x, w1) * GELU(FC2(x, w2))): u = (W_1 h + b_1) *
 * GELU(W_g h + b_g), computed by one GEMM over the two weight matrices' rows interleaved in
 * blocks of 32, whose epilogue writes only the product. */
typedef enum { JEPA_MLP_GELU = 0, JEPA_MLP_GATED = 1 } jepa_mlp_kind;

/* Predictor shape. Pre-LN transformer, block-causal over frame blocks of
 * T = patch_tokens + 2 tokens ([action, state, P patches]). */
typedef struct {
  int32_t layers;        /* L */
  int32_t width;         /* d, multiple of 32 (bf16: multiple of 64) */
  int32_t heads;         /* h; head dim d/h = 64 in bf16 mode, <= 128 in fp32 mode */
  int32_t mlp;           /* m, hidden width of the MLP (bf16 gated: multiple of 128) */
  int32_t patch_tokens;  /* P */
  int32_t embed_dim;     /* E, multiple of 32 (bf16: multiple of 64) */
  int32_t action_dim;    /* A (7 in the planning workloads) */
  int32_t state_dim;     /* S (7) */
  int32_t max_horizon;   /* largest H any call will use; sizes the KV cache */
  int32_t precision;     /* jepa_precision: FP32 = SIMT fp32 path, BF16 = tensor-core path,
                            FP8 = tensor-core path with fp8 LayerNorm-fed GEMMs */
  float ln_eps;          /* LayerNorm epsilon (1e-5) */
  int32_t max_chunk;     /* candidates per predictor pass (0 = library default); bounds workspace */
  int32_t mlp_kind;      /* jepa_mlp_kind */
} jepa_config;

typedef struct jepa_ctx jepa_ctx;

/* Optional per-round record of a plan. All device pointers; each may be NULL. */
typedef struct {
  float* mu;        /* [R+1, B, H, A]  mu_0 .. mu_R */
  float* sigma;     /* [R+1, B, H, A]  sigma_0 .. sigma_R */
  float* actions;   /* [R, B, N, H, A] clipped candidates of each round */
  float* energy;    /* [R, B, N]       energies of each round */
  int32_t* elites;  /* [R, B, K]       elite indices, ascending (energy, index) */
  int32_t* winner;  /* [B]             winner of the final round */
} jepa_cem_trace;

/* Create a context on CUDA device `device` for predictor shape *cfg.
 * Fails with JEPA_ERR_UNSUPPORTED unless the device is compute capability 10.3. */
jepa_status jepa_create(const jepa_config* cfg, int device, jepa_ctx** out);

/* Free the context and everything it owns. Synchronises the device first. NULL is a no-op. */
void jepa_destroy(jepa_ctx* ctx);

/* Text of the last error on this context ("" if none). Valid until the next call on ctx. */
const char* jepa_last_error(const jepa_ctx* ctx);

/* Static name of a status code. */
const char* jepa_status_string(jepa_status s);

/* Size in bytes of the weight blob for *cfg: a 64-byte header (int32 magic 0x4150454A,
 * version 1, layers, width, heads, mlp, patch_tokens, embed_dim, action_dim, state_dim,
 * mlp_kind, then zeros) followed by float32 tensors in this order, each row-major [out, in]:
 * W_in[d,E] b_in[d] W_a[d,A] b_a[d] W_s[d,S] b_s[d] pos[T,d], per layer
 * {ln1_g[d] ln1_b[d] W_qkv[3d,d] b_qkv[3d] W_o[d,d] b_o[d] ln2_g[d] ln2_b[d]
 *  W_1[m,d] b_1[m] (gated only: W_g[m,d] b_g[m]) W_2[d,m] b_2[d]},
 * lnf_g[d] lnf_b[d] W_out[E,d] b_out[E]. */
size_t jepa_weight_blob_bytes(const jepa_config* cfg);

/* Upload predictor weights from a host blob (format above). Validates the header
 * against the context's config (JEPA_ERR_SHAPE on mismatch), converts the GEMM
 * matrices to bf16 in bf16 mode, and blocks until the upload is done. On error the
 * previously loaded weights (if any) stay in place. */
jepa_status jepa_load_weights(jepa_ctx* ctx, const void* host_blob, size_t bytes);

/* Candidate sampler (the planning page, "Where the sixteen seconds actually goes": each
 * round's candidate action sequences are drawn from a Gaussian around the current guess).
 *   mu, sigma [B,H,A] dev; actions [B,N,H,A] dev (output).
 * eps[b,n,h,j] comes from Philox4x32-10 with key (seed lo, seed hi) and counter
 * (n, b, round*Q + q, 0), Q = ceil(H*A/4), q = (h*A+j)/4, word (h*A+j)%4, turned into
 * normals by Box-Muller on u = ((x>>9)+0.5)*2^-23 (cos for words 0/2, sin for 1/3);
 * actions = clip(mu + sigma*eps, -1, 1). Draws depend only on (seed, b, n, round, h, j). */
jepa_status jepa_sample_actions(jepa_ctx* ctx, const float* mu, const float* sigma, int B, int N,
                                int H, int round, uint64_t seed, float* actions, void* stream);

/* The sampler's generator alone: out[i] = Philox4x32-10(counter[i], key = (seed lo, seed hi)),
 * the four 32-bit output words of counter words counters[4i .. 4i+3] (uint32, dev; n >= 1).
 * Exposed so that integer outputs can be compared bit for bit. */
jepa_status jepa_philox4x32_10(jepa_ctx* ctx, const uint32_t* counters, uint64_t seed, int n,
                               uint32_t* out, void* stream);

/* Predictor rollout and L1 energy (the step of the same section that rolls every candidate
 * through the predictor and scores the outcome against the goal embedding; frame-causal
 * with a KV cache).
 *   z_ctx [B,P,E] dev   encoded context frame of each problem
 *   state0 [B,S] dev    state of each problem (s_k = s_{k-1} + a_{k-1})
 *   actions [B,N,H,A] dev
 *   goal [B,P,E] dev or NULL
 *   z_pred [B,N,P,E] dev or NULL   output: the last predicted frame z_H
 *   energy [B,N] dev or NULL       output: mean |z_H - goal| (needs goal)
 * 1 <= H <= cfg.max_horizon. */
jepa_status jepa_predictor_forward(jepa_ctx* ctx, const float* z_ctx, const float* state0,
                                   const float* actions, int B, int N, int H, const float* goal,
                                   float* z_pred, float* energy, void* stream);

/* Elite selection and Gaussian refit (the same section: the best K candidates are kept and
 * the Gaussian is moved onto them): per problem, the K lowest energies ordered by
 * (energy, index), NaN last; then
 * mu' = elite mean and sigma' = elite population std per (h, j).
 *   energy [B,N] dev; actions [B,N,H,A] dev; mu_out, sigma_out [B,H,A] dev (outputs);
 *   elites_out [B,K] int32 dev or NULL. 1 <= K <= N <= 8192. */
jepa_status jepa_cem_select_refit(jepa_ctx* ctx, const float* energy, const float* actions, int B,
                                  int N, int H, int K, float* mu_out, float* sigma_out,
                                  int32_t* elites_out, void* stream);

/* One full planning step: R rounds of sample -> predictor -> energy -> select/refit with
 * no host round-trip between rounds (one captured CUDA graph per (B,H,N,K,R), cached in
 * the context), then action_out[b] = first action of problem b's lowest-energy
 * candidate in the final round.
 *   z0, goal [B,P,E], state0 [B,S], mu0, sigma0 [B,H,A]: dev|host inputs
 *   action_out [B,A]: dev|host output
 *   trace: NULL or per-round record (device pointers, see jepa_cem_trace)
 * The first call for a new (B,H,N,K,R) allocates workspace and captures the graph. */
jepa_status jepa_cem_plan(jepa_ctx* ctx, const float* z0, const float* state0, const float* goal,
                          const float* mu0, const float* sigma0, int B, int H, int N, int K,
                          int rounds, uint64_t seed, float* action_out,
                          const jepa_cem_trace* trace, void* stream);

/* Warm start of the next planning step under receding-horizon control (planning page,
 * section "Further Optimization", B "Warm-started CEM": only the first action of a plan is
 * executed, and the rest of it may seed the next step instead of a fresh Gaussian).
 *   mu_prev [B,H,A] dev        the previous plan's last-round mean (the slice
 *                              trace->mu + rounds*B*H*A of jepa_cem_plan's trace)
 *   mu_prior, sigma_prior [B,H,A] dev   the fresh Gaussian
 *   mu_out, sigma_out [B,H,A] dev       outputs; mu_out may equal mu_prev and sigma_out may
 *                                       equal sigma_prior (no other overlap)
 * mu_out[b,h] = mu_prev[b,h+1] for h < H-1, mu_out[b,H-1] = mu_prior[b,H-1];
 * sigma_out = sigma_prior. With H = 1 this is the prior itself. */
jepa_status jepa_cem_warm_start(jepa_ctx* ctx, const float* mu_prev, const float* mu_prior,
                                const float* sigma_prior, int B, int H, float* mu_out,
                                float* sigma_out, void* stream);

/* One step of the world model playing the robot, as in that section's closed-loop
 * experiments: the executed action goes through the predictor with horizon 1.
 *   z [B,P,E], state [B,S], action [B,A]: dev inputs
 *   z_next [B,P,E] dev   output: the predicted next frame (must not overlap z)
 *   state_next [B,S] dev output: state + action (may equal state)
 *   goal [B,P,E] dev or NULL; distance [B] dev or NULL: mean |z_next - goal| (needs goal) */
jepa_status jepa_world_model_step(jepa_ctx* ctx, const float* z, const float* state,
                                  const float* action, int B, const float* goal, float* z_next,
                                  float* state_next, float* distance, void* stream);

/* Closed-loop episode: `steps` times (plan with jepa_cem_plan, execute the winner's first
 * action with jepa_world_model_step, replan from the predicted frame), all enqueued on
 * `stream` with no host synchronisation between steps. Step t plans with seed + t and
 * starts from the prior (warm = 0) or, for t >= 1, from jepa_cem_warm_start of step t-1's
 * last-round mean (warm = 1).
 *   z0, goal [B,P,E], state0 [B,S], mu_prior, sigma_prior [B,H,A]: dev|host inputs
 *   actions_out [steps,B,A]: dev|host output, the executed actions
 *   distance_out [steps,B]: dev|host output, mean |z_{t+1} - goal| after each action
 * Workspace for the episode is kept in the context and grows on demand (the first call
 * with larger sizes synchronises the device). */
jepa_status jepa_cem_closed_loop(jepa_ctx* ctx, const float* z0, const float* state0,
                                 const float* goal, const float* mu_prior,
                                 const float* sigma_prior, int B, int H, int N, int K, int rounds,
                                 int steps, int warm, uint64_t seed, float* actions_out,
                                 float* distance_out, void* stream);

/* Number of kernel launches one jepa_cem_plan call with these sizes makes (captures
 * the graph if needed). */
jepa_status jepa_plan_kernel_count(jepa_ctx* ctx, int B, int H, int N, int K, int rounds,
                                   int64_t* count);

/* Dense linear layer on the tensor-core GEMM used by the predictor (bf16 in, fp32
 * accumulate): out[M,N] = act(A[M,K] * W[N,K]^T + bias[N]).
 *   A, W: bf16 bit patterns (uint16) dev; bias [N] dev or NULL; out [M,N] float32 dev.
 *   gelu: 0 = identity, 1 = erf GELU, 2 = gated: W's rows are FC1 and gate blocks of 32
 *   interleaved (rows 64p..64p+31 = FC1 rows 32p.., rows 64p+32..64p+63 = gate rows 32p..),
 *   bias interleaved the same way (required), N a multiple of 256, and
 *   out[M,N/2][32p + c] = (acc[64p + c] + bias) * GELU(acc[64p + 32 + c] + bias).
 * K a multiple of 8. Needs a bf16 context. */
jepa_status jepa_linear_bf16(jepa_ctx* ctx, const uint16_t* A, const uint16_t* W,
                             const float* bias, int M, int N, int K, int gelu, float* out,
                             void* stream);

/* The residual GEMM of the predictor on caller data (the attention out-projection and the
 * MLP down-projection of a pre-LN block, "Real-time inference for JEPA world-model
 * architectures with Ray", the predictor of section "Measured on 8x A100"):
 *   x[M,N] += A[M,K] * W[N,K]^T + bias[N], fp32 accumulation, x fp32 updated in place.
 *   A, W: bf16 bit patterns dev, 16-byte aligned; bias [N] dev or NULL; x [M,N] fp32 dev.
 *   K a multiple of 8, N a multiple of 4. Needs a bf16 context. */
jepa_status jepa_linear_resid_bf16(jepa_ctx* ctx, const uint16_t* A, const uint16_t* W,
                                   const float* bias, int M, int N, int K, float* x,
                                   void* stream);

/* The QKV GEMM of the predictor on caller data, writing one rollout step's rows into the
 * candidates' K/V caches (KV cache across rollout steps, the planning page, "Measured on
 * 8x A100"): acc = A[M,K] * W[3d,K]^T + bias[3d] (fp32), rounded to bf16, and for each
 * row r < M, with candidate c = r / T and t = r % T,
 *   q[r, 0:d] = acc[r, 0:d],   kv[c][frame*T + t][0:2d] = acc[r, d:3d].
 * Other rows of kv are not written.
 *   A, W: bf16 bit patterns dev, 16-byte aligned; bias [3d] dev or NULL;
 *   q [M, d] and kv [ceil(M/T)][kv_rows][2d]: bf16 bit patterns dev.
 *   d a multiple of 32, K a multiple of 8, T >= 1, 0 <= frame, (frame + 1) * T <= kv_rows.
 * Needs a bf16 context. */
jepa_status jepa_linear_qkv_bf16(jepa_ctx* ctx, const uint16_t* A, const uint16_t* W,
                                 const float* bias, int M, int d, int K, int T, int kv_rows,
                                 int frame, uint16_t* q, uint16_t* kv, void* stream);

/* The fp8 GEMM of the FP8 mode on caller data: out[M,N] = act((A[M,K] * W[N,K]^T) *
 * a_scale[M] (rows) * w_scale[N] (columns) + bias[N]), A and W e4m3 codes (one byte each,
 * OCP E4M3: bias 7, no infinities, largest 448), fp32 accumulation, fp32 output.
 *   gelu: 0 identity, 1 erf GELU, 2 gated (as jepa_linear_bf16; out [M, N/2]).
 *   K a multiple of 16; A, W 16-byte aligned dev; scales and bias dev. Needs a BF16 or FP8
 *   context. */
jepa_status jepa_linear_fp8(jepa_ctx* ctx, const uint8_t* A, const float* a_scale,
                            const uint8_t* W, const float* w_scale, const float* bias, int M,
                            int N, int K, int gelu, float* out, void* stream);

/* Row-wise fp8 quantisation, the rule of the FP8 mode: per row r, scales[r] = max|x[r,:]| /
 * 448 (1 for an all-zero row) and codes[r,c] = e4m3(x[r,c] * (448 / max|x[r,:]|)), rounded to
 * nearest even and saturated (fp32 arithmetic: the division and the product each rounded).
 *   x [rows, cols] float32 dev; codes [rows, cols] uint8 dev; scales [rows] float32 dev. */
jepa_status jepa_quantize_rows_fp8(jepa_ctx* ctx, const float* x, int rows, int cols,
                                   uint8_t* codes, float* scales, void* stream);

/* Block-causal attention of one rollout step as the predictor runs it (bf16 mode): for each
 * candidate c and head h, queries q[c*T + t, h*64 : h*64+64] attend to cached key / value
 * rows [0, Lk) of kv[c] (keys at columns [h*64, h*64+64), values at [d + h*64, ...)) with
 * scale 1/8: out[c*T + t, h*64 + j] = sum_i softmax_i(q . k_i / 8) v_i[j]. (Frame-causal
 * predictor with a KV cache, the planning page, "Measured on 8x A100".)
 *   q [ncand*T, d], kv [ncand][kv_rows][2d], out [ncand*T, d]: bf16 bit patterns, dev.
 *   1 <= Lk <= kv_rows; d = heads * 64; rows of kv past Lk must hold finite values.
 * Runs the predictor's tcgen05 attention kernel. Needs a bf16 context. */
jepa_status jepa_attention_bf16(jepa_ctx* ctx, const uint16_t* q, const uint16_t* kv, uint16_t* out,
                                int ncand, int T, int Lk, int kv_rows, int heads, int d,
                                void* stream);

/* ---- 8-bit paged key/value cache, and attention over it and over packed prompts ----
 *
 * For histories longer than the planner's dense per-candidate caches hold well: sequences of
 * different lengths share one pool of pages, keys and values take a byte an element, and
 * sequences with a common context may name the same pages. Serving only (no gradients). All of
 * these entry points need a bf16 (or fp8) context (jepa_rope_table any) and no weights, enqueue on `stream`, allocate
 * nothing, and can be captured into a CUDA graph; what they read from the device (offsets,
 * lengths, page tables) is read when the graph runs. Tensors are bf16 bit patterns (uint16).
 * Token rows are [tokens][heads][head_dim] with `*_stride` elements between tokens (at least
 * heads * head_dim, a multiple of 8), so q, k and v may be slices of one projection's rows. What a
 * call writes overlaps nothing that it reads, but where it says so.
 *
 * Packed sequences: `cu` [batch + 1] int32 dev, ascending; sequence b owns packed tokens cu[b] ..
 * cu[b+1] - 1 (none is fine). Output rows ahead of the first sequence and behind the last are left
 * as they were.
 *
 * A page index, position, length or offset on the device that lies outside its buffer is never
 * followed: what depends on it is skipped or read as zero (those outputs are unspecified), and
 * the next jepa_sync_check reports JEPA_ERR_INVALID_ARG. A sequence whose two offsets descend or lie
 * outside [0, tokens] is skipped as a whole. */

/* One layer's cache. k, v [num_pages][kv_heads][page_size][head_dim] e4m3 codes; k_scale,
 * v_scale [num_pages][kv_heads] float32: an element stands for code * scale. page_table
 * [batch][max_pages] int32: token t of sequence b lies in page page_table[b][t / page_size],
 * slot t % page_size; entries past a sequence's length are not read. head_dim 64 or 128,
 * page_size 16, 32, 64 or 128, max_pages * page_size <= 2^30, num_pages * kv_heads < 2^31, batch at
 * most 65535, kv_heads at most 1024; k and v 16-byte aligned. Scales lie in [2^-40, 2^40] (others are read as the nearer end, NaN as the
 * least); those written here are powers of two. The codes and scales of fresh pages need no
 * initial values. */
typedef struct {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  const int32_t* page_table;
  int32_t num_pages, page_size, kv_heads, head_dim, batch, max_pages;
} jepa_kv8_cache;

/* Rotary table [positions][rot] float32, 16-byte aligned: cos of the angles in columns
 * [0, rot/2), sin in [rot/2, rot); angle = position / factor * base^(-2 i / rot), evaluated in
 * 64 bits (factor > 1 stretches positions for contexts longer than those trained on; a table
 * of another rule may be passed to jepa_rope_append_kv8 just as well). rot a multiple of 16. */
jepa_status jepa_rope_table(jepa_ctx* ctx, int positions, int rot, double base, double factor,
                            float* table, void* stream);

/* Append new tokens to the cache, with the queries' and keys' per-head norm and rotation on the
 * way. Token i of sequence b has position p = start[b] + i - cu[b]. For each head row x of q, k:
 *   x <- x * w / sqrt(mean(x^2) + norm_eps)      where w (q_norm / k_norm) is given;
 *   (x_i, x_j) <- (x_i cos - x_j sin, x_j cos + x_i sin) with the table's row p, for the pairs
 *   (i, i + rot/2), or (2i, 2i + 1) where interleaved, i < rot/2; elements past rot stay.
 * q_out = bf16 of the rotated q; the rotated k and v are quantised from fp32: scale of a (page,
 * head) = 2^e, the least e in [-40, 40] with max|x| <= 448 * 2^e over the page's new tokens,
 * codes = e4m3(x / scale), nearest even, saturating (infinities too; NaN stays NaN and does not
 * enter the maximum). Where a page holds earlier tokens its scale never shrinks, and where it
 * grows their codes are rounded to the new scale. Appending the same tokens again changes nothing.
 *   q [tokens][q_heads][head_dim] and q_out (dense) dev, or both NULL; k, v
 *   [tokens][kv_heads][head_dim] dev; k_out (dense, the rotated keys as bf16, as
 *   jepa_attention_packed wants them) dev or NULL; q_norm, k_norm [head_dim] float32 dev or NULL;
 *   rope_table [positions][rot]; cu [batch + 1], start [batch] int32 dev.
 *   q_heads a multiple of kv_heads, at most 65535; rot a multiple of 16, 0 <= rot <= head_dim (0: no rotation);
 *   q_out may be q and k_out may be k where those rows are dense; no other overlap.
 * A page that receives tokens belongs to one place of one sequence (shared pages are full). */
jepa_status jepa_rope_append_kv8(jepa_ctx* ctx, const jepa_kv8_cache* cache, const uint16_t* q,
                                 int64_t q_stride, const uint16_t* k, int64_t k_stride,
                                 const uint16_t* v, int64_t v_stride, int tokens, int q_heads,
                                 const float* q_norm, const float* k_norm, float norm_eps,
                                 const float* rope_table, int positions, int rot, int interleaved,
                                 const int32_t* cu, const int32_t* start, uint16_t* q_out,
                                 uint16_t* k_out, void* stream);

/* Read cached tokens back as bf16 (exact for power-of-two scales): row cu[b] + i of k_out, v_out
 * [tokens][kv_heads][head_dim] (dense) = token first[b] + i of sequence b. With
 * jepa_attention_packed this serves a prompt whose beginning is already cached. */
jepa_status jepa_kv8_read(jepa_ctx* ctx, const jepa_kv8_cache* cache, const int32_t* cu,
                          const int32_t* first, int tokens, uint16_t* k_out, uint16_t* v_out,
                          void* stream);

/* Bytes of jepa_attention_kv8's workspace for this cache's head_dim (the same for every batch,
 * length and head count). */
jepa_status jepa_attention_kv8_workspace(jepa_ctx* ctx, const jepa_kv8_cache* cache, size_t* bytes);

/* Attention of the newest q_tokens tokens of each sequence over its cached tokens (their own
 * keys and values, appended before, included): with n = kv_len[b], query t sees cached tokens
 * [0, n - q_tokens + t + 1) where causal, all n otherwise;
 *   out[b, t, h] = sum_j softmax_j(scale * q[b, t, h] . K_j) V_j,  key / value head
 *   h / (q_heads / kv_heads); lse[b, t, h] = ln sum_j exp(scale * q . K_j).
 * A query that sees nothing gives zeros and lse -inf; what it does not see does not reach it,
 * whatever it holds.
 *   q, out [batch][q_tokens][q_heads][head_dim], 16-byte aligned, dev; kv_len [batch] int32
 *   dev; lse [batch][q_tokens][q_heads] float32 dev or NULL; workspace: device memory of the
 *   size above, 256-byte aligned, its contents between calls without meaning. At most 65536 query
 *   rows a key/value head of a sequence (q_tokens * q_heads / kv_heads) and 2^30 in all. Calls that may
 *   overlap on the device (streams, graphs) need a workspace each. scale finite, > 0. */
jepa_status jepa_attention_kv8(jepa_ctx* ctx, const jepa_kv8_cache* cache, const uint16_t* q,
                               int q_tokens, int q_heads, const int32_t* kv_len, float scale,
                               int causal, uint16_t* out, float* lse, void* workspace,
                               size_t workspace_bytes, void* stream);

/* Attention of whole packed prompts. Sequence b has nq = cu_q[b+1] - cu_q[b] queries and nk =
 * cu_k[b+1] - cu_k[b] keys; query i stands at position p = i + nk - nq and sees keys
 * [0, min(nk, (p / frame + 1) * frame)), none where p < 0: frame 1 is causal, frame T is causal
 * over frames of T tokens (the predictor's mask), frame >= nk sees everything.
 *   q [tokens_q][q_heads][head_dim], k, v [tokens_k][kv_heads][head_dim] with strides, 16-byte
 *   aligned, dev; cu_q, cu_k [batch + 1]; out [tokens_q][q_heads][head_dim] dense, 16-byte
 *   aligned; lse [tokens_q][q_heads] float32 or NULL, as in jepa_attention_kv8, whose promises
 *   for unseen keys and empty rows hold here too. head_dim 64 or 128, q_heads a multiple of
 *   kv_heads with at most 128 per key/value head and 65535 in all, scale finite and > 0, frame >= 1,
 *   batch at most 65535, tokens_q and tokens_k at most 2^27, and
 *   (tokens_q / (2 * (128 / group)) + min(batch, tokens_q)) * kv_heads at most 2^28 with group =
 *   q_heads / kv_heads. A value of v that is not finite reaches the queries that see it; where many
 *   of them lie behind some query's limit in its block of 256 rows, that block costs up to 0.15 us a
 *   key more. */
jepa_status jepa_attention_packed(jepa_ctx* ctx, const uint16_t* q, int64_t q_stride,
                                  const uint16_t* k, int64_t k_stride, const uint16_t* v,
                                  int64_t v_stride, int tokens_q, int tokens_k, int batch,
                                  int q_heads, int kv_heads, int head_dim, const int32_t* cu_q,
                                  const int32_t* cu_k, float scale, int frame, uint16_t* out,
                                  float* lse, void* stream);

/* ---- 4-bit paged key/value cache, eviction from it, and the norm ahead of 8-bit products ----
 *
 * Everything said above of the 8-bit cache's entry points (contexts, streams, capture, packed
 * sequences, strides, indices on the device) holds here as well. */

/* One layer's cache in 4 bits. k, v [num_pages][kv_heads][page_size][head_dim / 2]: e2m1 codes (sign,
 * two bits of exponent, one of mantissa: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), element 2i in the
 * low half of byte i; k_scale, v_scale [num_pages][kv_heads][page_size][head_dim / 16]: e4m3 scales of
 * 16 elements each; k_unit, v_unit [kv_heads] float32 or NULL (1): a power of two for each head, within
 * [2^-40, 2^40] (others are read as the power of two at or below, or the nearer end; NaN as the
 * least). An element stands for code * scale * unit. page_table, sizes and limits as in
 * jepa_kv8_cache; k, v, k_scale and v_scale 16-byte aligned. A unit near a sixth of the head's usual
 * magnitude (0.1 to 1000 times that) keeps the scales among e4m3's normal numbers. No token's codes depend on
 * another's: fresh pages need no initial values, and appends change nothing that is there. */
typedef struct {
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  const float* k_unit;
  const float* v_unit;
  const int32_t* page_table;
  int32_t num_pages, page_size, kv_heads, head_dim, batch, max_pages;
} jepa_kv4_cache;

/* Append new tokens to the cache: arguments, norm, rotation and q_out, k_out as in
 * jepa_rope_append_kv8. Each 16 elements of a rotated key or of a value are quantised from fp32: scale =
 * e4m3(max|x| / 6 / unit), nearest even, at least 2^-9 and at most 448; codes = e2m1(x / (scale * unit)),
 * nearest even, saturating. A block that holds a NaN or an infinity gets a NaN scale and reads as NaN. For
 * keys the norm's factor 1 / sqrt(mean(x^2) + norm_eps) is rounded once to fp32 (of any finite head: its squares may
 * leave fp32) and multiplied by the weight first, and each product and sum of the rotation is rounded to fp32. rope_start [batch] int32 dev or
 * NULL: token i of sequence b lies at place start[b] + i - cu[b] and is rotated for position rope_start[b] + i -
 * cu[b], as it has to be behind an eviction; NULL: both are start. */
jepa_status jepa_rope_append_kv4(jepa_ctx* ctx, const jepa_kv4_cache* cache, const uint16_t* q,
                                 int64_t q_stride, const uint16_t* k, int64_t k_stride,
                                 const uint16_t* v, int64_t v_stride, int tokens, int q_heads,
                                 const float* q_norm, const float* k_norm, float norm_eps,
                                 const float* rope_table, int positions, int rot, int interleaved,
                                 const int32_t* cu, const int32_t* start, const int32_t* rope_start,
                                 uint16_t* q_out, uint16_t* k_out, void* stream);

/* Read cached tokens back as bf16 (exact), as jepa_kv8_read. */
jepa_status jepa_kv4_read(jepa_ctx* ctx, const jepa_kv4_cache* cache, const int32_t* cu,
                          const int32_t* first, int tokens, uint16_t* k_out, uint16_t* v_out,
                          void* stream);

/* Bytes of jepa_attention_kv4's workspace for this cache's head_dim (the same for every batch,
 * length and head count). */
jepa_status jepa_attention_kv4_workspace(jepa_ctx* ctx, const jepa_kv4_cache* cache, size_t* bytes);

/* Attention of the newest q_tokens tokens of each sequence over its cached tokens: arguments,
 * promises and limits as in jepa_attention_kv8. Where mass_out is given (lse then has to be), also the
 * weight that each cached token received, summed over the new tokens and the query heads that share its
 * key/value head:
 *   mass_out[b, h, j] = decay * mass[b, h, j] + sum_{t, g} exp(scale * q[b, t, g] . K_j - lse[b, t, g])
 * for j < kv_len[b]; what lies behind is left as it was. mass, mass_out [batch][kv_heads][max_pages *
 * page_size] float32 dev; mass NULL: zeros; mass_out may be mass. A token that is appended starts
 * with what mass holds at its place, so fill it with zeros at first (jepa_kv4_evict does so behind what it
 * keeps). decay finite, and out apart from q (the weights come after out). The sums' order is fixed. */
jepa_status jepa_attention_kv4(jepa_ctx* ctx, const jepa_kv4_cache* cache, const uint16_t* q,
                               int q_tokens, int q_heads, const int32_t* kv_len, float scale,
                               int causal, uint16_t* out, float* lse, const float* mass,
                               float* mass_out, float decay, void* workspace, size_t workspace_bytes,
                               void* stream);

/* Bytes of jepa_kv4_evict's workspace: 4 * batch * kv_heads * keep. */
jepa_status jepa_kv4_evict_workspace(jepa_ctx* ctx, const jepa_kv4_cache* cache, int keep, size_t* bytes);

/* Evict cached tokens by accumulated weight. Of the n = kv_len[b] tokens of a sequence each key/value
 * head keeps its last `recent` and, of those before, the ones with the largest mass (as float32; ties go
 * to the lower place, NaN counts as the least), `keep` in all; all n where n <= keep. In their order they become
 * tokens 0, 1, .. of the pages that to->page_table names, codes and scales unchanged (keys keep the
 * rotation of their old positions); len_out[b] = min(n, keep), and mass_out [batch][kv_heads][to->max_pages *
 * to->page_size] (or NULL) their masses, zeros behind. Different heads of a sequence may keep different tokens.
 *   `to` may have the same buffers as `cache` with another table, the same units (pointers), batch, heads and
 *   head_dim; its pages page_size and number may differ. The pages that receive tokens belong to one place of
 *   one sequence and hold no token that `cache` names (shared pages are thus never written), but for
 *   sequences with n <= keep, which may name the same pages in both tables where the page sizes are equal.
 *   kv_len, len_out [batch] int32 dev; mass [batch][kv_heads][max_pages * page_size] float32 dev;
 *   0 <= recent <= keep, 1 <= keep <= 2^30; where to's table names fewer than keep tokens it counts as so many
 *   (recent too); workspace as above, 256-byte
 *   aligned. Calls that may overlap on the device need a workspace each. */
jepa_status jepa_kv4_evict(jepa_ctx* ctx, const jepa_kv4_cache* cache, const int32_t* kv_len,
                           const float* mass, int keep, int recent, const jepa_kv4_cache* to,
                           int32_t* len_out, float* mass_out, void* workspace, size_t workspace_bytes,
                           void* stream);

/* Residual addition, RMS norm and 8-bit codes of a row, ready for jepa_linear_fp8:
 *   s = x + delta (fp32), x_out = s in x's type, y = s * weight / sqrt(mean(s^2) + eps),
 *   codes, scales = y as jepa_quantize_rows_fp8 has it (from fp32), y also as bf16.
 * The norm is that of the unrounded s. x, x_out [rows][cols] float32 (x_bf16 0) or bf16 (1), delta float32
 * or bf16 (delta_bf16), each with `*_stride` elements between rows (at least cols, a multiple of 8);
 * delta NULL: none; x_out NULL: not wanted, or x: in place (equal strides; no other overlap). weight
 * [cols] float32; codes [rows][cols] with scales [rows] float32, or both NULL; y [rows][cols] bf16 or NULL (not
 * both left out). All dev, 16-byte aligned but scales. cols a multiple of 16, at most 32768. Any context. */
jepa_status jepa_add_rmsnorm_fp8(jepa_ctx* ctx, const void* x, int x_bf16, int64_t x_stride,
                                 const void* delta, int delta_bf16, int64_t delta_stride,
                                 const float* weight, float eps, int rows, int cols, void* x_out,
                                 int64_t x_out_stride, uint8_t* codes, float* scales, uint16_t* y,
                                 void* stream);

/* enable = 0: jepa_cem_plan launches the kernels of its captured graph one by one on the
 * stream instead of replaying the graph (same kernels, same results; for measuring what the
 * graph saves). enable != 0 (the default): graph replay. */
jepa_status jepa_set_use_graphs(jepa_ctx* ctx, int enable);

/* Kernel-level timing of the predictor GEMMs inside plan graphs. enable != 0 makes graphs
 * captured afterwards record a CUDA event pair around every GEMM launch (graphs captured
 * before keep their state). jepa_profile_read (after the stream is synchronised) returns
 * the summed event time, summed algorithmic FLOPs (2*M*N*K) and launch count of the
 * GEMMs in the most recent plan call, and resets nothing. */
jepa_status jepa_profile_enable(jepa_ctx* ctx, int enable);
jepa_status jepa_profile_read(jepa_ctx* ctx, double* gemm_ms, double* gemm_flops,
                              int64_t* gemm_launches);

/* L1 energy of already-predicted frames, for callers that cannot allocate device memory
 * (the planning pages have no counterpart: this is a deployment variant of the energy
 * step). Typical callers: a process running under a fixed device-memory budget owned by
 * a host framework, or a real-time control loop that must not pay for, or risk failure
 * of, an allocation in the middle of an episode. No context is needed and nothing is
 * allocated: the per-candidate partial sums go to one fixed device array inside this
 * library, 2^20 floats (4 MiB), which every GPU that loads the library keeps until the
 * process exits.
 *   z_pred [B,N,P,E] dev   predicted frames (e.g. the z_pred output of jepa_predictor_forward)
 *   goal   [B,P,E]   dev
 *   energy [B,N]     dev   output: mean |z_pred - goal| per candidate
 *   err, err_len           optional caller buffer for a text description of a failure
 * Limits: B*N*ceil(P/32) <= 2^20, otherwise JEPA_ERR_SHAPE (split the candidates over
 * several calls). Runs on the current CUDA device. The first call in a device's CUDA context
 * looks up the array's device address and caches it for that context (a device reset makes a
 * new context, and the next call looks the address up again), so make that first call before
 * any stream capture. All calls share the array: calls that can overlap on the GPU (on streams with
 * no ordering between them) race and can return wrong energies; calls ordered on one
 * stream are safe. */
jepa_status jepa_energy_l1_noalloc(const float* z_pred, const float* goal, int B, int N, int P,
                                   int E, float* energy, void* stream, char* err, size_t err_len);

/* Failure-detection self-test: launches one thread that waits, through the bounded mbarrier
 * wait every pipelined kernel of this library uses, on a barrier nothing will arrive on.
 * After the wait's limit (2 s) it gives up, raises this context's error flag and returns;
 * the next jepa_sync_check then reports JEPA_ERR_TIMEOUT (and clears the flag). Nothing
 * faults or hangs; the context stays usable. */
jepa_status jepa_selftest_bounded_wait(jepa_ctx* ctx, void* stream);

/* Synchronise `stream`, then report JEPA_ERR_TIMEOUT if a bounded device-side wait in
 * any kernel of this context gave up since the last check, or else JEPA_ERR_INVALID_ARG if a
 * kernel met a page index, position, length or offset outside its buffer (the flag is then
 * cleared). */
jepa_status jepa_sync_check(jepa_ctx* ctx, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* JEPA_CEM_H_ */
