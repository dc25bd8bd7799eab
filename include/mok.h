/*
 * mok.h -- C ABI of the MoE-layer hot path for AMD Instinct MI355X (gfx950).
 *
 * One GPU's share of a mixture-of-experts layer: a deterministic schedule
 * built from top-k routing, a grouped SwiGLU expert MLP with an always-on
 * shared expert, and a router-weighted combine back to token order, forward
 * and backward, in BF16 and in MXFP8 (E4M3 elements, one E8M0 scale per 32
 * elements along the contraction dimension).
 *
 * Pages this interface follows (titles as published):
 *   [R] "Mixture-of-Kittens: a deterministic MoE megakernel for NVL72 racks"
 *   [A] "nemo_automodel.components.moe.mok_experts" (NeMo AutoModel API docs)
 *   [B] the moses-y.github.io review "mixture-of-kittens"
 *
 * Conventions for every call:
 *   - Pointers named as device pointers must point to device memory of the
 *     workspace's device; every tensor is dense and row-major ("contiguous",
 *     [A] _MoKRuntime.forward parameters). bf16 tensors are passed as raw
 *     16-bit patterns (void*).
 *   - `stream` is a hipStream_t (NULL = the default stream). Calls that take a
 *     stream only enqueue work: they never synchronise with the host and never
 *     read device data on the host ([B] "What This Does": no CPU-GPU
 *     synchronization; [R] "What Mixture-of-Kittens solves").
 *   - Argument, shape and configuration errors are detected on the host
 *     before anything is enqueued and returned synchronously; nothing is
 *     enqueued when a call returns an error. A failed HIP launch returns
 *     MOK_ERR_HIP.
 *   - The library touches no device when it is loaded; a device is first used
 *     by mok_workspace_create ([A] _load_mok_functional: loading the extension
 *     before the process has picked its GPU leaves a stray context).
 *   - A workspace may be used by one stream at a time; calls that overlap on
 *     one workspace race on its scratch memory.
 */
#ifndef MOK_H_
#define MOK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOK_VERSION_MAJOR 0
#define MOK_VERSION_MINOR 1

typedef enum mok_status {
  MOK_OK = 0,
  MOK_ERR_INVALID_ARGUMENT = 1, /* null pointer, negative or inconsistent size */
  MOK_ERR_UNSUPPORTED = 2,      /* shape outside the kernels' contract ([A] _validate_model_mok_config) */
  MOK_ERR_CONFIG_MISMATCH = 3,  /* schedule/context built for another config or token count */
  MOK_ERR_BUFFER_TOO_SMALL = 4, /* caller buffer smaller than the *_bytes query says */
  MOK_ERR_HIP = 5               /* a HIP runtime call or launch failed */
} mok_status;

typedef enum mok_mode {
  MOK_MODE_BF16 = 0,  /* bf16 operands, fp32 accumulation */
  MOK_MODE_MXFP8 = 1  /* E4M3 operands with E8M0 block scales, fp32 accumulation ([R] "Tuning the five hyperparameters before production") */
} mok_mode;

/*
 * Layer configuration: the single-GPU reading of the pages' MoKConfig
 * ([R] "The two API layers and the schedule object", "Tuning the five
 * hyperparameters before production"). Set struct_size = sizeof(mok_config).
 *
 * Contract (MOK_ERR_UNSUPPORTED otherwise, MOK_ERR_INVALID_ARGUMENT for
 * negative sizes): hidden % 128 == 0;
 * intermediate % 64 == 0 and shared_intermediate % 64 == 0 (0 = no shared
 * expert); 1 <= num_experts <= 1024; 1 <= topk <= 64; expert_pad a positive
 * multiple of 32 (MXFP8 backward needs 32-row blocks inside one expert);
 * max_tokens >= 1 with max_tokens * topk < 2^31. Every operand a kernel
 * reads stays below 2 GiB: (max_tokens + 127) * max(hidden, intermediate,
 * shared_intermediate, 256) * 2 < 2^31, intermediate * hidden * 2 < 2^31 and
 * shared_intermediate * hidden * 2 < 2^31; and the schedule's row bound
 * rows_cap_max + max_tokens < 2^31.
 */
typedef struct mok_config {
  uint32_t struct_size;
  int32_t hidden;               /* H */
  int32_t intermediate;         /* I: routed expert intermediate size */
  int32_t num_experts;          /* E: local experts (all experts, on one GPU) */
  int32_t topk;                 /* k */
  int32_t shared_intermediate;  /* I_s: shared expert intermediate size, 0 = none */
  int64_t max_tokens;           /* T_max: sizes every buffer for the worst case */
  float capacity_multiplier;    /* per-expert capacity C = min(T, ceil(mult * T)) ([R] "Tuning...": schedule_capacity_multiplier) */
  int32_t expert_pad;           /* P: each expert segment padded to a multiple of P rows ([R] "Tuning...": expert padding) */
  int32_t minibatch_size;       /* tokens per minibatch: the schedule's sub-offsets, and the granularity of the
                                   forward's minibatch pipeline; 0 = one minibatch ([R] "Tuning...": minibatch_size) */
  int32_t num_mover_wgs;        /* mover workgroups of the forward's minibatch pipeline (rounded down to a multiple
                                   of 8, at most the compute units less 32); 0 = no pipeline. With 0 <
                                   minibatch_size < max_tokens, num_mover_wgs >= 8 and num_experts <= 256, the down
                                   GEMM and the combine run as one launch of one workgroup per compute unit: the
                                   others run the down tiles minibatch by minibatch and count each finished tile,
                                   and these combine minibatch b as soon as its count is complete, while the tiles
                                   of later minibatches run ([R] "Tuning...": fwd_num_comm_sms, minibatch_size).
                                   A mover's wait is bounded (about 2 s in all); one that runs out of time is
                                   counted in mok_workspace_read_status. The result bits do not depend on either
                                   value. */
  float swiglu_limit;           /* SwiGLU input limit L ([A] _MoKRuntime(mok_config, swiglu_limit); the pages give
                                   no formula): L > 0 computes h = silu(min(g, L)) * clamp(u, -L, L), and the
                                   backward passes no gradient where a clamp is active (g > L, |u| > L);
                                   0 or +inf = no limit. Negative or NaN: MOK_ERR_INVALID_ARGUMENT. */
  int32_t macrobatch_size;      /* tokens per pass of the workspace's token ring ([R] "Tuning...": macrobatch_size, the
                                   token ring buffer; a size at least max_tokens means the ring is used once).
                                   0 or >= max_tokens: one pass. Otherwise mok_forward streams the batch through
                                   scratch sized for macrobatch_size tokens, macrobatch by macrobatch, with the
                                   whole batch's schedule (capacity and drops as in one pass): the output bits are
                                   those of one pass. Requires forward_only = 1 (a backward contracts each expert's
                                   weight gradient over the whole batch), num_experts >= topk and, when
                                   minibatch_size > 0, a multiple of it (MOK_ERR_UNSUPPORTED otherwise). Each pass
                                   adds one small kernel (its schedule) and runs without the minibatch pipeline. */
  int32_t forward_only;         /* 1: an inference workspace, with no backward scratch (mok_backward returns
                                   MOK_ERR_UNSUPPORTED, mok_forward takes no context); 0: training */
} mok_config;

/* Routed and shared expert weights, layouts of [A] _MoKRuntime.forward:
 * gate/up [E, I, H], down [E, H, I], shared gate/up [I_s, H], shared down
 * [H, I_s]. In BF16 mode the data pointers are bf16 and the scale pointers
 * are ignored. In MXFP8 mode the data pointers are E4M3 bytes of the same
 * shapes and the scales are E8M0 bytes with one scale per 32 elements along
 * the last dimension (the contraction dimension of the forward GEMMs), as
 * written by mok_mxfp8_quantize(axis = 1): gate/up scales [E*I, H/32], down
 * [E*H, I/32], shared gate/up [I_s, H/32], shared down [H, I_s/32]. Shared
 * pointers must be NULL iff shared_intermediate == 0. */
typedef struct mok_weights {
  const void* routed_gate;
  const void* routed_up;
  const void* routed_down;
  const void* shared_gate;
  const void* shared_up;
  const void* shared_down;
  const uint8_t* routed_gate_scale;
  const uint8_t* routed_up_scale;
  const uint8_t* routed_down_scale;
  const uint8_t* shared_gate_scale;
  const uint8_t* shared_up_scale;
  const uint8_t* shared_down_scale;
} mok_weights;

/* Gradients written by mok_backward ([A] _MoKRuntime.backward: one gradient
 * per float input; the integer expert ids get none). dx bf16 [T, H];
 * d_router_weights fp32 [T, k] (0 for dropped or invalid assignments);
 * d_routed_gate/up bf16 [E, I, H]; d_routed_down bf16 [E, H, I];
 * d_shared_gate/up bf16 [I_s, H]; d_shared_down bf16 [H, I_s] (NULL iff
 * shared_intermediate == 0). Every element is written (experts that receive
 * no rows get zero weight gradients). */
typedef struct mok_grads {
  void* dx;
  float* d_router_weights;
  void* d_routed_gate;
  void* d_routed_up;
  void* d_routed_down;
  void* d_shared_gate;
  void* d_shared_up;
  void* d_shared_down;
} mok_grads;

/* Byte offsets of the schedule's fields inside the caller's schedule buffer
 * (every field int32, little endian). The schedule is the pages' "schedule
 * object": built once per layer and step from routing, before any expert
 * math, and passed unchanged to forward and backward ([R] "The two API
 * layers and the schedule object"). Fields (this call's token count T):
 *   header[16]: [0] T, [1] k, [2] E, [3] C, [4] P, [5] rows_cap(T),
 *               [6] n_mb, [7] minibatch size, [8] dropped, [9] invalid,
 *               [10] total padded rows = offsets[E], [11] config hash,
 *               [12..15] reserved
 *   counts[E]     valid assignments per expert
 *   kept[E]       min(counts, C)
 *   offsets[E+1]  exclusive prefix sum of kept rounded up to P
 *   mb_offsets[(n_mb_max+1)*E]  row where minibatch b of expert e starts
 *   row_src[rows_cap_max]  flat assignment a = t*k + j feeding each row, -1 for
 *                          padding and unused rows (valid up to rows_cap(T))
 *   slot_row[T_max*k]      row of assignment a, -1 if dropped or invalid
 *   tiles[4][E+2]          internal GEMM tile prefix sums (not part of the
 *                          method's result) */
typedef struct mok_schedule_layout {
  size_t total_bytes;
  size_t header;
  size_t counts;
  size_t kept;
  size_t offsets;
  size_t mb_offsets;
  size_t row_src;
  size_t slot_row;
  size_t tiles;
  int64_t rows_cap_max;
  int64_t n_mb_max;
} mok_schedule_layout;

typedef struct mok_workspace mok_workspace;  /* opaque; owns device scratch only */

/* ---- pure host queries (no device, no HIP call) ---------------------- */

/* Name of a status code. Never NULL. */
const char* mok_status_string(mok_status status);

/* Checks a configuration against the contract above. */
mok_status mok_validate_config(const mok_config* cfg);

/* Bytes of the caller-owned schedule buffer for this config; 0 if invalid.
 * "At most a few megabytes" at production shapes ([R] "Tuning..."). */
size_t mok_schedule_bytes(const mok_config* cfg);

/* Fills *out with the schedule buffer's field offsets. */
mok_status mok_schedule_layout_query(const mok_config* cfg, mok_schedule_layout* out);

/* Bytes of the caller-owned forward context (saved activations for
 * backward: G, U and h of every routed and shared row); 0 if invalid.
 * BF16 mode: G, U and h in bf16. MXFP8 mode: G and U in fp32 as the
 * forward accumulated them (the backward's SwiGLU derivative starts from the
 * values h came from) and h as the E4M3 codes and E8M0 scales the down GEMM
 * read; about twice the BF16 size. A context is read only by a backward of
 * the mode that wrote it. */
size_t mok_context_bytes(const mok_config* cfg, mok_mode mode);

/* Device scratch a workspace of this config allocates, in bytes. */
size_t mok_workspace_bytes(const mok_config* cfg);

/* ---- workspace ------------------------------------------------------- */

/* Allocates the workspace's scratch once on `device` ([R] "The two API
 * layers and the schedule object": one workspace per model, reused across
 * layers and steps). The config is copied. Writes NULL to *out on error. */
mok_status mok_workspace_create(const mok_config* cfg, int device, mok_workspace** out);

/* Frees the scratch (waits for the device). NULL is accepted. */
mok_status mok_workspace_destroy(mok_workspace* ws);

/* ---- the hot path ---------------------------------------------------- */

/*
 * Builds the schedule for T tokens from top_experts (device int64 [T, k],
 * expert ids; ids outside [0, E) are counted as invalid and never
 * dispatched). Per expert: counts, capacity C = min(T, ceil(mult*T)),
 * kept = first C assignments in flat order a = t*k + j (the rest are
 * dropped and counted), segments padded to P rows, exclusive prefix-sum
 * offsets, a stable permutation (rows of an expert in ascending a) and its
 * inverse, and per-minibatch sub-offsets. Deterministic: the same ids give
 * the same bytes ([R] "How MoK differs from a general MoE kernel library").
 * `schedule` is a device buffer of at least mok_schedule_bytes(cfg) bytes;
 * 0 <= T <= max_tokens. Runs 2 small kernels (3 with more than one minibatch).
 */
mok_status mok_build_schedule(mok_workspace* ws, const int64_t* top_experts, int64_t T,
                              void* schedule, size_t schedule_bytes, void* stream);

/*
 * Forward ([A] _MoKRuntime.forward; [A] GroupedExpertsMoK.forward): for each
 * token t, out[t] = sum over its kept assignments j of
 * w[t,j] * W_d[e] (silu(W_g[e] x_t) * (W_u[e] x_t)) + the shared expert's
 * S_d (silu(S_g x_t) * (S_u x_t)), with fp32 accumulation, summed in fixed
 * slot order (deterministic). x bf16 [T, H] (device); router_weights fp32
 * [T, k] (device); out bf16 [T, H] (device). T is taken from the schedule.
 * In MXFP8 mode x is quantized on the device inside this call and the
 * weights must be pre-quantized ([R] "Tuning...": MXFP8 workflow); h is
 * quantized along I before the down projection.
 * `context` (device, nullable, at least mok_context_bytes) receives the
 * activations mok_backward needs; pass NULL for inference.
 * x, router_weights and out must be non-NULL even for an empty batch (the
 * host cannot see T): with T = 0 they are never read or written, so any
 * device address will do.
 */
mok_status mok_forward(mok_workspace* ws, mok_mode mode, const void* schedule, size_t schedule_bytes,
                       const void* x, const float* router_weights, const mok_weights* weights,
                       void* out, void* context, size_t context_bytes, void* stream);

/*
 * The MXFP8 forward of mok_forward for tokens that are already in MXFP8
 * (codes from mok_rms_norm or mok_mxfp8_quantize): x_codes E4M3 [T, H] and
 * x_scale E8M0 [T, H/32], both dense, 16- and 4-byte aligned
 * (MOK_ERR_UNSUPPORTED otherwise). The launch that quantizes x is left out;
 * everything else, arguments and results, is as in mok_forward with
 * MOK_MODE_MXFP8, and with the codes that mok_mxfp8_quantize(axis = 1) gives
 * for a bf16 x the output bits are those of mok_forward on that x. A
 * backward on the context still takes x in bf16. A token with a NaN scale
 * (0xFF) gets a row of NaN and reaches no other token; with a swiglu_limit,
 * which clamps a NaN like any value, its row may be finite and means nothing.
 */
mok_status mok_forward_mxfp8(mok_workspace* ws, const void* schedule, size_t schedule_bytes, const uint8_t* x_codes,
                             const uint8_t* x_scale, const float* router_weights, const mok_weights* weights,
                             void* out, void* context, size_t context_bytes, void* stream);

/*
 * Backward ([A] _MoKRuntime.backward): gradients of sum(grad_out * out) for
 * every float input, reusing the forward's schedule and context. grad_out,
 * x bf16 [T, H]; router_weights fp32 [T, k]. In BF16 mode `weights` are the
 * BF16 weights (scale pointers ignored). In MXFP8 mode every backward GEMM
 * operand is quantized along that GEMM's own contraction dimension (grad_out
 * rows along H; dG, dU along I; the weight gradients' operands in 32-row
 * blocks of each expert's rows), the context must come from an MXFP8 forward
 * of the same schedule, and `weights` is either
 *   - the BF16 weights with every scale pointer NULL: they are transposed
 *     and quantized on the device in this call, or
 *   - the weights already transposed and quantized by
 *     mok_mxfp8_quantize_transposed, with every scale pointer set (the
 *     pages' workflow of weights pre-quantized by a separate call, [R]
 *     "Tuning the five hyperparameters before production"): routed_down
 *     [E, I, H] codes with [E*I, H/32] scales (W_d^T, blocks along H);
 *     routed_gate / routed_up [E, H, I] with [E*H, I/32] (blocks along I);
 *     shared_down [I_s, H] with [I_s, H/32]; shared_gate / shared_up
 *     [H, I_s] with [H, I_s/32].
 *   Some but not all scale pointers set: MOK_ERR_INVALID_ARGUMENT.
 * MXFP8 mode returns MOK_ERR_UNSUPPORTED unless H, I and I_s are multiples
 * of 128. Uses only the workspace's scratch (no allocation). Every weight
 * gradient is written in full (zero for experts with no kept rows, and for
 * all of them when T = 0); as in mok_forward, the token-sized pointers must
 * be non-NULL even when T = 0.
 */
mok_status mok_backward(mok_workspace* ws, mok_mode mode, const void* schedule, size_t schedule_bytes,
                        const void* context, size_t context_bytes, const void* grad_out, const void* x,
                        const float* router_weights, const mok_weights* weights, const mok_grads* grads,
                        void* stream);

/*
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the
 * inference forward of mok_forward (context = NULL) without a workspace.
 * Its scratch (h, the weighted down rows y, and x's MXFP8 codes) is a fixed
 * device array of the library, 128 MiB per GPU, held from the first call on
 * a GPU until the process ends; the call allocates nothing. Scratch needed,
 * with n = rows_cap_max * I + max_tokens * I_s (rows_cap_max from
 * mok_schedule_layout_query) and each part rounded up to 256 bytes: h, 2n
 * bytes (BF16) or n + n/32 (MXFP8); y, (rows_cap_max + max_tokens) * H * 2;
 * in MXFP8 also x's codes and scales, m + m/32 with m = max_tokens * H. A
 * config that needs more returns MOK_ERR_UNSUPPORTED before anything is
 * enqueued. cfg is the config of the workspace whose
 * mok_build_schedule wrote `schedule` (minibatch pipeline and token ring
 * fields are ignored: one pass, no pipeline; the bits are the same). Runs on the current device (`stream` must belong
 * to it). Arguments and results otherwise as mok_forward. Calls on one GPU
 * share the array: calls that overlap on one GPU race.
 */
mok_status mok_forward_static(const mok_config* cfg, mok_mode mode, const void* schedule, size_t schedule_bytes,
                              const void* x, const float* router_weights, const mok_weights* weights, void* out,
                              void* stream);

/*
 * MXFP8 quantization ([R] "Tuning the five hyperparameters before
 * production": the separate quantize call for pre-quantizing weights).
 * src: device [rows, cols] with row stride ld_src elements, bf16
 * (src_is_fp32 = 0) or fp32 (src_is_fp32 = 1).
 * axis = 1: blocks of 32 consecutive elements along a row (cols % 32 == 0);
 *           scales [rows, cols/32], row stride cols/32.
 * axis = 0: blocks of 32 consecutive rows in a column (rows % 32 == 0);
 *           scales [rows/32, cols], row stride cols.
 * dst: E4M3 bytes [rows, cols] with row stride ld_dst (cols % 8 == 0 and
 * ld_dst % 8 == 0, ld_src % 8 == 0). Per block: X = clamp(floor(log2 amax)
 * - 8, -127, 127) (X = -127 for an all-zero block), scale byte X + 127,
 * element = round-to-nearest-even of v / 2^X on the E4M3 grid, saturating
 * at +-448, sign kept. Inputs must be finite. The codes are exact: the
 * hardware scaled conversion gives the same bytes as the rule above.
 * MOK_ERR_UNSUPPORTED for bf16 sources along axis 1 with more than 2^24 rows
 * (one workgroup per row).
 */
mok_status mok_mxfp8_quantize(const void* src, int src_is_fp32, int64_t rows, int64_t cols, int64_t ld_src,
                              int axis, uint8_t* dst, int64_t ld_dst, uint8_t* dst_scale, void* stream);

/*
 * Transposed MXFP8 quantization of a batch of bf16 matrices, the weights'
 * form for the MXFP8 backward ([R] "Tuning the five hyperparameters before
 * production": weights are quantized by a separate call). src: device bf16
 * [batches, rows, cols], dense. dst: E4M3 [batches, cols, rows] (the
 * transpose), quantized in blocks of 32 consecutive elements along its rows
 * (the source's `rows` dimension, which is the backward GEMM's contraction);
 * dst_scale: E8M0 [batches, cols, rows/32]. Codes and scales follow the rule
 * of mok_mxfp8_quantize. rows % 128 == 0 and cols % 64 == 0, src and dst
 * 16-byte aligned, dst_scale 4-byte aligned (MOK_ERR_UNSUPPORTED otherwise).
 * Runs on the current device. For W_d [E, H, I]: batches E, rows H, cols I;
 * W_g / W_u [E, I, H]: rows I, cols H; the shared weights with batches 1.
 */
mok_status mok_mxfp8_quantize_transposed(const void* src, int64_t batches, int64_t rows, int64_t cols, uint8_t* dst,
                                         uint8_t* dst_scale, void* stream);

/* ---- the operators around the layer ----------------------------------
 *
 * What the block that holds the layer needs next to it: the norm in front,
 * the router, and the optimizer's step. They need no workspace and keep
 * nothing between calls; they run on the current device, to which `stream`
 * and every pointer must belong. As everywhere, they only enqueue work, and
 * are deterministic: the same inputs give the same bits. Row strides (ld_*)
 * are in elements and at least the row's length; outputs are dense. */

/*
 * RMS norm with the residual's addition. Per row of `cols` elements:
 *   s = x + residual (s = x without one)
 *   rstd = (mean(s^2) + eps)^-1/2,   y = s * rstd * weight
 * in fp32, each output rounded once: y comes from the fp32 sum, not from its
 * rounding. x is bf16 or fp32; residual (nullable) has x's type or, for bf16
 * x, may be fp32 (fp32 x with a bf16 residual: MOK_ERR_UNSUPPORTED); weight
 * [cols] bf16 or fp32. Outputs:
 *   sum    [rows, cols] in the residual's type; non-NULL iff residual is. It
 *          may be the residual's own buffer (dense), or x's if of its type.
 *   y      bf16 [rows, cols], nullable.
 *   codes, scale   y in MXFP8 along a row (both or neither): E4M3 [rows,
 *          cols] and E8M0 [rows, cols/32] by the rule of mok_mxfp8_quantize,
 *          taken from the fp32 y (not from its bf16 rounding), the form that
 *          mok_forward_mxfp8 reads. A block that holds an infinity or a NaN
 *          gets the NaN scale 0xFF. Needs cols % 32 == 0, cols <= 16384, row
 *          strides % 8 == 0, 16-byte aligned tensors and 8-byte aligned
 *          codes (MOK_ERR_UNSUPPORTED otherwise).
 *   rstd   fp32 [rows], nullable: what the backward needs besides s.
 * At least one output must be asked for. Without codes every width, stride
 * and alignment is accepted; cols % 8 == 0, cols <= 16384, strides % 8 == 0
 * and 16-byte alignment run the fast kernel. The sum of squares is an fp32
 * sum: rows with |s| above about 1e18 overflow it (rstd 0), and rows with all
 * |s| below about 1e-18 leave it inexact, which shows only with eps near 0.
 */
mok_status mok_rms_norm(const void* x, int x_is_fp32, int64_t ld_x, const void* residual, int residual_is_fp32,
                        int64_t ld_residual, const void* weight, int weight_is_fp32, int64_t rows, int64_t cols,
                        float eps, void* sum, void* y, uint8_t* codes, uint8_t* scale, float* rstd, void* stream);

/* Bytes of mok_rms_norm_backward's scratch; 0 if the sizes are invalid. */
size_t mok_rms_norm_scratch_bytes(int64_t rows, int64_t cols);

/*
 * Backward of mok_rms_norm from the saved s (the forward's sum, or its x
 * without a residual; bf16 or fp32) and rstd. dy bf16. With xh = s * rstd
 * and g = dy * weight:
 *   ds = rstd * (g - xh * mean(g * xh)) + d_sum,   d_weight = sum over rows of dy * xh
 * ds [rows, cols] in s's type is the gradient of both x and the residual;
 * dx (nullable) receives it in bf16 as well, for a bf16 x with an fp32
 * residual. d_sum (nullable, s's type) is the gradient that arrives through
 * the sum; ds may be its buffer (dense). d_weight [cols] in weight's type is
 * written in full, zeros for rows = 0. scratch: 16-byte aligned device
 * memory of at least mok_rms_norm_scratch_bytes(rows, cols), the call's own
 * until its work has run.
 */
mok_status mok_rms_norm_backward(const void* dy, int64_t ld_dy, const void* s, int s_is_fp32, int64_t ld_s,
                                 const float* rstd, const void* weight, int weight_is_fp32, const void* d_sum,
                                 int64_t ld_d_sum, int64_t rows, int64_t cols, void* ds, void* dx, void* d_weight,
                                 void* scratch, size_t scratch_bytes, void* stream);

/* Scores of the router. */
typedef enum mok_router_scoring {
  MOK_ROUTER_SOFTMAX = 0, /* softmax over the experts */
  MOK_ROUTER_SIGMOID = 1  /* sigmoid of each logit */
} mok_router_scoring;

/* Bytes of mok_router_topk's scratch (needed only with counts); 0 if the
 * sizes are invalid. */
size_t mok_router_scratch_bytes(int64_t T, int32_t experts);

/*
 * Top-k routing of T tokens from logits [T, experts] (bf16 or fp32): the
 * router_weights and top_experts that the layer takes.
 *   key   = logit + bias, one fp32 addition (bias fp32 [experts], nullable:
 *           it selects only, the weights do not see it)
 *   ids   int64 [T, k]: the k largest keys in descending order, ties to the
 *         lowest expert id (-0 and +0 tie). A key of -inf is never chosen:
 *         where fewer than k are left, id -1 and weight 0 (mok_build_schedule
 *         does not dispatch such an assignment).
 *   weights fp32 [T, k]: the scores of the chosen, divided by their sum if
 *         `renormalize`, times `scale`. A batch of 32768 tokens or more may
 *         add a token's scores in another order than a smaller one: its ids
 *         are the same, its weights up to 2^-17 of them apart.
 * token_mask (nullable, one byte per token): tokens with a 0 get ids -1 and
 * weights 0, whatever their logits hold. A row with a key that is NaN or
 * +inf has no order: ids -1 and weights NaN.
 * Statistics (counts and losses, both or neither; then scratch is needed):
 *   counts int32 [experts + 1]: choices of each expert, then the number n of
 *         live tokens: kept by the mask, with a key above -inf (or no order)
 *   losses fp32 [2], with p = the scores divided by their sum over the
 *         experts and N = max(n, 1): the load-balance loss experts / (k N^2)
 *         * sum_e counts_e * (sum of p_e over live tokens), and the z loss,
 *         the mean over live tokens of logsumexp(logits)^2 (0 for sigmoid).
 * 1 <= k <= min(experts, 64), experts <= 1024, T * k < 2^31, ld <= 2^22 for
 * T > 1.
 */
mok_status mok_router_topk(const void* logits, int logits_is_fp32, int64_t T, int64_t ld, int32_t experts, int32_t k,
                           const float* bias, const uint8_t* token_mask, int32_t scoring, int renormalize, float scale,
                           float* weights, int64_t* ids, int32_t* counts, float* losses, void* scratch,
                           size_t scratch_bytes, void* stream);

/*
 * Gradient to the logits: d_logits [T, experts] (dense, the logits' type),
 * every element written, from d_weights fp32 [T, k], the forward's ids and,
 * if the losses have a gradient, d_losses fp32 [2] with the forward's counts
 * (both or neither). The choice itself and counts are constants. Choices
 * with an id outside [0, experts) get no gradient, whatever their d_weights
 * hold; tokens that are masked out or have no key above -inf get zeros, a row
 * without an order NaN.
 */
mok_status mok_router_topk_backward(const float* d_weights, const void* logits, int logits_is_fp32, int64_t T,
                                    int64_t ld, int32_t experts, int32_t k, const float* bias,
                                    const uint8_t* token_mask, int32_t scoring, int renormalize, float scale,
                                    const int64_t* ids, const int32_t* counts, const float* d_losses, void* d_logits,
                                    void* stream);

/*
 * One AdamW step of `count` dense tensors. The arrays are host arrays of
 * `count` device pointers, read before the call returns. Set struct_size =
 * sizeof(mok_adamw). Per element, in fp32:
 *   g = grad * grad_scale,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
 *   p = p (1 - lr wd) - lr / (1 - b1^step) * m / (sqrt(v / (1 - b2^step)) + eps)
 * params bf16 or fp32; with masters (bf16 params only) p is the fp32 master
 * and the param receives its rounding. exp_avgs hold m, exp_avg_sqs v, in
 * fp32 (state_bits 32), or (state_bits 8) as E4M3 codes [numel] of m and of
 * sqrt(v), with one E8M0 scale byte per 32 consecutive elements (the last
 * block may be shorter), [ceil(numel/32)]; all-zero bytes are zero moments.
 * A block's scale 2^X is the smallest power of two that keeps its largest
 * magnitude within 448 of it (0xFF, NaN, in both moments if the block's v is
 * not finite). m is rounded to the nearest code, and an m half way between
 * two codes to the even one, or to the smaller one under those scales whose
 * 2^-X the math library's power function gives half a unit low (X = -16 to
 * -20 and some below): the codes are those of the elementary tensor
 * operations on the same GPU, bit for bit. sqrt(v) is rounded to one of the
 * two codes around it, chosen at random so that the mean of its square is v,
 * from `seed` and the element's number in the call (tensors are numbered one
 * after the other, each from a multiple of 32, modulo 2^32): the same seed
 * gives the same bits, and each step should have its own.
 * Tensors of the call must not overlap. grad_scale (nullable): a device
 * fp32, read when the kernel runs. lr, step and seed are values of the call:
 * a captured graph repeats them.
 */
typedef struct mok_adamw {
  uint32_t struct_size;
  int32_t count;
  void* const* params;
  const void* const* grads;
  void* const* masters;           /* NULL: none */
  void* const* exp_avgs;
  void* const* exp_avg_sqs;
  void* const* exp_avg_scales;    /* NULL iff state_bits is 32 */
  void* const* exp_avg_sq_scales;
  const int64_t* numels;
  const float* grad_scale;        /* device; NULL: 1 */
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;                   /* from 1 */
  int32_t param_fp32, grad_fp32;  /* 0: bf16 */
  int32_t state_bits;             /* 32 or 8 */
  uint32_t seed;
} mok_adamw;

mok_status mok_adamw_step(const mok_adamw* step, void* stream);

/* ---- diagnostics (these synchronise; never on the hot path) ---------- */

/* Per-kernel event timing inside a workspace: when enabled, every launch
 * the workspace makes is bracketed by HIP events on the launch stream. */
typedef enum mok_kernel_id {
  MOK_K_SCHED_COUNT = 0, /* per-chunk expert histograms */
  MOK_K_SCHED_SCAN,      /* reserved: the scans run inside the scatter kernel */
  MOK_K_SCHED_SCATTER,   /* scans, ranks and permutation */
  MOK_K_SCHED_MINIBATCH,
  MOK_K_QUANT_X,
  MOK_K_GATE_UP,
  MOK_K_DOWN,
  MOK_K_COMBINE,
  MOK_K_BWD_TRANSPOSE,
  MOK_K_BWD_GATHER,
  MOK_K_BWD_DH,
  MOK_K_BWD_DW_REDUCE,
  MOK_K_BWD_DX_ROWS,
  MOK_K_BWD_DX_SUM,
  MOK_K_BWD_DW,
  MOK_K_BWD_QUANT,
  MOK_K_SCHED_SLICE,     /* token ring: one pass's schedule */
  MOK_K_COUNT
} mok_kernel_id;

const char* mok_kernel_name(int kernel_id);
/* Waits for the device, then returns (and resets) two counts since the last
 * call: *pipeline_timeouts, mover waits of the forward's minibatch pipeline
 * that ran out of time (their minibatches' outputs are then incomplete; 0 in
 * normal operation), and *schedule_mismatches, launches of this workspace
 * that were given a schedule whose header carries another configuration's
 * hash (such a launch does nothing: its outputs are not written). Either
 * pointer may be NULL. Returns MOK_ERR_CONFIG_MISMATCH when
 * schedule_mismatches is non-zero. */
mok_status mok_workspace_read_status(mok_workspace* ws, int32_t* pipeline_timeouts, int32_t* schedule_mismatches);
/* enable != 0: time every kernel; 0: none. */
mok_status mok_workspace_set_timing(mok_workspace* ws, int enable);
/* Time only the kernels whose bit (1 << mok_kernel_id) is set; 0 = none.
 * Each timed launch records two events on its stream, a few microseconds
 * each, so a measurement of the whole step times only what it needs. */
mok_status mok_workspace_set_timing_mask(mok_workspace* ws, uint32_t kernel_mask);
/* Waits for recorded events and returns, per kernel id, the summed
 * milliseconds and number of launches since the last reset; then resets. */
mok_status mok_workspace_read_timing(mok_workspace* ws, float* total_ms, int64_t* launches, int n);

#ifdef __cplusplus
}
#endif

#endif /* MOK_H_ */
