/*
 * moe.h -- C ABI of the GB300 MoE layer hot path (route, dispatch, grouped
 * SwiGLU expert FFN, combine, and the layer's forward and backward).
 *
 * Method: "Enabling trillion-parameter models on AWS EFA" (Licker, Hu,
 * Zaytsev, Chen; 2025).  Section "Introduction": an MoE layer routes each token
 * to a few experts with a small linear router; dispatch groups tokens by
 * expert and combine, its dual, brings the expert outputs back and takes their
 * weighted average.  Section "Send and receive buffers": T tokens, each routed
 * to R of E experts.  Section "Dispatch and combine": per-expert counts and a
 * cumulative sum give the offsets that pack each expert's tokens contiguously
 * for the grouped GEMM.  Here everything runs on one GPU; the page's
 * network send/receive halves have no counterpart.
 *
 * Conventions shared by every entry point
 *  - All tensor pointers are DEVICE pointers owned by the caller; the library
 *    never allocates device memory and never synchronises, unless MOE_CHECK is
 *    passed (then the call waits for its own work and reads the device error
 *    word back).  Work is enqueued on `stream` (a cudaStream_t; NULL means the
 *    legacy default stream).
 *  - bf16 tensors cross the ABI as raw uint16_t bit patterns.  All tensors are
 *    dense row-major; every pointer must be 16-byte aligned and d, f must be
 *    multiples of 8 (rows move as 16-byte vectors), else MOE_ERR_UNSUPPORTED.
 *  - Shapes: T tokens, hidden size d, E experts, top-R routing, expert FFN
 *    width f, N = T*R routed rows.  A "slot" is s = t*R + r (token t, choice r).
 *    Limits: 1 <= R <= 32, R <= E <= 1024, T*R < 2^31.
 *  - Weight layout (nn.Linear [out, in]): W1, W3 bf16 [E, f, d]; W2 bf16
 *    [E, d, f]; the router weight W_g is fp32 [d, E], its bias fp32 [E].
 *  - Workspace: calls that need scratch memory take (ws, ws_bytes).  With
 *    ws == NULL the call only writes the required size to *ws_bytes and
 *    returns MOE_OK.  Otherwise *ws_bytes must be at least that size and ws
 *    256-byte aligned; the workspace must not be shared by calls that may run
 *    concurrently.
 *  - Errors: host-side argument checks return MOE_ERR_INVALID_ARG /
 *    MOE_ERR_UNSUPPORTED / MOE_ERR_WORKSPACE before anything is enqueued; a
 *    failed launch returns MOE_ERR_CUDA.  Kernels that detect bad routing
 *    (expert index outside [0,E) or repeated within a token) or a stalled
 *    pipeline wait set bits in a device error word inside the workspace and
 *    never trap; with MOE_CHECK the call returns MOE_ERR_BAD_ROUTING or
 *    MOE_ERR_TIMEOUT from it.
 */
#ifndef MOE_H_
#define MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,   /* null pointer, negative or inconsistent size */
  MOE_ERR_UNSUPPORTED = 2,   /* misaligned pointer, d or f not a multiple of 8, limits */
  MOE_ERR_WORKSPACE = 3,     /* workspace missing, too small or misaligned */
  MOE_ERR_BAD_ROUTING = 4,   /* device saw an expert index outside [0,E) or a repeat */
  MOE_ERR_TIMEOUT = 5,       /* a bounded pipeline wait gave up (kernel returned early) */
  MOE_ERR_CUDA = 6           /* a CUDA runtime call or launch failed */
} moe_status_t;

typedef void* moe_stream_t;  /* cudaStream_t */

/* flags */
#define MOE_LOGITS_IN 0x1u   /* moe_route: `logits` is an input; skip the gate projection */
#define MOE_CHECK 0x2u       /* wait for the call's work and report device-side errors */
#define MOE_WEIGHTS_PREPACKED 0x4u  /* moe_grouped_ffn / moe_layer_fwd: W1, W3, W2 are the
                                       tiles written by moe_prepack_weights */
#define MOE_SINGLE_CTA_TILES 0x8u   /* moe_grouped_ffn / moe_layer_fwd / moe_layer_bwd: run
                                       the expert GEMMs on single-CTA 128-row tiles instead
                                       of 256-row tiles on CTA pairs (same results, bit for
                                       bit; for comparison) */
#define MOE_SHARED_SERIAL 0x10u     /* moe_layer_fwd / moe_layer_bwd: run the shared expert on the
                                       caller's stream after the routed path instead of on the
                                       library's side stream beside it (same results, bit for
                                       bit; for comparison) */
#define MOE_FP8_DISPATCH 0x20u      /* moe_layer_fwd: dispatch the tokens in block-scaled fp8
                                       (as moe_dispatch_fp8) and give the grouped FFN their
                                       dequantised rows (as moe_dequant_fp8), which saved->x_perm
                                       keeps (a backward treats the quantisation as the
                                       identity); needs d % 128 == 0 and a workspace queried
                                       with this flag */
#define MOE_FP8_MX 0x40u            /* moe_layer_fwd: run the expert FFN on the fp8 tensor cores
                                       in the microscaled fp8 format (moe_dispatch_mx, then
                                       moe_grouped_ffn_mx on layer->mx's weights); saved->o gets
                                       the expert outputs, saved->x_perm, h, a and b are not
                                       written (may be NULL) and moe_layer_bwd does not apply;
                                       needs d, f multiples of 128 and a workspace queried with
                                       this flag */

/* Stages of moe_layer_fwd / moe_layer_bwd, for moe_trace_events. */
typedef enum {
  MOE_STAGE_GATE = 0,      /* router projection (logits) */
  MOE_STAGE_TOPK,          /* softmax top-R */
  MOE_STAGE_DISPATCH,      /* histogram, scan, stable rank, row copies */
  MOE_STAGE_GATEUP,        /* tile list + grouped x W1^T | x W3^T with the SwiGLU epilogue */
  MOE_STAGE_DOWN,          /* grouped h W2^T */
  MOE_STAGE_COMBINE,       /* weighted gather-sum */
  MOE_STAGE_BWD_ROUTE,     /* dw, do, router logit gradient */
  MOE_STAGE_BWD_DH,        /* tile list + grouped do W2 with the SwiGLU backward epilogue */
  MOE_STAGE_BWD_DX,        /* grouped [da|db] [W1;W3] */
  MOE_STAGE_BWD_WG2,       /* dW2 = do^T h per expert */
  MOE_STAGE_BWD_WG13,      /* [dW1;dW3] = [da|db]^T x_perm per expert */
  MOE_STAGE_BWD_DWG,       /* router weight gradient */
  MOE_STAGE_BWD_DXC,       /* W_g transpose + dx gather-sum */
  MOE_STAGE_SHARED_FWD,    /* shared expert forward (side stream unless MOE_SHARED_SERIAL) */
  MOE_STAGE_SHARED_BWD,    /* shared expert backward (same stream rule) */
  MOE_STAGE_COUNT
} moe_stage_t;

/*
 * moe_trace_events -- per-stage timing (utility; the page has no counterpart).
 * events: NULL to disable, else 2*MOE_STAGE_COUNT cudaEvent_t handles created
 * by the caller on the current device; while set, moe_layer_fwd and
 * moe_layer_bwd record events[2*i] on their stream just before stage i and
 * events[2*i+1] just after it (the shared-expert stages on the stream that
 * runs them).  The pointer is kept (not copied) until the
 * next call; one setting is shared by all threads of the process.
 */
moe_status_t moe_trace_events(void* const* events);

/* Number of CUDA kernels this library has launched in this process (utility). */
unsigned long long moe_kernel_launches(void);

/*
 * moe_selftest_wait_timeout -- failure-detection self-test (utility; the page
 * has no counterpart).  Launches one small block whose pipeline wait is on an
 * mbarrier that nothing ever arrives on, through the same bounded-wait routine
 * the GEMM pipelines use, with a limit of limit_us microseconds (1..10^6).  The
 * wait gives up, the kernel records the timeout in ws (at least 256 bytes,
 * 256-byte aligned, device memory) and returns; the call waits for it and
 * returns MOE_ERR_TIMEOUT when the timeout was detected and reported, MOE_OK if
 * the wait was (wrongly) satisfied.  The GPU context stays usable.
 */
moe_status_t moe_selftest_wait_timeout(unsigned limit_us, void* ws, moe_stream_t stream);

/* Human-readable name of a status code (static string). */
const char* moe_status_string(moe_status_t status);

/* Library version, major*10000 + minor*100 + patch. */
int moe_version(void);

/* The cudaError_t behind the calling thread's most recent MOE_ERR_CUDA (0 if
 * none yet); for diagnostics. */
int moe_last_cuda_error(void);

/*
 * moe_route -- the router: a small linear layer scores the experts and the R
 * best are chosen for each token (section "Introduction").
 *   logits[t,e] = sum_k x[t,k] * W_g[k,e] + bias[e]        (fp32 accumulation)
 *   idx[t,0..R-1] = the R experts of largest logit, ordered by (logit desc,
 *                   expert index asc): ties go to the lower index
 *   w[t,r] = exp(l_{idx[t,r]} - l_{idx[t,0]}) / sum_s exp(l_{idx[t,s]} - l_{idx[t,0]})
 *            (softmax over the chosen experts: the weights sum to 1)
 * x: bf16 [T,d]; w_gate: fp32 [d,E]; bias: fp32 [E] or NULL.
 * logits: fp32 [T,E], written (or read, with MOE_LOGITS_IN: then x, w_gate
 * and bias are ignored and may be NULL).  topk_idx: int32 [T,R]; topk_w: fp32
 * [T,R].  Logits must be finite.
 * Workspace (two-call convention; ignored with MOE_LOGITS_IN): when d is a
 * multiple of 64 the projection runs on the tensor cores with W_g split into
 * three bf16 terms (hi + mid + lo carry its fp32 significand; products with
 * the bf16 x are exact), which needs 6*E*d bytes of workspace; otherwise an
 * fp32 FMA kernel runs and the workspace holds only the error word.
 */
moe_status_t moe_route(const uint16_t* x, const float* w_gate, const float* bias,
                       int T, int d, int E, int R, float* logits,
                       int32_t* topk_idx, float* topk_w, void* ws, size_t* ws_bytes,
                       unsigned flags, moe_stream_t stream);

/*
 * moe_dispatch -- group the routed tokens by expert (section "Dispatch and
 * combine": per-expert counts, their cumulative sum as offsets, tokens packed
 * contiguously per expert into the grouped-GEMM input).
 *   counts[e]  = #{slots s : topk_idx[s] == e}
 *   offsets    = exclusive prefix sum of counts, offsets[E] = T*R
 *   rows offsets[e] .. offsets[e+1]-1 belong to expert e, in ascending token order
 *   row_slot[row] = s,  slot_row[s] = row  (inverse maps)
 *   x_perm[row]   = x[row_slot[row] / R]   (bit copy)
 * x: bf16 [T,d] (may be NULL together with x_perm: plan only); topk_idx:
 * int32 [T,R]; counts int32 [E]; offsets int32 [E+1]; row_slot, slot_row
 * int32 [T*R]; x_perm bf16 [T*R, d].  Needs a workspace (per-block expert
 * histograms and the error word).  Deterministic: the result does not depend
 * on scheduling.
 */
moe_status_t moe_dispatch(const uint16_t* x, const int32_t* topk_idx, int T, int d, int E, int R,
                          int32_t* counts, int32_t* offsets, int32_t* row_slot, int32_t* slot_row,
                          uint16_t* x_perm, void* ws, size_t* ws_bytes, unsigned flags,
                          moe_stream_t stream);

/*
 * moe_dispatch_fp8 -- dispatch in block-scaled fp8 (section "Evaluation": the
 * page dispatches tokens in block-scaled fp8 and combines in bf16).  Same plan
 * as moe_dispatch (counts, offsets, row_slot, slot_row); instead of bf16 rows
 * it writes, per row and per 128-channel block b of the row's token x_t:
 *   xscale_perm[row, b] = amax_b / 448          (fp32; amax_b = max |x_t| over the block)
 *   xq_perm[row, c]     = E4M3(x_t[c] / xscale) (OCP E4M3 codes, round to nearest
 *                                                even, saturating at +-448)
 * An all-zero block has scale 0 and zero codes; code * scale approximates x
 * within half an E4M3 step (2^-4 relative).  d must be a multiple of 128.
 * xq_perm: uint8 [T*R, d]; xscale_perm: fp32 [T*R, d/128].  Workspace as for
 * moe_dispatch.
 */
moe_status_t moe_dispatch_fp8(const uint16_t* x, const int32_t* topk_idx, int T, int d, int E,
                              int R, int32_t* counts, int32_t* offsets, int32_t* row_slot,
                              int32_t* slot_row, uint8_t* xq_perm, float* xscale_perm, void* ws,
                              size_t* ws_bytes, unsigned flags, moe_stream_t stream);

/*
 * moe_dequant_fp8 -- out[i, c] = bf16(E4M3 value of xq[i, c] * xscale[i, c/128])
 * for N rows of width d (d a multiple of 128): the identity expert on
 * fp8-dispatched rows.  xq: uint8 [N, d]; xscale: fp32 [N, d/128]; out: bf16
 * [N, d].  No workspace.
 */
moe_status_t moe_dequant_fp8(const uint8_t* xq, const float* xscale, int N, int d, uint16_t* out,
                             moe_stream_t stream);

/*
 * moe_grouped_ffn -- the grouped GEMMs that apply each expert's weights to its
 * rows (section "MoE all-to-all over EFA"), as a SwiGLU FFN.  For every expert
 * e and row i in [offsets[e], offsets[e+1]):
 *   a = x_perm[i] W1[e]^T,  b = x_perm[i] W3[e]^T      (fp32 accumulation)
 *   h[i]   = bf16(silu(a) * b),   silu(a) = a / (1 + exp(-a))
 *   out[i] = bf16(s_i * (h[i] W2[e]^T)),   s_i = row_scale[i], or 1 when row_scale is NULL
 * x_perm: bf16 [N,d]; offsets: int32 [E+1] on the device with offsets[E] == N;
 * W1, W3: bf16 [E,f,d]; W2: bf16 [E,d,f]; row_scale: fp32 [N] or NULL -- e.g.
 * each row's gate weight, so that an unweighted moe_combine (topk_w NULL) of
 * the outputs sums already-weighted rows (the weighting moved to the expert
 * side, before the output's bf16 rounding); h: bf16 [N,f] (written, kept for
 * the backward); a_save, b_save: bf16 [N,f] or NULL (bf16(a), bf16(b) for the
 * backward); out: bf16 [N,d].  Needs a workspace (tile list, error word).
 */
moe_status_t moe_grouped_ffn(const uint16_t* x_perm, const int32_t* offsets, int N, int d, int f,
                             int E, const uint16_t* W1, const uint16_t* W3, const uint16_t* W2,
                             const float* row_scale, uint16_t* a_save, uint16_t* b_save,
                             uint16_t* h, uint16_t* out, void* ws, size_t* ws_bytes,
                             unsigned flags, moe_stream_t stream);

/*
 * moe_grouped_ffn_fp8 -- moe_grouped_ffn on the block-scaled fp8 rows that
 * moe_dispatch_fp8 writes (section "Evaluation": tokens travel in
 * block-scaled fp8).  The rows are dequantised once, as moe_dequant_fp8 does
 * (bf16(code value * scale)), into the workspace, and the bf16 grouped FFN
 * runs on them: every output equals that of moe_dequant_fp8 followed by
 * moe_grouped_ffn, bit for bit, in one call.
 * xq_perm: uint8 [N, d], 16-byte aligned; xscale_perm: fp32 [N, d/128];
 * d must be a multiple of 128 (else MOE_ERR_UNSUPPORTED).  The workspace is
 * that of moe_grouped_ffn plus N * d * 2 bytes (rounded up to 256).  Every
 * other argument and the flags as for moe_grouped_ffn.
 */
moe_status_t moe_grouped_ffn_fp8(const uint8_t* xq_perm, const float* xscale_perm,
                                 const int32_t* offsets, int N, int d, int f, int E,
                                 const uint16_t* W1, const uint16_t* W3, const uint16_t* W2,
                                 const float* row_scale, uint16_t* a_save, uint16_t* b_save,
                                 uint16_t* h, uint16_t* out, void* ws, size_t* ws_bytes,
                                 unsigned flags, moe_stream_t stream);

/*
 * Microscaled fp8 ("MX") operands for expert GEMMs that take fp8 directly
 * (section "Evaluation": the tokens travel as block-scaled fp8; here the
 * tensor cores multiply the fp8 codes themselves).  A matrix [rows, K] becomes
 * E4M3 codes uint8 [rows, K] and one UE8M0 scale byte per 32 consecutive
 * elements of a row along K, stored in rows of sk = 16 * ceil(K / 512) bytes
 * (K/32 bytes, padded to a multiple of 16), uint8 [rows, sk].  A block's scale
 * is 2^k with k the smallest integer such that 448 * 2^k >= the block's
 * largest magnitude (clamped to [-127, 127]; an all-zero block gets k = -127),
 * stored as k + 127; codes are the E4M3 values nearest x / 2^k, ties to even
 * (no code saturates).  value = E4M3(code) * 2^(scale - 127).
 */

/*
 * moe_quantize_mx -- codes and scales of a bf16 matrix W [rows, K] along K (K a
 * multiple of 32): codes uint8 [rows, K], scales uint8 [rows, sk].  Used once for
 * the expert weights (W1, W3 as [E*f, d]; W2 as [E*d, f]) before
 * moe_grouped_ffn_mx.  All pointers 16-byte aligned.  No workspace.
 */
moe_status_t moe_quantize_mx(const uint16_t* W, long long rows, int K, uint8_t* codes,
                             uint8_t* scales, moe_stream_t stream);

/*
 * moe_dispatch_mx -- moe_dispatch whose rows are written in the microscaled
 * fp8 format above (codes xq_perm uint8 [T*R, d], scales xscale_perm uint8
 * [T*R, sk(d)]) instead of bf16: the same plan (counts, offsets, row_slot,
 * slot_row), each token's row quantised once and copied to its R rows.
 * d must be a multiple of 128.  Workspace as for moe_dispatch.
 */
moe_status_t moe_dispatch_mx(const uint16_t* x, const int32_t* topk_idx, int T, int d, int E, int R,
                             int32_t* counts, int32_t* offsets, int32_t* row_slot,
                             int32_t* slot_row, uint8_t* xq_perm, uint8_t* xscale_perm, void* ws,
                             size_t* ws_bytes, unsigned flags, moe_stream_t stream);

/*
 * moe_grouped_ffn_mx -- the grouped SwiGLU FFN with fp8 tensor-core GEMMs on
 * microscaled operands (tcgen05 block-scaled fp8 multiply, fp32 accumulation).
 * For every expert e and row i in [offsets[e], offsets[e+1]), with every
 * operand taken at its dequantised value:
 *   a = x_i W1[e]^T,  b = x_i W3[e]^T,  h_i = silu(a) * b           (fp32)
 *   (hq_i, hs_i) = the microscaled fp8 form of h_i along f
 *   out_i = bf16(s_i * (h~_i W2[e]^T))   h~ = dequantised h, s_i = row_scale[i] or 1
 * xq, xs: the rows (moe_dispatch_mx); W1q/W1s, W3q/W3s: [E*f, d] codes and
 * scales, W2q/W2s: [E*d, f] (moe_quantize_mx); hq uint8 [N, f] and hs uint8
 * [N, sk(f)] receive h (or NULL: kept in the workspace); out bf16 [N, d].
 * d and f must be multiples of 128 (else MOE_ERR_UNSUPPORTED).  Needs a
 * workspace (error word, tile list, and h when hq/hs are NULL).
 */
moe_status_t moe_grouped_ffn_mx(const uint8_t* xq, const uint8_t* xs, const int32_t* offsets,
                                int N, int d, int f, int E, const uint8_t* W1q,
                                const uint8_t* W1s, const uint8_t* W3q, const uint8_t* W3s,
                                const uint8_t* W2q, const uint8_t* W2s, const float* row_scale,
                                uint8_t* hq, uint8_t* hs, uint16_t* out, void* ws,
                                size_t* ws_bytes, unsigned flags, moe_stream_t stream);

/*
 * moe_prepack_weights -- copy the expert weights into the tile layout the
 * forward grouped GEMMs stream (a performance layout for forward-only use, e.g.
 * inference; the page's grouped GEMMs take the weights as they are):
 *   W1p, W3p[e][j][k][r][c] = W1, W3[e][128 j + r][64 k + c]   ([E][f/128][d/64][128][64])
 *   W2p[e][j][k][r][c]      = W2[e][256 j + r][64 k + c]       ([E][d/256][f/64][256][64])
 * so that every 128x64 (W1, W3) or 256x64 (W2) box the GEMM loads is one
 * contiguous 16 or 32 KB region.  Requires d % 256 == 0 and f % 128 == 0.
 * Pass MOE_WEIGHTS_PREPACKED to moe_grouped_ffn / moe_layer_fwd to use them
 * (same results, bit for bit); moe_layer_bwd takes the plain layout only.
 * W1p, W3p, W2p: bf16, the sizes of W1, W3, W2; must not alias them.
 */
moe_status_t moe_prepack_weights(const uint16_t* W1, const uint16_t* W3, const uint16_t* W2, int E,
                                 int d, int f, uint16_t* W1p, uint16_t* W3p, uint16_t* W2p,
                                 moe_stream_t stream);

/*
 * moe_combine -- bring each token's R expert outputs back and take their
 * gate-weighted sum (sections "Introduction" and "Dispatch and combine"):
 *   y[t] = bf16( sum_{r=0..R-1} topk_w[t,r] * expert_out[slot_row[t*R+r]] )
 * accumulated in fp32 in r order (bitwise reproducible).  topk_w NULL means
 * unweighted.  expert_out: bf16 [T*R,d]; slot_row: int32 [T*R]; y: bf16 [T,d].
 * Rows outside [0, T*R) contribute nothing.  No workspace.
 */
moe_status_t moe_combine(const uint16_t* expert_out, const int32_t* slot_row, const float* topk_w,
                         int T, int d, int R, uint16_t* y, moe_stream_t stream);

/*
 * moe_dispatch_noalloc -- moe_dispatch without a workspace argument, for
 * callers that cannot allocate device memory: code running inside a host
 * application or framework whose allocator owns all device memory, and
 * latency-critical loops that cannot afford cudaMalloc's implicit device
 * synchronisation.  (The page has no counterpart; this is a packaging of the
 * dispatch step above.)
 * Same arguments, results and error behaviour as moe_dispatch.  Its scratch
 * (the device error word and 2*E*ceil(T/256) int32 histogram entries) lives in
 * a 4 MiB array that the library reserves statically on every GPU that loads
 * it, until the process exits; calls whose scratch would not fit
 * (256 + 8*E*ceil(T/256) bytes, rounded up to 256, above 4 MiB) return
 * MOE_ERR_WORKSPACE before anything is enqueued.  It calls no cudaMalloc,
 * cudaFree or other allocating routine.  The first call on each device looks
 * up the array's device address (set-up; make that first call before any
 * stream capture).  Every call uses the same array and clears its error word
 * first; calls that may overlap on the GPU (different streams, or different
 * host threads) race on it and must be serialised by the caller.
 */
moe_status_t moe_dispatch_noalloc(const uint16_t* x, const int32_t* topk_idx, int T, int d, int E,
                                  int R, int32_t* counts, int32_t* offsets, int32_t* row_slot,
                                  int32_t* slot_row, uint16_t* x_perm, unsigned flags,
                                  moe_stream_t stream);

/* Layer parameters (device pointers, caller-owned). */
/*
 * Optional shared expert (section "Introduction": while dispatch is in
 * flight the GPU can do other work, such as the shared expert's
 * multiplication).  A SwiGLU FFN that every token passes through, added to
 * the routed experts' weighted sum with weight 1:
 *   s_t = bf16( bf16(silu(x_t Ws1^T) * (x_t Ws3^T)) Ws2^T ),
 *   y_t = bf16( s_t + sum_r w[t,r] o[slot_row[t*R+r]] ).
 * The forward runs it on a side stream the library owns (one per device),
 * forked from the caller's stream after the gate projection and joined before
 * combine, so it overlaps top-R and dispatch; the backward forks it at the
 * start and joins it before the dx gather.  Callers see ordinary stream
 * semantics on their stream.
 */
typedef struct {
  int fs;               /* hidden size; multiple of 8 (of 64 for the backward) */
  const uint16_t* W1;   /* bf16 [fs,d] */
  const uint16_t* W3;   /* bf16 [fs,d] */
  const uint16_t* W2;   /* bf16 [d,fs] */
  float* dW1;           /* moe_layer_bwd outputs, fp32 [fs,d], [fs,d], [d,fs]; */
  float* dW3;           /*   unused by the forward (may be NULL there)        */
  float* dW2;
} moe_shared_t;

/* The expert weights in the microscaled fp8 format (moe_quantize_mx along each
 * matrix's K): W1q, W3q uint8 [E*f, d] with scales uint8 [E*f, sk(d)]; W2q
 * uint8 [E*d, f] with scales uint8 [E*d, sk(f)]. */
typedef struct {
  const uint8_t* W1q;
  const uint8_t* W1s;
  const uint8_t* W3q;
  const uint8_t* W3s;
  const uint8_t* W2q;
  const uint8_t* W2s;
} moe_mx_weights_t;

typedef struct {
  int T, d, E, R, f;
  const float* w_gate;  /* fp32 [d,E] */
  const float* bias;    /* fp32 [E] or NULL */
  const uint16_t* W1;   /* bf16 [E,f,d] */
  const uint16_t* W3;   /* bf16 [E,f,d] */
  const uint16_t* W2;   /* bf16 [E,d,f] */
  const moe_shared_t* shared;   /* NULL: no shared expert */
  const moe_mx_weights_t* mx;   /* microscaled fp8 expert weights for MOE_FP8_MX, or NULL */
} moe_layer_t;

/* Forward intermediates (caller-owned device buffers, written by the forward,
 * read by the backward).  N = T*R. */
typedef struct {
  float* logits;       /* fp32 [T,E] */
  int32_t* topk_idx;   /* int32 [T,R] */
  float* topk_w;       /* fp32 [T,R] */
  int32_t* counts;     /* int32 [E] */
  int32_t* offsets;    /* int32 [E+1] */
  int32_t* row_slot;   /* int32 [N] */
  int32_t* slot_row;   /* int32 [N] */
  uint16_t* x_perm;    /* bf16 [N,d] */
  uint16_t* a;         /* bf16 [N,f] or NULL (inference: nothing saved for the backward) */
  uint16_t* b;         /* bf16 [N,f] or NULL (must be NULL iff a is) */
  uint16_t* h;         /* bf16 [N,f] */
  uint16_t* o;         /* bf16 [N,d] expert outputs */
  /* shared expert (only read when the layer has one): its pre-activations
   * and hidden rows for the backward, bf16 [T,fs]; all three NULL for
   * inference (the forward then keeps its hidden rows in the workspace) */
  uint16_t* sa;
  uint16_t* sb;
  uint16_t* sh;
} moe_saved_t;

/*
 * moe_layer_fwd -- y = combine(FFN(dispatch(x, route(x)))): route, dispatch,
 * grouped SwiGLU FFN and combine, as the entry points above define them.
 * x: bf16 [T,d]; y: bf16 [T,d]; saved: all intermediates (a and b may be NULL).
 * With layer->shared, y also adds the shared expert's output (moe_shared_t);
 * saved->sa, sb, sh then hold its intermediates (all NULL for inference).
 */
moe_status_t moe_layer_fwd(const moe_layer_t* layer, const uint16_t* x, uint16_t* y,
                           const moe_saved_t* saved, void* ws, size_t* ws_bytes, unsigned flags,
                           moe_stream_t stream);

/*
 * moe_layer_bwd -- gradients of a loss L given dy = dL/dy (bf16 [T,d]), from
 * the intermediates of moe_layer_fwd (which must have saved a and b):
 *   dw[t,r]  = <dy_t, o_row>,  do_row = bf16(w[t,r] dy_t)      (row = slot_row[t*R+r])
 *   per expert: dh = do W2[e];  da = bf16(dh * b * silu'(a)),  db = bf16(dh * silu(a))
 *               dx_perm = bf16(da W1[e] + db W3[e])
 *               dW2[e] = do^T h,  dW1[e] = da^T x_perm,  dW3[e] = db^T x_perm
 *   router:  dlogits[t, idx[t,q]] = w_q (dw_q - sum_r w_r dw_r), 0 for unchosen experts
 *            dW_gate = x^T dlogits
 *   dx_t = bf16( sum_r dx_perm[row(t,r)] + dlogits_t W_g^T [+ dxs_t] )
 *   shared expert (layer->shared; saved->sa, sb, sh required), with dy as its
 *   output gradient:  dhs = dy Ws2;  das = bf16(dhs * sb * silu'(sa)),
 *   dbs = bf16(dhs * silu(sa));  dxs = bf16(das Ws1 + dbs Ws3);
 *   shared->dW2 = dy^T sh,  shared->dW1 = das^T x,  shared->dW3 = dbs^T x
 * (a, b as saved in bf16; silu'(a) = s(a)(1 + a(1 - s(a))), s the logistic
 * function.)  x: bf16 [T,d]; dx: bf16 [T,d]; dW_gate: fp32 [d,E]; dW1, dW3:
 * fp32 [E,f,d]; dW2: fp32 [E,d,f] -- all overwritten (experts with no rows get
 * zero gradients).  The router bias is treated as a constant.
 */
moe_status_t moe_layer_bwd(const moe_layer_t* layer, const uint16_t* x, const moe_saved_t* saved,
                           const uint16_t* dy, uint16_t* dx, float* dW_gate, float* dW1,
                           float* dW3, float* dW2, void* ws, size_t* ws_bytes, unsigned flags,
                           moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Around the layer in a training step: rows sorted for experts of the
 * caller's own and brought back, with their gradients; the embedding that
 * makes x out of token ids, with its gradient; the optimiser step on the
 * gradients that moe_layer_bwd writes.  (The page has no counterpart of the
 * last two.)  These calls take bf16, fp16 and fp32 data, any row length, rows
 * apart by any stride (in elements, at least the row length) and pointers
 * aligned to their element; 16-byte aligned rows of a multiple of 16 bytes
 * move fastest.  Outputs must not overlap inputs.
 */
typedef enum {
  MOE_BF16 = 0,
  MOE_F16 = 1,
  MOE_F32 = 2
} moe_dtype_t;

#define MOE_ACCUMULATE 0x80u        /* moe_embed_bwd, moe_product_fp8_dw: add to the output instead
                                       of overwriting it */

/*
 * moe_sort_rows_bound -- the number of rows that holds every plan of moe_sort
 * for these arguments, whatever the routing:
 *   min( floor_to_align(T*R + min(E, T*R) * (align - 1)), E * ceil_to_align(capacity) )
 * (the second term only with capacity > 0).  -1 for arguments moe_sort refuses.
 */
long long moe_sort_rows_bound(int T, int R, int E, int align, int capacity);

/*
 * moe_sort -- the plan that groups slots by expert, for experts that moe_dispatch
 * does not serve: slots may be empty, an expert may take a limited number of
 * rows, and each expert's rows may start at a multiple of a tile.
 *   topk_idx[t,r] = -1: the slot is empty (e.g. its expert lives elsewhere)
 *   counts[e]  = min(#{slots s : topk_idx[s] == e}, capacity)   (capacity <= 0: no limit)
 *   offsets[e] = sum_{e' < e} counts[e'] rounded up to a multiple of align; offsets[E] = the end
 *   rows offsets[e] .. offsets[e] + counts[e] - 1 are expert e's first counts[e]
 *   slots, in ascending slot order
 *   row_slot[row] = s, or -1 for a row without a slot;  slot_row[s] = row, or -1
 * topk_idx, slot_row: int32 [T,R]; counts int32 [E]; offsets int32 [E+1]; row_slot
 * int32 [N] with N at least moe_sort_rows_bound(...) (all N entries are written).
 * An expert may appear twice in a token.  Entries outside [-1, E) count as
 * empty and are reported (MOE_ERR_BAD_ROUTING with MOE_CHECK).  1 <= align <= 4096;
 * T*R and N below 2^31.  Needs a workspace (error word).  Deterministic.
 */
moe_status_t moe_sort(const int32_t* topk_idx, int T, int E, int R, int align, int capacity, int N,
                      int32_t* counts, int32_t* offsets, int32_t* row_slot, int32_t* slot_row,
                      void* ws, size_t* ws_bytes, unsigned flags, moe_stream_t stream);

/*
 * moe_permute -- tokens to their rows, optionally times their weights:
 *   rows[slot_row[t,r]] = w[t,r] * x[t]   (fp32 product, one rounding; w NULL: a copy)
 *   rows[i] = 0 where row_slot[i] < 0
 * x: [T,d], rows: [N,d] of type dtype, row strides ldx, ld_rows; w fp32 [T,R] or
 * NULL; row_slot [N] and slot_row [T,R] from moe_sort.  No workspace.
 */
moe_status_t moe_permute(const void* x, long long ldx, const float* w, const int32_t* row_slot,
                         const int32_t* slot_row, int T, int d, int R, int N, int dtype,
                         void* rows, long long ld_rows, moe_stream_t stream);

/*
 * moe_permute_bwd -- gradient of moe_permute, given drows = dL/drows:
 *   dx[t]   = sum_r w[t,r] * drows[slot_row[t,r]]      (fp32 sum in r order, one rounding)
 *   dw[t,r] = <x[t], drows[slot_row[t,r]]>             (fp32; dw and x both NULL: not computed)
 * Slots without a row contribute nothing and get dw = 0; rows without a slot are
 * not read.
 */
moe_status_t moe_permute_bwd(const void* drows, long long ld_drows, const int32_t* slot_row,
                             const float* w, const void* x, long long ldx, int T, int d, int R,
                             int N, int dtype, void* dx, long long ld_dx, float* dw,
                             moe_stream_t stream);

/*
 * moe_unpermute -- rows back to their tokens, summed with their weights:
 *   y[t] = sum_r w[t,r] * rows[slot_row[t,r]]     (fp32 sum in r order, one rounding)
 * w NULL: weight 1.  A token without rows gets zeros.
 */
moe_status_t moe_unpermute(const void* rows, long long ld_rows, const int32_t* slot_row,
                           const float* w, int T, int d, int R, int N, int dtype, void* y,
                           long long ldy, moe_stream_t stream);

/*
 * moe_unpermute_bwd -- gradient of moe_unpermute, given dy = dL/dy:
 *   drows[slot_row[t,r]] = w[t,r] * dy[t],  drows[i] = 0 where row_slot[i] < 0
 *   dw[t,r] = <dy[t], rows[slot_row[t,r]]>  (fp32; dw and rows both NULL: not computed)
 */
moe_status_t moe_unpermute_bwd(const void* dy, long long ld_dy, const int32_t* row_slot,
                               const int32_t* slot_row, const float* w, const void* rows,
                               long long ld_rows, int T, int d, int R, int N, int dtype,
                               void* drows, long long ld_drows, float* dw, moe_stream_t stream);

/*
 * moe_embed -- out[i] = scale * table[ids[i]], zeros where ids[i] is outside
 * [0, V) (a position without a token).  ids: int32 or int64 (ids_bytes 4 or 8)
 * [n]; table [V,d] of table_dtype, out [n,d] of out_dtype, row strides ld_table,
 * ld_out.  n < 2^31.  No workspace.
 */
moe_status_t moe_embed(const void* ids, int ids_bytes, long long n, const void* table,
                       long long ld_table, int V, int d, int table_dtype, float scale, void* out,
                       long long ld_out, int out_dtype, moe_stream_t stream);

/*
 * moe_embed_bwd -- gradient of moe_embed with respect to the table:
 *   dtable[v] = scale * sum_{i : ids[i] == v} dout[i]
 * (fp32 sums in an order fixed by the ids, one rounding).  Every row is written;
 * with MOE_ACCUMULATE the sum is added to dtable and rows without a token are
 * left alone.  Ids below 0 contribute nothing; ids >= V neither, and are
 * reported (MOE_ERR_BAD_ROUTING with MOE_CHECK).  dout [n,d] of dout_dtype;
 * dtable [V,d] of dtable_dtype.  n < 2^30, V <= 2^30.  Needs a workspace (error
 * word, sorted ids, partial sums).
 */
moe_status_t moe_embed_bwd(const void* dout, long long ld_dout, const void* ids, int ids_bytes,
                           long long n, int V, int d, int dout_dtype, float scale, void* dtable,
                           long long ld_dtable, int dtable_dtype, void* ws, size_t* ws_bytes,
                           unsigned flags, moe_stream_t stream);

/*
 * One tensor of an optimiser step: n elements, contiguous.  p_dtype MOE_BF16 or
 * MOE_F32; g_dtype MOE_BF16 or MOE_F32.  master: fp32 [n] copy that the step
 * updates in p's place (p then gets its rounding), or NULL; only with a bf16 p.
 * state_bits 32: m, v fp32 [n], scales NULL.  state_bits 8: E4M3 codes uint8 [n]
 * with one fp32 scale per 256 consecutive elements (m_scale, v_scale:
 * fp32 [ceil(n/256)]), m = code * m_scale and sqrt(v) = code * v_scale.  All
 * zeros is the state before the first step.
 */
typedef struct {
  void* p;
  float* master;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  long long n;
  double weight_decay;
  int p_dtype;
  int g_dtype;
  int state_bits;
} moe_adamw_tensor_t;

/* Settings of a step; step counts from 1.  seed: dither of the 8-bit states,
 * another one each step (e.g. the step's number). */
typedef struct {
  double lr, beta1, beta2, eps;
  long long step;
  uint32_t seed;
} moe_adamw_t;

/*
 * moe_grad_norm -- the L2 norm over all gradients of a list and the factor that
 * clips it, left on the device for moe_adamw_step:
 *   norm[0] = sqrt(sum g^2),  norm[1] = min(1, max_norm / (norm[0] + 1e-6))
 *   (1 when max_norm <= 0),   norm[2] = 1 if norm[0] is finite, else 0,  norm[3] = 0
 * tensors: host array of n_tensors (only g, g_dtype and n are used; read before
 * the call returns).  norm: fp32 [4] on the device.  Squares are summed in fp32
 * over eight elements and in pairs of fp32 numbers (46 bits) from there, in a
 * fixed order.  A norm above 1.8e19 (its square above the fp32 range) is infinite,
 * as with an infinite gradient: norm[1] is then 0 with a limit; with a NaN norm[0]
 * and norm[1] are NaN.  Needs a workspace.
 */
moe_status_t moe_grad_norm(const moe_adamw_tensor_t* tensors, int n_tensors, double max_norm,
                           float* norm, void* ws, size_t* ws_bytes, moe_stream_t stream);

/*
 * moe_adamw_step -- one AdamW step on every tensor of a list, in place:
 *   g' = norm[1] * g  (norm NULL: g)
 *   m = beta1 m + (1 - beta1) g',   v = beta2 v + (1 - beta2) g'^2
 *   p = p (1 - lr * weight_decay) - lr / (1 - beta1^step) * m /
 *       (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * in fp32, p rounded once to its type; the quotient by an approximate reciprocal,
 * with 32-bit states the root too (each within 2^-23 of itself).  With norm and
 * norm[2] == 0 nothing is changed.
 * 8-bit states are rounded after the update has used them: per block, scale =
 * max * (1/448) and code = |value| * (1/scale) rounded to one of its two E4M3
 * neighbours by adding 20 dither bits below the kept mantissa bits; sqrt(v) > 0
 * never rounds to 0.  Their m, v, sqrt(v), scales and codes are computed operation
 * by operation, each rounded to nearest, so they can be reproduced bit for bit.
 * Element i of the k-th tensor takes the dither
 *   h = mix(floor(i/2) * 0x9E3779B1 + mix(seed + k * 0x9E3779B1))   (mod 2^32)
 *   mix(x): x = (x ^ x>>16) * 0x6A09E667; x = (x ^ x>>15) * 0xBB67AE85; x ^ x>>16
 *   dither = 16 * (i even ? h mod 2^16 : h >> 16) + 8
 * Without norm the gradients and their squares have to be finite in fp32: one that
 * is not makes its parameter NaN or leaves the states of its block without meaning.
 * Arrays aligned to eight of their elements move fastest; a tensor with one that is
 * not takes up to 2.2 times as long.
 * No workspace; the list and the settings travel in the launch.  In a captured
 * graph that makes every replay the same step, with the lr, bias correction and
 * dither of the capture: capture the rest of a training step and call this one
 * itself, or capture it anew and update the graph before each step.  Tensors must
 * not overlap.
 * step >= 1, 0 <= beta < 1, eps at least the smallest normal fp32 number.
 */
moe_status_t moe_adamw_step(const moe_adamw_tensor_t* tensors, int n_tensors,
                            const moe_adamw_t* settings, const float* norm, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Routing by scores, and products of the experts on block-scaled fp8.  (The pages
 * name a linear router and block-scaled fp8 rows; scores, groups and products on
 * those rows are this library's.)  Around experts of the caller's own: moe_route_scores
 * -> moe_sort -> moe_permute -> moe_quantize_fp8 -> moe_product_fp8 -> ... ->
 * moe_unpermute, and back.  Outputs must not overlap inputs.
 */
typedef enum {
  MOE_SCORE_SOFTMAX = 0,   /* over all E experts */
  MOE_SCORE_SIGMOID = 1
} moe_score_t;

typedef struct {
  int score;         /* moe_score_t */
  int groups;        /* groups of E / groups neighbouring experts; 1..32, divides E */
  int top_groups;    /* groups whose experts may be chosen */
  int group_keys;    /* 1 or 2: a group's worth is the sum of its so many largest keys */
  int renormalise;   /* the weights are divided by their sum */
  float scale;       /* and multiplied by this */
} moe_router_t;

/*
 * moe_route_scores -- the experts of each token from its logits:
 *   s = softmax(l) or sigmoid(l);  key = s + bias (a balance bias, e.g. raised for
 *   experts with few tokens; NULL: none)
 *   the top_groups groups of largest worth take part (ties: the lower group)
 *   idx[t,:] = the R experts of largest key, in that order, ties to the lower expert
 *   w[t,r] = scale * s[idx]                      renormalise == 0
 *   w[t,r] = scale * s[idx] / sum_j s[idx[t,j]]  renormalise != 0
 * The choice is that of keys computed in 64 bits from the logits and biases as they are
 * stored; without a bias experts (and groups, with group_keys 1) are ordered by their logits,
 * which for numbers is the same order.
 * A logit of -inf closes its expert for the token: it has score 0 and is never chosen; nor
 * is one whose bias is -inf.  Slots that no expert is left for get idx -1, w 0 (as moe_sort
 * takes them).  NaN comes before all other keys and logits.  A sigmoid of NaN is NaN; a softmax
 * over a logit of NaN or +inf is NaN for all its experts: where the choice goes by keys the lowest
 * come first, and every filled slot has weight NaN.  bias takes no part in the weights.
 * A logit of -inf costs nothing.  A bias that is not finite, or finite keys (large negative
 * logits as a mask, without a bias; a large negative bias) far below all others, have every
 * token's choice made in 64 bits, in about thirty times the time: close experts by their logits.
 * logits: [T,E] of bf16, fp16 or fp32, rows ld_logits elements apart; bias fp32 [E];
 * topk_idx int32 [T,R]; topk_w fp32 [T,R].  R <= 32, E <= 1024, R at most the experts of
 * top_groups groups; group_keys 2 needs groups of two.  No workspace.
 */
moe_status_t moe_route_scores(const void* logits, long long ld_logits, int dtype,
                              const float* bias, int T, int E, int R, const moe_router_t* router,
                              int32_t* topk_idx, float* topk_w, moe_stream_t stream);

/*
 * moe_route_scores_bwd -- dlogits = dL/dlogits given dw = dL/dtopk_w (fp32 [T,R]) and the
 * experts that the forward chose (constants).  Every logit is written: those of experts
 * that the weights do not depend on get 0.  Slots with idx outside [0, E) and closed
 * experts contribute nothing (their dw is not read for an empty slot); an expert named
 * twice gets the sum.  For renormalised weights only the chosen experts' logits are read: one
 * of NaN elsewhere shows in the weights, not here.  dlogits: [T,E] of the logits' type, rows ld_dlogits apart.
 */
moe_status_t moe_route_scores_bwd(const void* logits, long long ld_logits, int dtype,
                                  const int32_t* topk_idx, const float* dw, int T, int E, int R,
                                  const moe_router_t* router, void* dlogits,
                                  long long ld_dlogits, moe_stream_t stream);

/*
 * moe_quantize_fp8 -- E4M3 codes and fp32 scales of a matrix x [N,K]:
 *   scale = largest |x| of a block / 448,  code = E4M3(x / scale)  (the fp32 quotient to
 *   nearest even, saturating, a zero with x's sign; under a scale of 0 such a zero)
 *   row_codes uint8 [N,K],  row_scales fp32 [N, ceil(K/128)]: 128 elements of a row
 *   col_codes uint8 [N,K],  col_scales fp32 [ceil(N/128), K]: 128 elements of a column
 * Either pair may be NULL; both are written in one pass over x.  The last block of a row
 * or column may be shorter.  For finite x the row form is that of moe_dispatch_fp8 (which makes
 * +0 of the zeros of a block of zeros).  A NaN gets a code of NaN, of either sign, and does not
 * enter its block's scale; an infinity makes the scale infinite.
 * x: bf16, fp16 or fp32, rows ldx elements apart; K a multiple of 16; codes 16-byte
 * aligned.  No workspace.
 */
moe_status_t moe_quantize_fp8(const void* x, long long ldx, int dtype, int N, int K,
                              uint8_t* row_codes, float* row_scales, uint8_t* col_codes,
                              float* col_scales, moe_stream_t stream);

/*
 * moe_quantize_fp8_tiles -- the same of a stack w [E,n,K] (dense) with one scale per tile
 * of 128 x 128: codes uint8 [E,n,K], scales fp32 [E, ceil(n/128), ceil(K/128)].
 */
moe_status_t moe_quantize_fp8_tiles(const void* w, int dtype, int E, int n, int K, uint8_t* codes,
                                    float* scales, moe_stream_t stream);

/*
 * moe_product_fp8 -- each expert's product on its rows, on the fp8 tensor cores:
 *   out[i] = x_i w[e]^T   for the rows i in [offsets[e], offsets[e+1])
 * with x and w the values of their codes and scales; the codes' products of a block of 128
 * are summed in fp32, those sums times the product of both scales, in fp32, one rounding at the
 * end.  (A product of two scales above the fp32 range is infinite and makes infinities and NaN;
 * one below the normal range keeps fewer bits.)
 * xq, xs: rows [N,K] in the row form; wq, wscale: [E,n,K] in tiles; out: [N,n] of bf16, fp16
 * or fp32, rows ld_out elements apart.  offsets: int32 [E+1] on the device, not falling, in
 * [0, N]; NULL with E == 1: all N rows (a plain matrix product).  Rows of xq outside every
 * segment have no effect, those of out are left as they are.  Offsets that are not valid are
 * reported (MOE_ERR_BAD_ROUTING with MOE_CHECK) and nothing is computed; with N = 0 they are not
 * read.  Without MOE_CHECK a wait inside the kernel that gives up (MOE_ERR_TIMEOUT) is not
 * reported either, and the output is then incomplete.
 * n and K are multiples of 16, N <= 2^30, E <= 1024; codes 16-byte aligned.  The workspace
 * (error word; sums of few tiles split over several CTAs) has one size for the three products
 * of one N, n, K, E; calls that may overlap need one each.  Bitwise reproducible.
 */
moe_status_t moe_product_fp8(const uint8_t* xq, const float* xs, const int32_t* offsets, int N,
                             int n, int K, int E, const uint8_t* wq, const float* wscale,
                             void* out, long long ld_out, int out_dtype, void* ws,
                             size_t* ws_bytes, unsigned flags, moe_stream_t stream);

/*
 * moe_product_fp8_dx -- its gradient with respect to the rows:
 *   dx[i] = dy_i w[e]
 * dyq, dys: dL/dout [N,n] in the row form; dx: [N,K]; the rest as above.
 */
moe_status_t moe_product_fp8_dx(const uint8_t* dyq, const float* dys, const int32_t* offsets,
                                int N, int n, int K, int E, const uint8_t* wq,
                                const float* wscale, void* dx, long long ld_dx, int dx_dtype,
                                void* ws, size_t* ws_bytes, unsigned flags, moe_stream_t stream);

/*
 * moe_product_fp8_dw -- its gradient with respect to the weights:
 *   dw[e] = sum over the rows i of e of dy_i^T x_i     (zeros for an expert without rows)
 * dyq, dys: dL/dout [N,n], xq, xs: [N,K], both in the column form.  Blocks of 128 rows
 * belong to one expert: offsets are multiples of 128 (moe_sort with align 128), a segment
 * that ends at N may end anywhere.  dw: [E,n,K] of bf16, fp16 or fp32, dense, 16-byte
 * aligned; with MOE_ACCUMULATE the sum is added to it (fp32: a value below the normal range
 * counts as zero; 16-bit types: rounded once, in several times the time of overwriting it).
 * Offsets are checked with N = 0 too.  xs and dys 16-byte aligned.
 */
moe_status_t moe_product_fp8_dw(const uint8_t* dyq, const float* dys, const uint8_t* xq,
                                const float* xs, const int32_t* offsets, int N, int n, int K,
                                int E, void* dw, int dw_dtype, void* ws, size_t* ws_bytes,
                                unsigned flags, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H_ */
