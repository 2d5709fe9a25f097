/*
 * edit_attn.h -- C ABI of the B200 (sm_100a) EDiT linear compressed attention
 * library (libedit_attn.so).
 *
 * What it computes. The paper-notes page "EDiT: Efficient Diffusion
 * Transformers with Linear Compressed Attention" (ICCV 2025, arXiv
 * 2503.16726), section "Method in detail", defines one attention layer:
 *   - ConvFusion query, eq. (Q^EDiT):
 *       Q = ReLU(Linear_Q(X + Conv1x1(LeakyReLU(GN(Conv3x3(X))))))
 *     on the token sequence viewed as its H x W grid; the 3x3 conv compresses
 *     C -> c_red channels, the 1x1 conv restores c_red -> C.
 *   - Spatial Compressor, eq. (phi_SC): K = ReLU(DW(Linear_K(X))),
 *     V = DW(Linear_V(X)), DW a 3x3 depthwise conv of stride 2 (padding 1),
 *     leaving M = ceil(H/2) * ceil(W/2) key/value tokens.
 *   - Linear attention per head, eq. (y_i):
 *       y_i = (Q_i S) / (Q_i z + attn_eps),  S = sum_j K_j^T V_j,  z = sum_j K_j
 *     with heads = contiguous blocks of d = C/heads channels, no 1/sqrt(d)
 *     and no output projection.
 * Section "MM-EDiT", eq. (A^Hybrid), mixes it with softmax attention for
 * every interaction with prompt tokens, with eta = N_I / (N_I + N_T):
 *   out_img = eta * y + (1 - eta) * A(Q_I, K_P, V_P)
 *   out_txt = eta * A(Q_P, K_I, V_I) + (1 - eta) * A(Q_P, K_P, V_P)
 * where A(q,k,v) = softmax(q k^T / sqrt(d)) v per head, Q_I/K_I/V_I are the
 * EDiT query and compressed keys/values above, and Q_P/K_P/V_P are plain
 * Linear projections of the prompt tokens.
 *
 * Conventions for every entry point below.
 *   Layout:  x, out: [B, H*W, C], token n = h*W + w, channels innermost.
 *            x_txt, out_txt: [B, N_T, C].
 *   dtype:   x, out and every weight/bias share one dtype (EDIT_F32 or
 *            EDIT_BF16); all accumulation is fp32.
 *   Memory:  every pointer except the weights struct itself is DEVICE memory,
 *            owned by the caller, 16-byte aligned. The library never
 *            allocates, frees or synchronises (except edit_attn_read_status).
 *            Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *            default stream). Outputs must not alias inputs or the workspace.
 *            The library creates no streams or events either.
 *   Streams: a caller may lend a second stream (side_stream, a cudaStream_t
 *            of the same device, with EDIT_SIDE_EVENTS cudaEvent_t handles in
 *            side_events, all owned by the caller). bf16 calls then run part
 *            of their kernels there: the query's weight folding, and for
 *            layers of at most 32768 tokens (B*H*W) also the key/value branch
 *            and MM-EDiT's prompt-side attention. The side stream is forked
 *            from `stream` and joined back into it within the call, so
 *            everything still completes in `stream` order and the call can be
 *            captured in a CUDA graph. Calls that share a side stream or its
 *            events must be ordered on one `stream`. With side_stream NULL
 *            every kernel runs on `stream`, one after the other (identical
 *            results). Stage events (below) and the key-ConvFusion variant
 *            also keep every kernel on `stream`.
 *   Workspace: caller-allocated device buffer of at least the size returned by
 *            the matching *_workspace_bytes query, 256-byte aligned. Distinct
 *            concurrent calls need distinct workspaces.
 *   Errors:  the return value is 0 (EDIT_OK) or a negative EDIT_ERR_* code.
 *            Arguments are validated on the host before any launch; on a
 *            validation error nothing is enqueued. Device-side problems (a
 *            bounded wait that ran out) are recorded in the workspace status
 *            word and read back with edit_attn_read_status. Kernel faults
 *            surface at the caller's next synchronisation. Nothing traps.
 */
#ifndef EDIT_ATTN_H_
#define EDIT_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define EDIT_API __attribute__((visibility("default")))
#else
#define EDIT_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { EDIT_F32 = 0, EDIT_BF16 = 1 } edit_dtype;

/* Events that go with a caller-provided side stream (see Streams above). */
#define EDIT_SIDE_EVENTS 4

enum {
  EDIT_OK = 0,
  EDIT_ERR_NULL = -1,      /* a required pointer is NULL                          */
  EDIT_ERR_SHAPE = -2,     /* B, H, W < 1; C % heads; c_red % gn_groups; N_T < 0 ...*/
  EDIT_ERR_ALIGN = -3,     /* pointer not 16-byte aligned (workspace: 256-byte)    */
  EDIT_ERR_DTYPE = -4,     /* unsupported dtype                                    */
  EDIT_ERR_WORKSPACE = -5, /* workspace smaller than the query returned            */
  EDIT_ERR_CUDA = -6,      /* a CUDA runtime/driver call or launch failed          */
  EDIT_ERR_TIMEOUT = -7,   /* (device) a bounded wait ran out; results invalid     */
  EDIT_ERR_UNSUPPORTED = -8, /* shape outside what the kernels are built for       */
  EDIT_ERR_SCRATCH = -9     /* request needs more than the library's fixed scratch */
};

/* Weights and declared constants of one EDiT layer. Shapes (row-major):
 *   cf3_w [c_red][3][3][C]  3x3 conv C->c_red (torch [c_red,C,3,3] permuted to
 *                           channels-last: tap (kh,kw) reads pixel (h+kh-1, w+kw-1))
 *   cf3_b [c_red]           gn_gamma, gn_beta [c_red]
 *   cf1_w [C][c_red]        1x1 conv c_red->C; cf1_b [C]
 *   q_w, k_w, v_w [C][C]    Linear, torch [out][in] layout; q_b, k_b, v_b [C]
 *   kdw_w, vdw_w [C][3][3]  depthwise stride-2 conv taps; kdw_b, vdw_b [C]
 * Constants: gn_eps (GroupNorm, biased variance), leaky_slope, attn_eps (added
 * to the linear-attention denominator). None is defaulted by the library. */
typedef struct {
  int dtype; /* edit_dtype */
  int c_red;
  int gn_groups;
  float gn_eps;
  float leaky_slope;
  float attn_eps;
  const void *cf3_w, *cf3_b;
  const void *gn_gamma, *gn_beta;
  const void *cf1_w, *cf1_b;
  const void *q_w, *q_b;
  const void *k_w, *k_b;
  const void *v_w, *v_b;
  const void *kdw_w, *kdw_b;
  const void *vdw_w, *vdw_b;
  void *workspace; /* device, 256-byte aligned, >= edit_attn_workspace_bytes() */
  size_t workspace_bytes;
  void *side_stream;                   /* optional cudaStream_t (see Streams), or NULL */
  void *side_events[EDIT_SIDE_EVENTS]; /* cudaEvent_t handles; required with side_stream */
} edit_attn_weights;

/* Bytes of workspace edit_attn_forward needs for this shape (0 on a shape or
 * dtype error). Host-only: no allocation and no launch; the plan reads the
 * current device's SM count (148 when no device is visible), so query with
 * the device current that will run the layer. */
EDIT_API size_t edit_attn_workspace_bytes(int B, int H, int W, int C, int heads, const edit_attn_weights *w);

/* One EDiT attention layer: out[B, H*W, C] from x[B, H*W, C] (equations
 * above). Enqueues all kernels on `stream` and returns without waiting. */
EDIT_API int edit_attn_forward(const void *x, int B, int H, int W, int C, int heads, const edit_attn_weights *w,
                      void *out, void *stream);

/* Ablation variants of the query / key / value processing and an optional
 * output Linear. The ablation table of the notes page (section 消融实验,
 * "Query/Key/Value processing") compares the EDiT layer (CF, SC, SC) with
 * (CF, CF, -), (-, SC, SC) and (CF, -, -), where CF is ConvFusion, SC the
 * Spatial Compressor and - no processing beyond the Linear. Readings of the
 * table used here (it names the processing, not the formulas):
 *   q_proc  EDIT_PROC_CF:   Q = ReLU(Linear_Q(X + Conv1x1(LeakyReLU(GN(Conv3x3(X))))))
 *           EDIT_PROC_NONE: Q = ReLU(Linear_Q(X))
 *   k_proc  EDIT_PROC_SC:   K = ReLU(DW_K(Linear_K(X)))              (M keys)
 *           EDIT_PROC_CF:   K = ReLU(Linear_K(X + Conv1x1_K(LeakyReLU(GN_K(Conv3x3_K(X))))))
 *                           with the key's own ConvFusion weights below (N keys)
 *           EDIT_PROC_NONE: K = ReLU(Linear_K(X))                    (N keys)
 *   v_proc  EDIT_PROC_SC:   V = DW_V(Linear_V(X)); EDIT_PROC_NONE: V = Linear_V(X)
 * Keys and values must have equal counts, so (k_proc, v_proc) is one of
 * (SC, SC), (CF, NONE), (NONE, NONE); any other combination returns
 * EDIT_ERR_UNSUPPORTED. The attention step is eq. (y_i) over the M or N
 * key/value tokens. With o_w non-NULL the layer ends with the attention
 * block's output Linear, out = y o_w^T + o_b (o_w [C][C] torch layout, o_b
 * [C]); the page's layer has none, so it is optional.
 * kcf3_w [c_red][3][3][C], kcf3_b, kgn_gamma, kgn_beta [c_red], kcf1_w
 * [C][c_red], kcf1_b [C] are read only when k_proc is EDIT_PROC_CF; they use
 * the c_red, gn_groups, gn_eps and leaky_slope of the edit_attn_weights.
 * Weights a variant does not read may be NULL in both structs (for example
 * all ConvFusion weights, c_red and gn_groups when neither q_proc nor k_proc
 * is EDIT_PROC_CF; the depthwise weights without the compressor). */
enum { EDIT_PROC_NONE = 0, EDIT_PROC_CF = 1, EDIT_PROC_SC = 2 };

typedef struct {
  int q_proc;
  int k_proc;
  int v_proc;
  const void *kcf3_w, *kcf3_b;
  const void *kgn_gamma, *kgn_beta;
  const void *kcf1_w, *kcf1_b;
  const void *o_w, *o_b;
} edit_attn_variant;

/* Workspace bytes of edit_attn_variant_forward (0 on a shape, dtype or
 * processing error, or a NULL variant). Host-only. */
EDIT_API size_t edit_attn_variant_workspace_bytes(int B, int H, int W, int C, int heads, const edit_attn_weights *w,
                                                  const edit_attn_variant *v);

/* One layer with the processing chosen in `v` (conventions as
 * edit_attn_forward; the workspace is w->workspace and must hold
 * edit_attn_variant_workspace_bytes). {CF, SC, SC} with o_w == NULL computes
 * exactly what edit_attn_forward computes. Stage events (the hook below) are
 * the EDiT layer's 0-8, plus 9 after the output Linear when there is one. */
EDIT_API int edit_attn_variant_forward(const void *x, int B, int H, int W, int C, int heads,
                                       const edit_attn_weights *w, const edit_attn_variant *v, void *out,
                                       void *stream);

/* Mixing weights of the MM-EDiT hybrid (eta_mode below).
 *   EDIT_ETA_RATIO  the page's approximation: eta_I = eta_P = N_I / (N_I + N_T)
 *                   (section "MM-EDiT", the sentence after eq. (A^Hybrid)).
 *   EDIT_ETA_EXACT  the normaliser that ratio stands in for (the page calls it
 *                   the exact computation but does not write it out; reading
 *                   used here): each query normalises once over all keys.
 *                   Image row i, head h: eta = (Q_i z + eps) /
 *                   (Q_i z + eps + sum_P exp(q.k/sqrt(d))), i.e. image keys
 *                   weighted by the linear kernel Q_i . K_j and prompt keys by
 *                   exp(q . k / sqrt(d)) under one denominator. Prompt row:
 *                   eta = Z_I / (Z_I + Z_P) with Z the sums of
 *                   exp(q . k / sqrt(d)) over the image / prompt keys, i.e.
 *                   one softmax over both key sets. */
enum { EDIT_ETA_RATIO = 0, EDIT_ETA_EXACT = 1 };

/* Weights of the MM-EDiT hybrid: the EDiT image-stream weights (`img`, its
 * dtype field is the dtype of everything) plus the prompt-token projections
 * tq_w, tk_w, tv_w [C][C] (torch Linear layout) and their biases [C]. The
 * workspace and side-stream fields of `img` are ignored; the ones here are
 * used. eta_mode: EDIT_ETA_RATIO (0, the page's choice) or EDIT_ETA_EXACT;
 * anything else returns EDIT_ERR_UNSUPPORTED. */
typedef struct {
  edit_attn_weights img;
  const void *tq_w, *tq_b;
  const void *tk_w, *tk_b;
  const void *tv_w, *tv_b;
  void *workspace;
  size_t workspace_bytes;
  void *side_stream;
  void *side_events[EDIT_SIDE_EVENTS];
  int eta_mode;
} mmedit_weights;

EDIT_API size_t mmedit_workspace_bytes(int B, int H, int W, int N_T, int C, int heads, const mmedit_weights *w);

/* MM-EDiT hybrid attention (section "MM-EDiT", eq. (A^Hybrid)):
 * out_img[B, H*W, C] and out_txt[B, N_T, C] from x_img[B, H*W, C] and
 * x_txt[B, N_T, C]. N_T may be 0 (then eta = 1 and out_img is the EDiT
 * layer; x_txt/out_txt may be NULL). */
EDIT_API int mmedit_hybrid_forward(const void *x_img, const void *x_txt, int B, int H, int W, int N_T, int C, int heads,
                          const mmedit_weights *w, void *out_img, void *out_txt, void *stream);

/* Copy the device status word of a workspace to *status (0 = no device-side
 * error since the last forward call on it) and synchronise `stream`. This is
 * the only call that waits. When a tensor-core kernel's bounded wait ran out
 * (EDIT_ERR_TIMEOUT), the seven int32 words after the status word (offset
 * layout.status + 4) name the first wait that gave up: site (2: MMA issuer
 * waiting for a free accumulator, 3: MMA issuer waiting for operands,
 * 4: conv MMA issuer waiting for its input patch,
 * 10 + w: producer warp w waiting for a free stage, 20 + 10 r + q: epilogue
 * warp q of pair rank r waiting for an accumulator), block, tile, k-block (or
 * tiles done), stage or accumulator, barrier parity, globaltimer low bits. */
EDIT_API int edit_attn_read_status(const void *workspace, void *stream, int *status);

/* Text for a status code (static storage). */
EDIT_API const char *edit_status_string(int status);

/* Byte offsets of the intermediates kept in an edit_attn_forward workspace,
 * for inspection after the call completes (-1 when absent). Each tensor is
 * stored in the call's dtype unless noted:
 *   U [B,H,W,c_red]; G = LeakyReLU(GN(U)) [B,H*W,c_red]; Q [B,H*W,C];
 *   KVp [B,H*W,2C] (Linear_K(X) | Linear_V(X) per token);
 *   K, V [B,M,C] token-major (fp32 calls and MM-EDiT calls only);
 *   KT [B][C][Mp], VTx [B][heads][NP][Mp] channel-major (bf16 only): token
 *     t = i*Wop + j of the compressed grid padded to Wop columns (padding
 *     tokens are 0); rows d.. of each VTx head block are not written (the
 *     KV-state kernel forms the [V | 1] operand's ones row itself);
 *   gn_stats fp32 [B][gn_groups][2] (mean, rstd);
 *   Sz fp32 [B][heads][d][d+1] (S_h with z_h as the last column).
 * Mp, Wop, NP give the padded sizes (Mp = M, Wop = ceil(W/2), NP = 0 for fp32). */
typedef struct {
  int64_t status, U, G, Q, KVp, K, V, gn_stats, Sz, KT, VTx, Mp, Wop, NP;
} edit_ws_layout;

EDIT_API int edit_attn_workspace_layout(int B, int H, int W, int C, int heads, const edit_attn_weights *w,
                               edit_ws_layout *layout);

/* The same for an edit_attn_variant_forward workspace (v NULL: the EDiT
 * layer). Without the compressor, KT and VTx hold all N tokens in one padded
 * row (Mp = Wop = N rounded up to a multiple of 8). */
EDIT_API int edit_attn_variant_workspace_layout(int B, int H, int W, int C, int heads, const edit_attn_weights *w,
                                                const edit_attn_variant *v, edit_ws_layout *layout);

/* The DiT block around the attention (a text-to-image transformer block of
 * the PixArt-Sigma kind with EDiT as its self-attention; the notes page says
 * EDiT replaces the attention of PixArt-Sigma's blocks, section 整体框架 /
 * overall framework, but does not spell the block out: the block used here is
 * that model family's, read as follows).
 *   m = sst + t6[b] = (shift_a, scale_a, gate_a, shift_f, scale_f, gate_f)
 *   x1 = x + gate_a * (EDiT(LN(x) (1 + scale_a) + shift_a) o_w^T + o_b)
 *   x2 = x1 + softmax-attention(x1 cq_w^T + cq_b, y ck_w^T + ck_b, y cv_w^T + cv_b) co_w^T + co_b
 *   out = x2 + gate_f * (GELU(LN(x2) (1 + scale_f) + shift_f) fc1_w^T + fc1_b) fc2_w^T + fc2_b)
 * LN: LayerNorm over C without affine weights (eps ln_eps); GELU: the tanh
 * form; the cross-attention is per head with scale 1/sqrt(d), over the N_T
 * caption tokens y. Shapes (row-major, dtype of attn.dtype):
 *   x, out [B, H*W, C]; y [B, N_T, C] (N_T >= 1); t6 [B, 6, C] (the sample's
 *   timestep modulation); sst [6][C]; o_w, cq_w, ck_w, cv_w, co_w [C][C] and
 *   their biases [C]; fc1_w [hidden][C], fc1_b [hidden], fc2_w [C][hidden],
 *   fc2_b [C].
 * The EDiT attention weights and constants are those of `attn` (its workspace
 * and side-stream fields are ignored; the ones here are used). bf16 needs
 * hidden % 128 == 0 and head widths d of 32, 64 or 72 (the softmax kernel's);
 * other shapes return EDIT_ERR_UNSUPPORTED. */
typedef struct {
  edit_attn_weights attn;
  const void *o_w, *o_b;
  const void *sst;
  const void *cq_w, *cq_b, *ck_w, *ck_b, *cv_w, *cv_b, *co_w, *co_b;
  const void *fc1_w, *fc1_b, *fc2_w, *fc2_b;
  int hidden;
  float ln_eps;
  void *workspace;
  size_t workspace_bytes;
  void *side_stream;
  void *side_events[EDIT_SIDE_EVENTS];
} edit_dit_block_weights;

EDIT_API size_t edit_dit_block_workspace_bytes(int B, int H, int W, int N_T, int C, int heads,
                                               const edit_dit_block_weights *w);
EDIT_API int edit_dit_block_forward(const void *x, const void *y, const void *t6, int B, int H, int W, int N_T, int C,
                                    int heads, const edit_dit_block_weights *w, void *out, void *stream);

/* Row bands: one image split over several ranks (sequence parallelism).
 *
 * The notes page scales EDiT to 8192 x 8192 images (section 延迟分析, the
 * latency table); one such layer is 262,144 tokens. Its only global steps are
 * two reductions: the GroupNorm statistics of U = Conv3x3(X) (eq. (Q^EDiT))
 * and the per-head sums S = sum_j K_j^T V_j, z = sum_j K_j of eq. (y_i).
 * Everything else reads at most a 3 x 3 neighbourhood of a pixel. So the rows
 * of one image can be split into bands, one per rank:
 *   1. each rank takes its band of x plus one halo row above and one below
 *      from its neighbours (none at the image borders) and calls
 *      edit_attn_band_partials, which writes the band's record of partial
 *      sums;
 *   2. the ranks all-gather the records, in band order;
 *   3. each rank calls edit_attn_band_finish with all records, which sums them
 *      in band order (so every rank forms the same totals) and writes the
 *      band's rows of out.
 * Shapes and rules:
 *   band   rows [row0, row0 + rows) of an image of H rows: row0 even, and
 *          row0 + rows even unless it equals H, so that no stride-2 key/value
 *          token straddles two bands.
 *   x_ext  [rows + top + bottom][W][C]: the band with its halo rows, top = 1
 *          when row0 > 0, bottom = 1 when row0 + rows < H (else 0).
 *   record device buffer of edit_attn_band_record_bytes, 256-byte aligned:
 *          fp64 GroupNorm sums [gn_groups][2] (sum, sum of squares of the
 *          band's U), then, at the next 256-byte boundary, the band's fp32
 *          [S | z] [heads][d][d + 1].
 *   records the records of all nrecords bands, in band order, each
 *          edit_attn_band_record_bytes apart (256-byte aligned).
 *   out    [rows][W][C]: the band's rows of the layer output.
 * bf16 only (EDIT_ERR_UNSUPPORTED for fp32), one image. The workspace
 * (w->workspace, at least edit_attn_band_workspace_bytes) carries the band's
 * intermediates from the first call to the second: pass the same band, x_ext
 * and workspace to both, on the same stream. Errors as for edit_attn_forward;
 * a band that breaks the rules above is EDIT_ERR_SHAPE. */
typedef struct {
  int H;    /* rows of the whole image */
  int row0; /* first row of this band */
  int rows; /* rows of this band */
} edit_band;

EDIT_API size_t edit_attn_band_workspace_bytes(int W, int C, int heads, const edit_band *band,
                                               const edit_attn_weights *w);
EDIT_API size_t edit_attn_band_record_bytes(int C, int heads, const edit_attn_weights *w);
EDIT_API int edit_attn_band_partials(const void *x_ext, int W, int C, int heads, const edit_band *band,
                                     const edit_attn_weights *w, void *record, void *stream);
EDIT_API int edit_attn_band_finish(const void *x_ext, int W, int C, int heads, const edit_band *band,
                                   const edit_attn_weights *w, const void *records, int nrecords, void *out,
                                   void *stream);

/* Measurement hooks (no counterpart on the page; used by the benchmark).
 *
 * edit_attn_set_stage_events: when `events` is non-NULL, the next forward
 * calls made by this host thread record events[i] (cudaEvent_t handles
 * created by the caller) on the call's stream at stage boundary i:
 *   0 start, 1 K|V Linear GEMM, 2 depthwise conv, 3 KV state,
 *   4 weight folding, 5 3x3 conv GEMM (the conv kernel alone), 6 GroupNorm
 *   (statistics, finalize, apply; plus the conv's last-wave fixup when
 *   used), 7 query GEMM, 8 apply GEMM; MM-EDiT adds 9 prompt projections,
 *   10 image-row softmax attention, 11 prompt-row softmax attention.
 * Recording events between kernels serialises the programmatic overlap of
 * consecutive kernels at those points, so timed steps are fastest without
 * the hook.
 * `n` is the number of handles (events beyond n are not recorded). NULL
 * clears the hook. Returns EDIT_OK or EDIT_ERR_SHAPE for n < 0.
 *
 * edit_attn_kernel_launches: number of kernels this host thread's forward
 * calls have enqueued since the library was loaded. */
enum { EDIT_STAGE_EVENTS_EDIT = 9, EDIT_STAGE_EVENTS_MM = 12 };

EDIT_API int edit_attn_set_stage_events(void *const *events, int n);

EDIT_API uint64_t edit_attn_kernel_launches(void);

/* Wait drill for the device-side failure path (no counterpart on the page).
 *
 * Every device-side wait in the library is bounded and reports
 * EDIT_ERR_TIMEOUT through the workspace status word instead of hanging. This
 * hook lets a test make one such wait run out on purpose, without a fault.
 * bf16 layers at least 128 pixels wide normalise through a cooperative
 * GroupNorm kernel (statistics, grid barrier, apply in one grid); narrower ones
 * take the statistics from column sums their conv writes (in its epilogue, or
 * in the fixup of tiles split over k).
 * While the drill is armed (gn_extra_arrivals > 0), the calling thread's bf16
 * forward calls always run the cooperative kernel, which waits at its barrier for
 * gn_extra_arrivals more blocks than it launched, and gives up after
 * limit_ns nanoseconds (1e3 .. 2e9). Each block then records EDIT_ERR_TIMEOUT
 * and the first one the wait site (word 1 = 30, word 3 = arrivals seen,
 * word 4 = arrivals expected, word 5 = blocks launched) and returns without
 * applying the normalisation; later kernels of the call still run, and their
 * results are invalid. The GPU context stays usable. The cooperative kernel
 * runs for bf16 layers with at least 8 channels per group and c_red <= 4096.
 * (0, 0) disarms it. Returns EDIT_ERR_SHAPE for arguments out of range. */
EDIT_API int edit_attn_set_wait_drill(int gn_extra_arrivals, uint64_t limit_ns);

/* Linear attention step without any caller-provided scratch (the paper has
 * no counterpart; this is a deployment convenience).
 *
 * Some callers cannot allocate device memory at the point where they run the
 * layer: code running inside a framework's memory pool that forbids ad-hoc
 * cudaMalloc, plugins handed only their input and output buffers, or hosts
 * that must not grow device memory after start-up. For them this entry point
 * computes y from q, k, v exactly like the last step of edit_attn_forward
 * (per head: S = sum_j k_j^T v_j, z = sum_j k_j, y_i = q_i S / (q_i z + eps))
 * using a scratch array compiled into the library instead of a workspace.
 *
 *   q, out [B, N, C]; k, v [B, M, C] (device, dtype `dtype`, 16-byte aligned);
 *   heads divide C; the call is asynchronous on `stream`.
 *
 * The scratch is a static device array of EDIT_NOALLOC_SCRATCH_BYTES bytes
 * that every GPU which loads the library keeps until the process exits. Each
 * [S | z] block is B * heads * d * (d + 1) * 4 bytes (d = C / heads); a call
 * uses chunks + 1 such blocks (partial sums of each chunk of keys, then the
 * combined one), at least 3, and they must fit in the scratch: larger
 * requests return EDIT_ERR_SCRATCH without launching anything. d above 128,
 * or B or heads above 65535, return EDIT_ERR_UNSUPPORTED. The
 * library never calls cudaMalloc, cudaFree or any allocating routine here.
 * The first call on a device looks up the array's device address (with that
 * device current) and caches it; make that first call before any stream
 * capture. All calls share the one array and it keeps the last call's
 * contents (every value a call reads is written earlier in the same call), so
 * calls whose kernels may overlap on the GPU (different streams without
 * ordering) race on it: order them on one stream. */
#define EDIT_NOALLOC_SCRATCH_BYTES (4u << 20)

EDIT_API int edit_linear_attention_noalloc(const void *q, const void *k, const void *v, int B, int N, int M, int C,
                                           int heads, int dtype, float attn_eps, void *out, void *stream);

/* Operators on packed sequences: softmax attention, the gated delta rule and
 * the norms between them (the notes page has no counterpart: its layers take
 * rectangular batches with one prompt length; these are the mixers and norms
 * that text encoders and decoders next to such a layer run on prompts of
 * different lengths).
 *
 * Conventions, on top of those above.
 *   Rows:     a tensor is [rows][heads][d] (or [rows][C]) with `ld*` elements
 *             from one row to the next, so that slices of a wider projection
 *             can be passed as they are; heads and channels are contiguous.
 *             Sequence s has the rows offsets[s] .. offsets[s + 1] - 1. Rows of
 *             an output that belong to no sequence are left as they were.
 *   Offsets:  int32 DEVICE arrays, non-decreasing, inside the rows given. They
 *             are not read on the host, so a captured call can be replayed with
 *             other lengths. The kernels clamp whatever they read there to the
 *             rows given, so that bad values cannot make them read or write
 *             outside; attention and the delta rule then record EDIT_ERR_SHAPE
 *             in the workspace's status word (edit_attn_read_status), and the
 *             results of the call are not to be used. Every call sets the word.
 *   Head groups: heads is a multiple of kv_heads (or qk_heads); head h reads
 *             the shared head h / (heads / kv_heads).
 *   Row counts of attention and the delta rule are at most 2^31 - 512 (else
 *   EDIT_ERR_UNSUPPORTED); elements are addressed with 64 bits.
 *   Outputs must not overlap the inputs unless a function says so. Tensors of
 *   no rows may be NULL. All memory belongs to the current device, whose SM
 *   count the plans read (query the workspace with that device current). */

/* Softmax attention over packed sequences. For row i (0-based) of a sequence
 * with a query rows and b keys, and per head:
 *   out_i = sum_j p_ij v_j,  p_i = softmax over the visible j of scale (q_i . k_j),
 *   visible: j < b, and with `causal` also j <= i + b - a (the last query row
 *   sees the last key, so that a sequence's newest rows can follow a cache of
 *   its earlier keys). A row that sees no key (b = 0, or b < a) gets zeros.
 * q, out [rows_q][heads][d]; k, v [rows_k][kv_heads][d]. Sequence s has the
 * keys k_offsets[s] .. k_offsets[s + 1] - 1, or, with k_lens, the first
 * k_lens[s] of them (a cache filled in part; what lies behind is not used,
 * whatever it holds). k_lens may be NULL. max_k bounds every sequence's key
 * count (it sizes the split of long key lists over several blocks, joined in a
 * fixed order; a longer sequence is cut there and recorded as
 * EDIT_ERR_SHAPE). Scores and sums are fp32; bf16 calls round the weights
 * p_ij to bf16 before the product with v. A NaN or an infinity in k or v
 * reaches the rows that see that key and no others.
 * d a multiple of 8 up to 128, ld* multiples of 8, heads / kv_heads at most 64,
 * scale positive and below 2^127; else EDIT_ERR_UNSUPPORTED. */
typedef struct {
  int dtype; /* edit_dtype of q, k, v, out */
  int heads, kv_heads, d;
  int nseq;
  int causal;
  int max_k;
  float scale; /* not defaulted by the library */
  int64_t rows_q, rows_k;
  int64_t ldq, ldk, ldv, ldo;
  const int32_t *q_offsets; /* [nseq + 1] */
  const int32_t *k_offsets; /* [nseq + 1] */
  const int32_t *k_lens;    /* [nseq] or NULL */
  void *workspace; /* device, 256-byte aligned */
  size_t workspace_bytes;
} edit_packed_attention;

/* Workspace bytes for calls of at most a->rows_q query rows (0 on an argument
 * error). Host-only; reads dtype, heads, kv_heads, d, nseq, max_k, rows_q. */
EDIT_API size_t edit_packed_attention_workspace_bytes(const edit_packed_attention *a);
EDIT_API int edit_packed_attention_forward(const void *q, const void *k, const void *v,
                                           const edit_packed_attention *a, void *out, void *stream);

/* The gated delta rule over packed sequences: causal linear attention whose
 * state decays and, before a token's value is added under its key, gives up
 * what it held there. Per head, with S [d_k][d_v] (fp32), for each token t:
 *   S  = exp(g_t) S
 *   u  = beta_t (v_t - S^T k_t)
 *   S  = S + k_t u^T
 *   o_t = scale S^T q_t
 * q, k [rows][qk_heads][d_k]; v, out [rows][heads][d_v]; g, beta fp32
 * [rows][heads] with ldg elements between rows (g is a log decay, at most 0;
 * it is limited below at -200, where exp is 0 in fp32, so that -infinity means
 * "forget all"). With qk_norm the operator first divides each q_t and k_t by
 * sqrt(|.|^2 + qk_eps). state_in, state_out fp32 [nseq][heads][d_k][d_v]:
 * state_in NULL starts from zeros, state_out NULL drops the final states; the
 * two may be the same buffer (not overlap in another way). A sequence of no rows
 * copies its state.
 * Sums and states are fp32. bf16 calls of edit_delta_rule_forward with 32 rows a
 * sequence or more on average run in chunks of 64 tokens: states are then within
 * some 2^-22 of the largest value of their columns (v's index) a chunk, and o_t,
 * besides its own rounding, within some 2^-11 of scale |q_t| times that value and
 * 2^-9 of each of the chunk's own terms. A token's results depend on no later token,
 * and a column's on no other column of v: a value that is not finite (from
 * 2^128 - 2^119 on in chunks) makes the results of its token and the later ones not
 * finite, as NaN in chunks, in v of that column and in k, g, beta of all.
 * d_k a multiple of 8 up to 128, d_v a multiple of 8 up to 256, ldq .. ldo
 * multiples of 8, nseq at most 65535; else EDIT_ERR_UNSUPPORTED.
 * edit_delta_rule_step is one token for each of nseq sequences (row s belongs
 * to sequence s; offsets and rows are not read, no workspace and so no status
 * word): `state` is updated in place. A (sequence, head) whose state did not
 * arrive on the chip within the time limit of every wait here gets NaN in out,
 * its state left as it was. */
typedef struct {
  int dtype; /* edit_dtype of q, k, v, out */
  int qk_heads, heads, d_k, d_v;
  int nseq;
  int qk_norm;
  float scale, qk_eps;
  int64_t rows;
  int64_t ldq, ldk, ldv, ldo, ldg, ldb; /* ldg: g, ldb: beta */
  const int32_t *offsets; /* [nseq + 1] */
  void *workspace; /* device, 256-byte aligned */
  size_t workspace_bytes;
} edit_delta_rule;

/* Workspace bytes for calls of at most a->rows rows (0 on an argument error).
 * Host-only. */
EDIT_API size_t edit_delta_rule_workspace_bytes(const edit_delta_rule *a);
EDIT_API int edit_delta_rule_forward(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                     const edit_delta_rule *a, const float *state_in, float *state_out, void *out,
                                     void *stream);
EDIT_API int edit_delta_rule_step(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                  const edit_delta_rule *a, float *state, void *out, void *stream);

/* The step between two branches of a block, in one pass: the norm after a
 * branch, its gate, the residual, and the norm before the next branch.
 *   r = x + res_scale * act(gate0 + gate[b]) * N_post(y)
 *   h = N_pre(r) * (1 + scale0 + scale[b]) + shift0 + shift[b]
 * for each row, b its sample. N_post, N_pre: EDIT_NORM_NONE (identity),
 * EDIT_NORM_LAYER ((z - mean) / sqrt(var + eps), biased variance) or
 * EDIT_NORM_RMS (z / sqrt(mean z^2 + eps)), then * w + b with the optional
 * weights post_w, post_b, pre_w, pre_b [C] (w 1 and b 0 where NULL; not
 * allowed with EDIT_NORM_NONE). act: EDIT_GATE_LINEAR or EDIT_GATE_TANH.
 * x, y, r, h [rows][C] with ldx .. ldh; y may be NULL (then r = x, and only h
 * is formed); r or h may be NULL (not both); r may be x or y and h may be y or
 * x (same pointer and row stride: each row is read before it is written), and
 * r and h are two buffers. gate, scale, shift: one vector of C for each sample,
 * ld_mod elements apart; gate0, scale0, shift0 [C] are common to all samples.
 * Each of the six may be NULL: missing scale and shift terms count as 0; the
 * gate is 1 when gate and gate0 are both NULL. Row r belongs to sample s with
 * offsets[s] <= r < offsets[s + 1] (rows in no sample are left as they were),
 * or, with offsets NULL, to sample r / rows_per_sample (rows then is at most
 * samples * rows_per_sample). Sums and norms are fp32 over the unrounded r.
 * Any C up to 16384 and any strides (16-byte vectors are used where pointers,
 * strides and C allow). */
enum { EDIT_NORM_NONE = 0, EDIT_NORM_LAYER = 1, EDIT_NORM_RMS = 2 };
enum { EDIT_GATE_LINEAR = 0, EDIT_GATE_TANH = 1 };

typedef struct {
  int dtype; /* edit_dtype of every tensor */
  int norm_post, norm_pre, gate_act;
  int C;
  int samples;
  float eps, res_scale; /* not defaulted by the library */
  int64_t rows, rows_per_sample;
  int64_t ldx, ldy, ldr, ldh, ld_mod;
  const int32_t *offsets; /* [samples + 1] or NULL */
  const void *post_w, *post_b, *pre_w, *pre_b;
  const void *gate0, *scale0, *shift0;
  const void *gate, *scale, *shift;
} edit_block_norm;

EDIT_API int edit_block_norm_forward(const void *x, const void *y, const edit_block_norm *a, void *r, void *h,
                                     void *stream);

/* The DiT block of edit_dit_block_forward with other norms, and norms after its
 * branches as well (a block with norms on both sides of each branch), its
 * residual steps run by the block norm above:
 *   x1 = x + gate_a * N_post(EDiT(N_pre(x) (1 + scale_a) + shift_a) o_w^T + o_b)
 *   x2 = x1 + N_post(softmax-attention(..) co_w^T + co_b)
 *   out = x2 + gate_f * N_post(GELU(N_pre(x2) (1 + scale_f) + shift_f) ..)
 * norm_pre, norm_post: EDIT_NORM_* (eps: the block's ln_eps), each followed by
 * its optional weight [C] (NULL: 1; a post weight needs a post norm).
 * EDIT_NORM_LAYER before and EDIT_NORM_NONE after, without weights, is the
 * block of edit_dit_block_forward. The rest, workspace included, as there. */
typedef struct {
  int norm_pre, norm_post;
  const void *pre_attn_w, *pre_ffn_w;
  const void *post_attn_w, *post_cross_w, *post_ffn_w;
} edit_dit_block_norms;

EDIT_API int edit_dit_block_normed_forward(const void *x, const void *y, const void *t6, int B, int H, int W, int N_T,
                                           int C, int heads, const edit_dit_block_weights *w,
                                           const edit_dit_block_norms *norms, void *out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* EDIT_ATTN_H_ */
