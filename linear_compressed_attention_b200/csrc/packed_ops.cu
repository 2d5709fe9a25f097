// C ABI of the packed-sequence operators (include/edit_attn.h): argument
// checks, launch rules and workspace plans of the packed softmax attention, the
// gated delta rule and the block norm.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>
#include <utility>

#include "block_norm.cuh"
#include "common.cuh"
#include "delta_chunk.cuh"
#include "delta_rule.cuh"
#include "host.h"
#include "packed_attn.cuh"
#include "packed_attn_tc.cuh"

using namespace edit;

namespace {

#define EDIT_TRY(expr)              \
  do {                              \
    const int rc_ = (expr);         \
    if (rc_ != EDIT_OK) return rc_; \
  } while (0)

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align256(size_t v) { return (v + 255) / 256 * 256; }
long ceil_div(long a, long b) { return (a + b - 1) / b; }

// One kernel on `st`, with programmatic stream serialization as every kernel of
// the library; counted for edit_attn_kernel_launches. A launch fails when static
// and dynamic shared memory together pass 48 KB and the dynamic limit has not been
// raised: it is from 32 KB on (no kernel here has 16 KB of static memory).
template <typename... KArgs, typename... Args>
int launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args&&... args) {
  if (smem > 32 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
    return EDIT_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...) == cudaSuccess ? EDIT_OK : EDIT_ERR_CUDA;
}

// Leading dimension of rows of `width` values: wide enough, rows 16-byte
// aligned for the vector accesses (8 elements cover both dtypes).
int check_ld(int64_t ld, int64_t width) {
  if (ld < width) return EDIT_ERR_SHAPE;
  return ld % 8 == 0 ? EDIT_OK : EDIT_ERR_UNSUPPORTED;
}

// Most rows of a call: row indexes of attention and the delta rule are 32-bit, and
// their loops step up to a tile (256 rows) past a sequence's end.
constexpr int64_t kMaxRows = INT32_MAX - 511;

// ------------------------------------------------------------ packed attention
constexpr size_t kStatusBytes = 256;

struct AttnPlan {
  int slots, nsplit;
  size_t part_o, part_ml, total;
};

// bf16 calls whose sequences have at most 128 packed rows on average take one
// row tile a block and two blocks an SM, others two row tiles a block, which halves
// the keys read (8 sequences over 2048 keys, 16 heads of 128, us with one / two: 32
// rows 46 / 51, 128 rows 68 / 82, 256 rows 112 / 114; 4 x 4096 rows over 333 keys, 16
// heads of 72: 90 / 79).
int attn_row_tiles(const edit_packed_attention* a, int64_t rows) {
  return rows * (a->heads / a->kv_heads) <= 128 * static_cast<int64_t>(a->nseq) ? 1 : 2;
}
int attn_rows(const edit_packed_attention* a, int64_t rows) {
  const int G = a->heads / a->kv_heads;
  return a->dtype == EDIT_BF16 ? attn_row_tiles(a, rows) * (128 / G) : 64 / G;
}

int attn_args(const edit_packed_attention* a, bool query) {  // query: what the workspace depends on
  if (!a) return EDIT_ERR_NULL;
  if (a->dtype != EDIT_F32 && a->dtype != EDIT_BF16) return EDIT_ERR_DTYPE;
  if (a->heads < 1 || a->kv_heads < 1 || a->heads % a->kv_heads != 0 || a->d < 1 || a->nseq < 1 || a->max_k < 0 ||
      a->rows_q < 0 || (!query && a->rows_k < 0))
    return EDIT_ERR_SHAPE;
  if (a->d % 8 != 0 || a->d > 128 || a->heads / a->kv_heads > 64 || a->kv_heads > 65535) return EDIT_ERR_UNSUPPORTED;
  if (a->rows_q > kMaxRows || (!query && a->rows_k > kMaxRows)) return EDIT_ERR_UNSUPPORTED;
  if (a->rows_q + a->nseq > INT32_MAX) return EDIT_ERR_UNSUPPORTED;
  return EDIT_OK;
}

// Parts of the key lists when there are `slots` row tiles for each key/value
// head: about 12 items an SM, at least 256 keys a part, so that blocks end
// together whatever the lengths (one token of 32 sequences over caches of up to
// 8192 keys, 8 heads: 143 us with 1 part, 125 with 4, 120 with 6, 127 with 9, 143
// with 18, where the parts' own start and the join weigh more).
int attn_nsplit(long slots, const edit_packed_attention* a, int sms) {
  const long want = 12L * sms / (slots * a->kv_heads), most = ceil_div(a->max_k, 256);
  const long n = want < most ? want : most;
  return static_cast<int>(n < 1 ? 1 : n);
}

// The plan of `rows` query rows in tiles of R.
void attn_plan(const edit_packed_attention* a, int64_t rows, int R, AttnPlan& pl) {
  pl.slots = static_cast<int>(rows / R + a->nseq);
  pl.nsplit = rows > 0 ? attn_nsplit(pl.slots, a, device_sms()) : 1;
  const size_t items = static_cast<size_t>(pl.nsplit) * rows * a->heads;
  pl.part_o = kStatusBytes;
  pl.part_ml = pl.part_o + (pl.nsplit > 1 ? align256(items * a->d * 4) : 0);
  pl.total = pl.part_ml + (pl.nsplit > 1 ? align256(items * 8) : 0);
}

template <typename T, int DP>
int attn_simt(const PackedAttnParams& p, cudaStream_t st) {
  const size_t smem = (2 * 64 * (DP + 4) + 64 * DP + 64 * 68) * sizeof(float);
  return launch(packed_attn_simt_kernel<T, DP>, dim3(p.slots, p.kv_heads, p.nsplit), dim3(256), smem, st, p);
}

template <int DP, int NQ>
int attn_tc(const PackedAttnParams& p, cudaStream_t st) {
  using Cfg = AttnTcCfg<DP, NQ>;
  const int G = p.heads / p.kv_heads;
  const cuuint64_t d = p.d, gl = G, kl = p.kv_heads;
  CUtensorMap mq, mk, mv;
  {
    const cuuint64_t dims[4] = {d, gl, kl, static_cast<cuuint64_t>(p.rows_q)};
    const cuuint64_t strides[3] = {d * 2, gl * d * 2, static_cast<cuuint64_t>(p.ldq) * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(G), 1, static_cast<cuuint32_t>(128 / G)};
    if (!bf16_tensor_map(&mq, 4, p.q, dims, strides, box)) return EDIT_ERR_CUDA;
  }
  const cuuint32_t box[3] = {64, 1, 128};
  const cuuint64_t dims[3] = {d, kl, static_cast<cuuint64_t>(p.rows_k)};
  const cuuint64_t sk[2] = {d * 2, static_cast<cuuint64_t>(p.ldk) * 2}, sv[2] = {d * 2, static_cast<cuuint64_t>(p.ldv) * 2};
  if (!bf16_tensor_map(&mk, 3, p.k, dims, sk, box) || !bf16_tensor_map(&mv, 3, p.v, dims, sv, box))
    return EDIT_ERR_CUDA;
  const long items = static_cast<long>(p.slots) * p.kv_heads * p.nsplit, most = (NQ == 1 ? 2L : 1L) * device_sms();
  if (items > INT32_MAX - 64 * most) return EDIT_ERR_UNSUPPORTED;  // (a block's steps stay in 32 bits)
  return launch(packed_attn_tc_kernel<DP, NQ>, dim3(static_cast<unsigned>(items < most ? items : most)),
                dim3(Cfg::THREADS), Cfg::SMEM, st, mq, mk, mv, p, static_cast<int>(items));
}

template <int NQ>
int attn_tc_width(const PackedAttnParams& p, cudaStream_t st) {
  if (p.d <= 64) return attn_tc<64, NQ>(p, st);
  if (p.d <= 80) return attn_tc<80, NQ>(p, st);
  return attn_tc<128, NQ>(p, st);
}

template <typename T>
int attn_run(PackedAttnParams p, int row_tiles, cudaStream_t st) {
  if constexpr (sizeof(T) == 2) {
    if (p.rows_q == 0 || p.rows_k == 0) {  // no tensor to describe: the offsets are checked, rows get zeros
      p.slots = p.rows_q / (64 / (p.heads / p.kv_heads)) + p.nseq;
      p.nsplit = 1;
      EDIT_TRY((attn_simt<T, 128>(p, st)));
    } else {
      EDIT_TRY(row_tiles == 1 ? attn_tc_width<1>(p, st) : attn_tc_width<2>(p, st));
    }
  } else {
    EDIT_TRY(p.d <= 64 ? (attn_simt<T, 64>(p, st)) : (attn_simt<T, 128>(p, st)));
  }
  if (p.nsplit == 1) return EDIT_OK;
  return launch(packed_attn_join_kernel<T>, dim3(static_cast<unsigned>(ceil_div(static_cast<long>(p.rows_q) * p.heads, 4))),
                dim3(128), 0, st, p);
}

// ------------------------------------------------------------ delta rule
constexpr int kDeltaMaxSeg = 16;  // most parts of a sequence (delta_nseg)

int delta_args(const edit_delta_rule* a, bool step) {
  if (!a) return EDIT_ERR_NULL;
  if (a->dtype != EDIT_F32 && a->dtype != EDIT_BF16) return EDIT_ERR_DTYPE;
  if (a->qk_heads < 1 || a->heads < 1 || a->heads % a->qk_heads != 0 || a->d_k < 1 || a->d_v < 1 || a->nseq < 1 ||
      (!step && a->rows < 0))
    return EDIT_ERR_SHAPE;
  if (a->d_k % 8 != 0 || a->d_k > 128 || a->d_v % 8 != 0 || a->d_v > 256 || a->heads > 65535)
    return EDIT_ERR_UNSUPPORTED;
  if (!step && a->rows > kMaxRows) return EDIT_ERR_UNSUPPORTED;
  if (static_cast<long>(a->nseq) * 8 * kDeltaMaxSeg > INT32_MAX || (!step && a->nseq > 65535)) return EDIT_ERR_UNSUPPORTED;
  return EDIT_OK;
}

int delta_call(const void* q, const void* k, const void* v, const float* g, const float* beta,
               const edit_delta_rule* a, int64_t rows, const void* out) {
  if (rows > 0 && (!q || !k || !v || !g || !beta || !out)) return EDIT_ERR_NULL;
  EDIT_TRY(check_ld(a->ldq, static_cast<int64_t>(a->qk_heads) * a->d_k));
  EDIT_TRY(check_ld(a->ldk, static_cast<int64_t>(a->qk_heads) * a->d_k));
  EDIT_TRY(check_ld(a->ldv, static_cast<int64_t>(a->heads) * a->d_v));
  EDIT_TRY(check_ld(a->ldo, static_cast<int64_t>(a->heads) * a->d_v));
  if (a->ldg < a->heads || a->ldb < a->heads) return EDIT_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(g, 4) ||
      !aligned(beta, 4))
    return EDIT_ERR_ALIGN;
  return EDIT_OK;
}

DeltaParams delta_params(const void* q, const void* k, const void* v, const float* g, const float* beta,
                         const edit_delta_rule* a, void* out) {
  DeltaParams p = {};
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = g;
  p.beta = beta;
  p.out = out;
  p.rows = a->rows;
  p.ldq = a->ldq;
  p.ldk = a->ldk;
  p.ldv = a->ldv;
  p.ldo = a->ldo;
  p.ldg = a->ldg;
  p.ldb = a->ldb;
  p.qk_heads = a->qk_heads;
  p.heads = a->heads;
  p.d_k = a->d_k;
  p.d_v = a->d_v;
  p.nseq = a->nseq;
  p.qk_norm = a->qk_norm;
  p.scale = a->scale;
  p.qk_eps = a->qk_eps;
  return p;
}

template <typename T, bool STEP>
int delta_recurrent(const DeltaParams& p, cudaStream_t st) {
  const int cb = static_cast<int>(ceil_div(p.d_v, 16 * kDeltaCpt<STEP>));
  const dim3 grid(static_cast<unsigned>(p.nseq) * cb, p.heads), block(128);
  if (p.d_k <= 32) return launch(delta_recurrent_kernel<T, 32, STEP>, grid, block, 0, st, p, cb);
  if (p.d_k <= 64) return launch(delta_recurrent_kernel<T, 64, STEP>, grid, block, 0, st, p, cb);
  if (p.d_k <= 96) return launch(delta_recurrent_kernel<T, 96, STEP>, grid, block, 0, st, p, cb);
  return launch(delta_recurrent_kernel<T, 128, STEP>, grid, block, 0, st, p, cb);
}

// Single tokens: whole states through shared memory where most SMs get one, else
// smaller blocks (16 heads of 128 x 128, us: 4 sequences 5.5 against 4.5, 8: 5.7 /
// 6.8, 16: 7.6 / 11.3, 32: 13.3 / 20.2; with d_v = 64 the two are the same, 7.3 /
// 6.9 for 32 sequences).
template <typename T>
int delta_single(const DeltaParams& p, cudaStream_t st) {
  const long blocks = static_cast<long>(p.nseq) * p.heads;
  if (p.d_v == kDeltaStepDv && 4 * blocks >= 3L * device_sms())
    return launch(delta_step_kernel<T>, dim3(static_cast<unsigned>(p.nseq), p.heads), dim3(256),
                  static_cast<size_t>(p.d_k) * kDeltaStepDv * 4, st, p);
  return delta_recurrent<T, true>(p, st);
}

// bf16 calls with sequences of at least this many rows on average run in chunks
// of 64 tokens, others token by token (16 heads of 128, us for 64 sequences of 16 /
// 32 / 64 tokens: 117 / 121 / 129 in chunks, 88 / 156 / 291 token by token; one
// sequence: 22 / 22 / 23 and 12 / 16 / 28).
constexpr int kDeltaChunkedRows = 32;

struct DeltaPlan {
  bool chunked;
  int DK, slots, nseg;
  size_t blobs, kq, trans, starts, total;
};

// Parts each sequence's chunks are cut into: with few (sequence, head) pairs the
// walk over the chunks leaves SMs idle. A part's effect is found first (pass 1,
// on d_v + d_k columns), the effects are joined part after part, then the parts
// run side by side (pass 2). The number with the least time, in chunks of pass 2
// (a chunk of pass 1 counts 0.87, a join 1.5; 8192 tokens of 16 heads of 128: 927 us
// in one part, 463 in 4, 397 in 5, 358 in 9, 418 in 16; 4096 tokens of 4 heads: 446,
// 223, 193, 145, 130, where it takes 8 parts, 146; 1500 and 1100 tokens of 20 heads of
// 128: 199 in one, 198 in 3, 217 in 4). It knows the mean length only.
int delta_nseg(const edit_delta_rule* a, int64_t chunks, int sms) {
  const int64_t heads = static_cast<int64_t>(a->nseq) * a->heads;
  const int64_t b1 = heads * ceil_div(a->d_v + a->d_k, kDeltaCols), b2 = heads * ceil_div(a->d_v, kDeltaCols);
  chunks = chunks < 1024 ? chunks : 1024;  // (longer ones as these: the workspace query asks for each length up to it)
  int best = 1;
  double least = static_cast<double>(ceil_div(b2, sms)) * chunks;
  for (int n = 2; n <= kDeltaMaxSeg; ++n) {
    const double t = (0.87 * ceil_div(b1 * (n - 1), sms) + ceil_div(b2 * n, sms)) * ceil_div(chunks, n) + 1.5 * n;
    if (t < least) {
      least = t;
      best = n;
    }
  }
  return best;
}

void delta_plan(const edit_delta_rule* a, DeltaPlan& pl) {
  pl = DeltaPlan{};
  pl.total = kStatusBytes;
  pl.chunked = a->dtype == EDIT_BF16 && a->rows >= static_cast<int64_t>(kDeltaChunkedRows) * a->nseq;
  if (!pl.chunked) return;
  pl.DK = a->d_k <= 64 ? 64 : 128;
  pl.slots = static_cast<int>(a->rows / kDeltaL + a->nseq);
  pl.nseg = delta_nseg(a, ceil_div(a->rows, static_cast<int64_t>(kDeltaL) * a->nseq), device_sms());
  const size_t heads = static_cast<size_t>(a->nseq) * a->heads;
  auto take = [&](size_t bytes) {
    const size_t at = pl.total;
    pl.total += align256(bytes);
    return at;
  };
  pl.blobs = take(static_cast<size_t>(pl.slots) * a->heads * kDeltaBlob);
  pl.kq = take(static_cast<size_t>(pl.slots) * a->qk_heads * delta_kq_bytes(pl.DK));
  pl.trans = take(heads * (pl.nseg - 1) * a->d_k * (a->d_v + a->d_k) * 4);
  pl.starts = take(pl.nseg > 1 ? heads * pl.nseg * a->d_k * a->d_v * 4 : 0);
}

template <int DK>
int delta_chunked(const DeltaChunkParams& p, cudaStream_t st) {
  const DeltaParams& d = p.d;
  EDIT_TRY(launch(delta_prep_kernel<DK>, dim3(p.slots, d.heads), dim3(128), DeltaPrepCfg<DK>::SMEM, st, p));
  auto blocks = [&](int cols, int parts) {
    return dim3(static_cast<unsigned>(ceil_div(cols, kDeltaCols) * parts * d.nseq), d.heads);
  };
  auto warps = [](int cols) { return static_cast<int>(ceil_div(cols < kDeltaCols ? cols : kDeltaCols, 16)); };
  if (p.nseg > 1) {
    const int cols = d.d_v + d.d_k;
    EDIT_TRY(launch(delta_chunk_kernel<DK, false>, blocks(cols, p.nseg - 1), dim3(32 * warps(cols) + 32),
                    DeltaChunkCfg<DK>::smem(warps(cols)), st, p,
                    static_cast<int>(ceil_div(cols, kDeltaCols))));
    EDIT_TRY(launch(delta_join_kernel<DK>, dim3(static_cast<unsigned>(ceil_div(d.d_v, 16)), d.heads, d.nseq), dim3(2 * DK),
                    DeltaJoinCfg<DK>::SMEM, st, p));
  }
  return launch(delta_chunk_kernel<DK, true>, blocks(d.d_v, p.nseg), dim3(32 * warps(d.d_v) + 32),
                DeltaChunkCfg<DK>::smem(warps(d.d_v)), st, p,
                static_cast<int>(ceil_div(d.d_v, kDeltaCols)));
}

// ------------------------------------------------------------ block norm
template <typename T, int VEC, int TPR, int NV>
int norm_launch(const BlockNormParams& p, cudaStream_t st) {
  const long blocks = ceil_div(p.rows, 256 / TPR);
  if (blocks > INT32_MAX) return EDIT_ERR_UNSUPPORTED;
  return launch(block_norm_kernel<T, VEC, TPR, NV>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, p);
}

template <typename T, int VEC, int TPR, int NV>
int norm_rows(const BlockNormParams& p, cudaStream_t st) {
  // three blocks an SM where there are rows for them (each folds a sample's vectors once)
  const long most = 3L * device_sms(), per = ceil_div(p.rows, 256 / TPR) <= most ? 256 / TPR : ceil_div(p.rows, most);
  return launch(block_norm_rows_kernel<T, VEC, TPR, NV>, dim3(static_cast<unsigned>(ceil_div(p.rows, per))), dim3(256),
                static_cast<size_t>((p.C + 3) / 4) * 64, st, p, static_cast<int>(per));
}

// Threads a row: a warp where its registers hold the row (40 values a thread in
// bf16, 16 in fp32, which fills an SM with warps all the same), two for wider bf16
// rows (30000 rows of 1536: 67 us, with four 82; fp32 the other way, 133 / 124), four
// for the others and where rows are few. Rows without 16-byte vectors: 16 values a
// thread where there are rows enough (20000 rows of 1001 bf16 130 us, with 4 or 8
// values 172; fp32 63 / 106), which is bound by its 2- and 4-byte accesses.
template <typename T>
int norm_run(const BlockNormParams& p, bool vec, cudaStream_t st) {
  if (p.C > kBnNarrow) {
    if (!vec) return norm_launch<T, 1, 256, 64>(p, st);
    return p.C <= 4096 ? norm_launch<T, 8, 256, 2>(p, st) : norm_launch<T, 8, 256, 8>(p, st);
  }
  if (!vec) {
    if (p.rows <= 2L * device_sms()) return p.C <= 512 ? norm_rows<T, 1, 128, 4>(p, st) : norm_rows<T, 1, 256, 8>(p, st);
    if (p.C <= 256) return norm_rows<T, 1, 32, 8>(p, st);
    if (p.C <= 512) return norm_rows<T, 1, 32, 16>(p, st);
    if (p.C <= 1024) return norm_rows<T, 1, 64, 16>(p, st);
    return norm_rows<T, 1, 128, 16>(p, st);
  }
  const int nv = p.C / 8;
  if (p.rows > 2L * device_sms()) {
    if (nv <= 32) return norm_rows<T, 8, 32, 1>(p, st);
    if (nv <= 64) return norm_rows<T, 8, 32, 2>(p, st);
    if constexpr (sizeof(T) == 2) {
      if (nv <= 96) return norm_rows<T, 8, 32, 3>(p, st);
      if (nv <= 128) return norm_rows<T, 8, 32, 4>(p, st);
      if (nv <= 160) return norm_rows<T, 8, 32, 5>(p, st);
      return nv <= 192 ? norm_rows<T, 8, 64, 3>(p, st) : norm_rows<T, 8, 64, 4>(p, st);
    }
  }
  return nv <= 128 ? norm_rows<T, 8, 128, 1>(p, st) : norm_rows<T, 8, 128, 2>(p, st);
}

}  // namespace

extern "C" {

size_t edit_packed_attention_workspace_bytes(const edit_packed_attention* a) {
  if (attn_args(a, true) != EDIT_OK) return 0;
  // Fewer rows can mean more parts: the most over all row counts up to rows_q and
  // both tile heights. Rows with the same number of slots have the same parts, so
  // the last of each are enough, and more slots never have more parts (no rows at
  // all have one part whatever the slots: with one row a tile the scan meets them
  // first, and goes on).
  size_t most = kStatusBytes;
  const int G = a->heads / a->kv_heads;
  const int heights[2] = {a->dtype == EDIT_BF16 ? 128 / G : 64 / G, a->dtype == EDIT_BF16 ? 2 * (128 / G) : 64 / G};
  for (int R : heights) {
    for (int64_t rows = R - 1;; rows += R) {
      AttnPlan pl;
      attn_plan(a, rows < a->rows_q ? rows : a->rows_q, R, pl);
      if (pl.total > most) most = pl.total;
      if ((pl.nsplit == 1 && rows > 0) || rows >= a->rows_q) break;
    }
  }
  return most;
}

int edit_packed_attention_forward(const void* q, const void* k, const void* v, const edit_packed_attention* a,
                                  void* out, void* stream) {
  EDIT_TRY(attn_args(a, false));
  // (the kernels' exponents are in base 2: scale log2(e), at most twice scale, has to be finite too)
  if (!(a->scale > 0.f) || std::isinf(2.f * a->scale)) return EDIT_ERR_UNSUPPORTED;
  if (!a->q_offsets || !a->k_offsets || !a->workspace) return EDIT_ERR_NULL;
  if (a->rows_q > 0 && (!q || !out)) return EDIT_ERR_NULL;
  if (a->rows_k > 0 && (!k || !v)) return EDIT_ERR_NULL;
  const int64_t wq = static_cast<int64_t>(a->heads) * a->d, wk = static_cast<int64_t>(a->kv_heads) * a->d;
  EDIT_TRY(check_ld(a->ldq, wq));
  EDIT_TRY(check_ld(a->ldo, wq));
  EDIT_TRY(check_ld(a->ldk, wk));
  EDIT_TRY(check_ld(a->ldv, wk));
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(a->workspace, 256) ||
      !aligned(a->q_offsets, 4) || !aligned(a->k_offsets, 4) || !aligned(a->k_lens, 4))
    return EDIT_ERR_ALIGN;
  AttnPlan pl;
  attn_plan(a, a->rows_q, attn_rows(a, a->rows_q), pl);
  if (a->workspace_bytes < pl.total) return EDIT_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  PackedAttnParams p = {};
  p.q = q;
  p.k = k;
  p.v = v;
  p.out = out;
  p.q_offsets = a->q_offsets;
  p.k_offsets = a->k_offsets;
  p.k_lens = a->k_lens;
  p.ldq = a->ldq;
  p.ldk = a->ldk;
  p.ldv = a->ldv;
  p.ldo = a->ldo;
  p.rows_q = static_cast<int>(a->rows_q);
  p.rows_k = static_cast<int>(a->rows_k);
  p.heads = a->heads;
  p.kv_heads = a->kv_heads;
  p.d = a->d;
  p.nseq = a->nseq;
  p.causal = a->causal;
  p.max_k = a->max_k;
  p.scale = a->scale;
  p.slots = pl.slots;
  p.nsplit = pl.nsplit;
  p.part_o = reinterpret_cast<float*>(ws + pl.part_o);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.part_ml);
  p.status = reinterpret_cast<int*>(ws);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a->dtype == EDIT_BF16 ? attn_run<__nv_bfloat16>(p, attn_row_tiles(a, a->rows_q), st) : attn_run<float>(p, 0, st);
}

size_t edit_delta_rule_workspace_bytes(const edit_delta_rule* a) {
  if (delta_args(a, false) != EDIT_OK) return 0;
  // Fewer rows take fewer slots, but can take more parts: room for the most parts of
  // any row count.
  DeltaPlan pl;
  delta_plan(a, pl);
  if (!pl.chunked) return pl.total;
  const int64_t chunks = ceil_div(a->rows, static_cast<int64_t>(kDeltaL) * a->nseq);
  int most = 1;
  for (int64_t c = chunks < 1024 ? chunks : 1024; c >= 1; --c) {
    const int n = delta_nseg(a, c, device_sms());
    most = n > most ? n : most;
  }
  const size_t heads = static_cast<size_t>(a->nseq) * a->heads, more = most > pl.nseg ? most : 0;
  return pl.total + align256(heads * more * a->d_k * (a->d_v + a->d_k) * 4) + align256(heads * more * a->d_k * a->d_v * 4);
}

int edit_delta_rule_forward(const void* q, const void* k, const void* v, const float* g, const float* beta,
                            const edit_delta_rule* a, const float* state_in, float* state_out, void* out,
                            void* stream) {
  EDIT_TRY(delta_args(a, false));
  EDIT_TRY(delta_call(q, k, v, g, beta, a, a->rows, out));
  if (!a->offsets || !a->workspace) return EDIT_ERR_NULL;
  if (!aligned(a->workspace, 256) || !aligned(a->offsets, 4) || !aligned(state_in, 16) || !aligned(state_out, 16))
    return EDIT_ERR_ALIGN;
  DeltaPlan pl;
  delta_plan(a, pl);
  if (a->workspace_bytes < pl.total) return EDIT_ERR_WORKSPACE;
  DeltaParams p = delta_params(q, k, v, g, beta, a, out);
  p.offsets = a->offsets;
  p.state_in = state_in;
  p.state_out = state_out;
  p.status = static_cast<int*>(a->workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (pl.chunked) {
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    DeltaChunkParams c = {};
    c.d = p;
    c.blobs = ws + pl.blobs;
    c.kq = ws + pl.kq;
    c.slots = pl.slots;
    c.nseg = pl.nseg;
    c.trans = reinterpret_cast<float*>(ws + pl.trans);
    c.starts = reinterpret_cast<float*>(ws + pl.starts);
    return pl.DK == 64 ? delta_chunked<64>(c, st) : delta_chunked<128>(c, st);
  }
  return a->dtype == EDIT_BF16 ? delta_recurrent<__nv_bfloat16, false>(p, st) : delta_recurrent<float, false>(p, st);
}

int edit_delta_rule_step(const void* q, const void* k, const void* v, const float* g, const float* beta,
                         const edit_delta_rule* a, float* state, void* out, void* stream) {
  EDIT_TRY(delta_args(a, true));
  EDIT_TRY(delta_call(q, k, v, g, beta, a, a->nseq, out));
  if (!state) return EDIT_ERR_NULL;
  if (!aligned(state, 16)) return EDIT_ERR_ALIGN;
  DeltaParams p = delta_params(q, k, v, g, beta, a, out);
  p.rows = a->nseq;
  p.state_in = state;
  p.state_out = state;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a->dtype == EDIT_BF16 ? delta_single<__nv_bfloat16>(p, st) : delta_single<float>(p, st);
}

int edit_block_norm_forward(const void* x, const void* y, const edit_block_norm* a, void* r, void* h, void* stream) {
  if (!a) return EDIT_ERR_NULL;
  if (a->dtype != EDIT_F32 && a->dtype != EDIT_BF16) return EDIT_ERR_DTYPE;
  if (a->C < 1 || a->samples < 1 || a->rows < 0) return EDIT_ERR_SHAPE;
  if (a->norm_post < EDIT_NORM_NONE || a->norm_post > EDIT_NORM_RMS || a->norm_pre < EDIT_NORM_NONE ||
      a->norm_pre > EDIT_NORM_RMS || a->gate_act < EDIT_GATE_LINEAR || a->gate_act > EDIT_GATE_TANH)
    return EDIT_ERR_UNSUPPORTED;
  if ((a->norm_post == EDIT_NORM_NONE && (a->post_w || a->post_b)) ||
      (a->norm_pre == EDIT_NORM_NONE && (a->pre_w || a->pre_b)))
    return EDIT_ERR_UNSUPPORTED;
  if (a->C > 16384 || a->rows > INT32_MAX) return EDIT_ERR_UNSUPPORTED;
  if (a->rows > 0 && (!x || (!r && !h))) return EDIT_ERR_NULL;
  if (r && r == h) return EDIT_ERR_SHAPE;
  const bool mods = a->gate || a->scale || a->shift;
  if (a->ldx < a->C || (y && a->ldy < a->C) || (r && a->ldr < a->C) || (h && a->ldh < a->C) ||
      (mods && a->samples > 1 && a->ld_mod < a->C))
    return EDIT_ERR_SHAPE;
  if (!a->offsets) {
    if (a->rows_per_sample < 1 || ceil_div(a->rows, a->rows_per_sample) > a->samples) return EDIT_ERR_SHAPE;
  } else if (!aligned(a->offsets, 4)) {
    return EDIT_ERR_ALIGN;
  }
  // an output may be an input's buffer only row for row
  if ((r && r == x && a->ldr != a->ldx) || (h && h == x && a->ldh != a->ldx) || (r && r == y && a->ldr != a->ldy) ||
      (h && h == y && a->ldh != a->ldy))
    return EDIT_ERR_SHAPE;
  const uintptr_t es = a->dtype == EDIT_BF16 ? 2 : 4;
  const void* ptrs[] = {x, y, r, h, a->post_w, a->post_b, a->pre_w, a->pre_b,
                        a->gate0, a->scale0, a->shift0, a->gate, a->scale, a->shift};
  bool vec = a->C % 8 == 0 && a->ldx % 8 == 0 && (!y || a->ldy % 8 == 0) && (!r || a->ldr % 8 == 0) &&
             (!h || a->ldh % 8 == 0) && (!mods || a->samples == 1 || a->ld_mod % 8 == 0);
  for (const void* t : ptrs) {
    if (!aligned(t, es)) return EDIT_ERR_ALIGN;
    vec = vec && aligned(t, 16);
  }
  if (a->rows == 0) return EDIT_OK;
  BlockNormParams p = {};
  p.x = x;
  p.y = y;
  p.r = r;
  p.h = h;
  p.post_w = a->post_w;
  p.post_b = a->post_b;
  p.pre_w = a->pre_w;
  p.pre_b = a->pre_b;
  p.gate0 = a->gate0;
  p.scale0 = a->scale0;
  p.shift0 = a->shift0;
  p.gate = a->gate;
  p.scale = a->scale;
  p.shift = a->shift;
  p.offsets = a->offsets;
  p.rows = a->rows;
  p.rows_per_sample = a->rows_per_sample;
  p.ldx = a->ldx;
  p.ldy = a->ldy;
  p.ldr = a->ldr;
  p.ldh = a->ldh;
  p.ld_mod = a->samples > 1 ? a->ld_mod : 0;
  p.C = a->C;
  p.samples = a->samples;
  p.post = a->norm_post;
  p.pre = a->norm_pre;
  p.act = a->gate_act;
  p.eps = a->eps;
  p.rho = a->res_scale;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a->dtype == EDIT_BF16 ? norm_run<__nv_bfloat16>(p, vec, st) : norm_run<float>(p, vec, st);
}

}  // extern "C"
