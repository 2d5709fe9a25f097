// The gated delta rule over whole prompts (bf16 calls of
// edit_delta_rule_forward): chunks of 64 tokens on the tensor cores.
//
// With G the running sum of g within a chunk, k^ = rk k (rk the inverse norm, or
// 1), S0 the state before the chunk and Gamma_ij = exp(G_i - G_j):
//   T  = (I + strictly-lower(diag(beta) K^ K^^T . Gamma))^-1 diag(beta)
//   U  = T (V - diag(e^G) K^ S0)
//   O  = scale (diag(e^G) Q^ S0 + lower(Q^ K^^T . Gamma) U)
//   S1 = e^G_64 S0 + (diag(e^(G_64 - G)) K^)^T U
// T and P = lower(..) depend on no state: delta_prep_kernel forms them for all
// chunks at once. delta_chunk_kernel then walks the chunks of one (sequence,
// head); its columns of V, U, S and O are independent of each other, so a warp
// owns 16 of them and keeps the transposed products in registers: the
// accumulator layout of S^T, X^T = V^T - .., U^T is the operand layout of the
// next product (mma.sync m16n8k16), and the whole chain of a chunk needs no
// shared memory between its products and no block-wide wait. (The chain is three
// dependent products of 16 x 64 x 128 and less for each warp: too small and too
// serial for tcgen05's 128-row tiles to pay; whole heads on one tile are not.) 8192
// tokens of 16 heads of 128 take 357 us in 9 parts; profiled one by one, with cold
// caches, inverses 63, effects of the parts 164, join 36, walk 119. The walks are bound
// by mma.sync and its operands' splitting (tensor pipe half busy), 6.7 us a chunk of 8
// warps.
//
// Precision: the state is fp32. Its products take fp16 operands: a column of the
// state (of the decayed U in the state's sum) is scaled by a power of two to
// below 2 and split into two fp16 halves, a row of k likewise but in one half;
// errors are 2^-22 of the column's largest value (the dropped part, and the fp16
// floor of 2^-25 below the scale), as much of k's row for its values below 2^-15 of
// the largest. (Two bf16 halves would leave 2^-17 and three would cost half as many
// products again.) U = T X takes three bf16 parts of each, six products and 2^-24
// of each term: there the tokens of a chunk meet, and with one scale for all of them
// a large value, even of a later token or of a state since forgotten, rounded small
// ones away (three products of fp16 halves: the two walks took 264 us, now 283). O is
// rounded to bf16, so Q^ S0 takes one fp16 half, 2^-11 of the column's largest value
// for each term, and P U, whose terms a decay may set many powers of two apart, P in
// bf16 and U in two bf16 halves (with U in one, O was 1.5 times as far off as its own
// rounding).
// Values that are not finite reach what comes after them and nothing before: see
// `cut` in the walk, and the zeros above diagonals that the inverse skips.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "delta_rule.cuh"

namespace edit {

constexpr int kDeltaL = 64;    // tokens a chunk

// Lower triangles (T, P) are kept by 16-row blocks: rows of block t have the 16 (t + 1) columns up to the diagonal
// block and 8 of padding (16-byte rows without bank conflicts).
__host__ __device__ constexpr int delta_tri_ld(int t) { return 16 * t + 24; }
__host__ __device__ constexpr int delta_tri_at(int t) { return 128 * t * (t + 2); }  // first value of block t
constexpr int kDeltaMat = delta_tri_at(kDeltaL / 16) * 2;
// Per (chunk slot, head): T in three bf16 parts, the scalars, P in bf16.
enum { DS_FX, DS_W, DS_FO, DS_A, DS_COUNT };  // rows of 64 fp32 scalars
constexpr int kDeltaScal = DS_COUNT * kDeltaL * 4;
constexpr int kDeltaBlob = 4 * kDeltaMat + kDeltaScal;
// Per (chunk slot, qk head): K, Q [64][DK + 8] fp16, each row scaled to below 2.
__host__ __device__ constexpr int delta_kq_bytes(int DK) { return 2 * kDeltaL * (DK + 8) * 2; }

struct DeltaChunkParams {
  DeltaParams d;
  uint8_t* blobs;     // [slots][heads] kDeltaBlob
  uint8_t* kq;        // [slots][qk_heads] delta_kq_bytes
  int slots;
  int nseg;           // parts of a sequence's chunks (1: none)
  float* trans;       // [nseq][heads][nseg - 1][d_k][d_v + d_k]: a part's [added state | transition]
  float* starts;      // [nseq][heads][nseg][d_k][d_v]: the state before each part
};

// Power of two that brings |m| below 2 (down), and its inverse.
__device__ __forceinline__ void pow2_scale(float m, float& down, float& up) {
  int e = static_cast<int>((__float_as_uint(m) >> 23) & 0xff);
  e = e < 1 ? 1 : (e > 253 ? 253 : e);
  down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
  up = __uint_as_float(static_cast<uint32_t>(e) << 23);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
// x (a pair) as the fp16 pair nearest to it and the fp16 pair nearest to what is left.
__device__ __forceinline__ void split_f16(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 f = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = pack_f16x2(x0 - f.x, x1 - f.y);
}
// x (a pair) as three bf16 pairs, each nearest to what the ones before it leave: fp32's 24 bits and exponents.
__device__ __forceinline__ void split_bf16(float x0, float x1, uint32_t (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    p[i] = pack_bf16x2(x0, x1);
    x0 -= __uint_as_float(p[i] << 16);
    x1 -= __uint_as_float(p[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stsm_x4_t(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------- chunks by themselves
// One block a (chunk, head). Warp w forms rows 16 w .. 16 w + 15 of K K^T and
// Q K^T (exact bf16 products, fp32 sums). The unit triangular matrix is inverted
// in fp32 by blocks: four 16 x 16 blocks by forward substitution, one column a
// thread, then twice (I + A)^-1_21 = -T22 A21 T11 with small register tiles. (All
// 64 columns by forward substitution, unrolled, took 125 us for 2064 chunks and
// heads of 128, most of it fetching instructions.)
template <int DK>
struct DeltaPrepCfg {
  static constexpr int LD = DK + 8;
  static constexpr int KQ = 2 * kDeltaL * LD * 2, AT = 2 * kDeltaL * 68 * 4;
  static constexpr int SMEM = (KQ > AT ? KQ : AT) + 11 * kDeltaL * 4;  // K and Q, later A and T; rows of scalars
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool real) {  // zeros where not real
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(real ? 16 : 0)
               : "memory");
}

template <int DK>
__global__ void __launch_bounds__(128, 5) delta_prep_kernel(const DeltaChunkParams p) {
  pdl_wait();
  const DeltaParams& d = p.d;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    check_offsets(d.offsets, d.rows, nullptr, 0, nullptr, 0, d.nseq, d.status);
  using Cfg = DeltaPrepCfg<DK>;
  constexpr int L = kDeltaL, LD = Cfg::LD;
  extern __shared__ __align__(128) uint8_t dsm[];
  __nv_bfloat16* sK = reinterpret_cast<__nv_bfloat16*>(dsm);
  __nv_bfloat16* sQ = sK + L * LD;
  float* sA = reinterpret_cast<float*>(dsm);  // [64][68], over K and Q
  float* sT = sA + L * 68;                    // [64][68]
  float* sGh = reinterpret_cast<float*>(dsm + Cfg::SMEM - 11 * L * 4);  // running sum of g: high and low part
  float *sGl = sGh + L, *sB = sGl + L, *sRk = sB + L, *sRq = sRk + L, *sKd = sRq + L, *sKu = sKd + L, *sQd = sKu + L,
        *sQu = sQd + L, *sNk = sQu + L, *sNq = sNk + L;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slot = blockIdx.x, h = blockIdx.y, share = d.heads / d.qk_heads, hq = h / share;
  const int seq = seq_of_slot(d.offsets, d.nseq, static_cast<int>(d.rows), L, slot);
  const SeqRows sr = seq_rows(d.offsets, seq, static_cast<int>(d.rows));
  const int c = slot - (sr.begin / L + seq);
  if (c < 0 || c * static_cast<long>(L) >= sr.len) return;
  const int n = min(L, sr.len - c * L);
  const long row0 = sr.begin + static_cast<long>(c) * L;

  {
    const __nv_bfloat16* kg = static_cast<const __nv_bfloat16*>(d.k) + row0 * d.ldk + hq * d.d_k;
    const __nv_bfloat16* qg = static_cast<const __nv_bfloat16*>(d.q) + row0 * d.ldq + hq * d.d_k;
#pragma unroll
    for (int e = tid; e < L * (DK / 8); e += 128) {
      const int r = e / (DK / 8), x = (e % (DK / 8)) * 8;
      const bool real = r < n && x < d.d_k;
      cp_async16(sK + r * LD + x, real ? kg + r * d.ldk + x : kg, real);
      cp_async16(sQ + r * LD + x, real ? qg + r * d.ldq + x : qg, real);
    }
  }
  double G = 0.0;
  if (tid < L) {  // running sums of g in fp64: differences of far sums keep their fp32 precision
    if (tid < n) G = static_cast<double>(log_decay(d.g[(row0 + tid) * d.ldg + h]));
    sB[tid] = tid < n ? d.beta[(row0 + tid) * d.ldb + h] : 0.f;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double a = __shfl_up_sync(0xffffffffu, G, o);
      if (lane >= o) G += a;
    }
    if (tid == 31) {
      sGh[0] = static_cast<float>(G);
      sGl[0] = static_cast<float>(G - static_cast<double>(sGh[0]));
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  if (warp == 1) G += static_cast<double>(sGh[0]) + static_cast<double>(sGl[0]);
  uint8_t* blob = p.blobs + (static_cast<long>(slot) * d.heads + h) * kDeltaBlob;
  float* scal = reinterpret_cast<float*>(blob + 3 * kDeltaMat);
  // K K^T and Q K^T of this warp's 16 rows, columns up to its diagonal block; |q|^2 from the diagonal of Q Q^T
  const int gr = lane >> 2, q2 = 2 * (lane & 3);
  float kk[8][4] = {}, qk[8][4] = {}, qq[2][4] = {};
  {
    const uint32_t ka = smem_u32(sK), qa = smem_u32(sQ);
    const uint32_t arow = (16 * warp + (lane & 15)) * LD * 2 + (lane >> 4) * 16;
    const uint32_t brow = ((lane & 7) + ((lane >> 4) << 3)) * LD * 2 + ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int k = 0; k < DK / 16; ++k) {
      uint32_t a[4], q[4], b[4];
      ldsm_x4(ka + arow + 32 * k, a);
      ldsm_x4(qa + arow + 32 * k, q);
      ldsm_x4(qa + brow + warp * 16 * LD * 2 + 32 * k, b);
      mma_bf16(qq[0], q, b[0], b[1]);
      mma_bf16(qq[1], q, b[2], b[3]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (t > warp) break;
        ldsm_x4(ka + brow + t * 16 * LD * 2 + 32 * k, b);
        mma_bf16(kk[2 * t], a, b[0], b[1]);
        mma_bf16(kk[2 * t + 1], a, b[2], b[3]);
        mma_bf16(qk[2 * t], q, b[0], b[1]);
        mma_bf16(qk[2 * t + 1], q, b[2], b[3]);
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)  // diagonal: row gr (+ 8) of the block in its first (second) 8 columns
      if (t == warp) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (q2 + e == gr) {
            sNk[16 * t + gr] = kk[2 * t][e];
            sNk[16 * t + gr + 8] = kk[2 * t + 1][2 + e];
            sNq[16 * t + gr] = qq[0][e];
            sNq[16 * t + gr + 8] = qq[1][2 + e];
          }
      }
  }
  __syncthreads();
  {
    const int t = tid & 63;
    const float s = (tid < 64 ? sNk : sNq)[t];
    float m = sqrtf(s), down, up;  // no value is larger than the norm, where its square has not left fp32's range
    if (!(s > 1e-30f && s < 1e38f)) {
      const uint32_t* row = reinterpret_cast<const uint32_t*>((tid < 64 ? sK : sQ) + t * LD);
      uint32_t most = 0;
      for (int x = 0; x < DK / 2; ++x) most = max(most, max(row[x] << 16 & 0x7fff0000u, row[x] & 0x7fff0000u));
      m = __uint_as_float(most);
    }
    pow2_scale(m, down, up);
    (tid < 64 ? sRk : sRq)[t] = t >= n ? 0.f : (d.qk_norm ? 1.f / sqrtf(s + d.qk_eps) : 1.f);
    (tid < 64 ? sKd : sQd)[t] = down;
    (tid < 64 ? sKu : sQu)[t] = up;
    if (tid < 64) {
      const float hi = static_cast<float>(G);
      sGh[tid] = hi;
      sGl[tid] = static_cast<float>(G - static_cast<double>(hi));
    }
  }
  __syncthreads();
  if (tid < L) {
    const float eG = expf(sGh[tid]), rest = expf((sGh[L - 1] - sGh[tid]) + (sGl[L - 1] - sGl[tid]));
    scal[DS_FX * L + tid] = eG * sRk[tid] * sKu[tid];
    scal[DS_W * L + tid] = rest * sRk[tid] * sKu[tid];
    scal[DS_FO * L + tid] = d.scale * eG * sRq[tid] * sQu[tid];
    scal[DS_A * L + tid] = expf(sGh[L - 1]);
  }
  {
    __nv_bfloat16* P = reinterpret_cast<__nv_bfloat16*>(blob + 3 * kDeltaMat + kDeltaScal) + delta_tri_at(warp);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t > 2 * warp + 1) break;
      const int j = 8 * t + q2;
      const float2 gh = *reinterpret_cast<const float2*>(sGh + j), gl = *reinterpret_cast<const float2*>(sGl + j),
                   rk = *reinterpret_cast<const float2*>(sRk + j);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int i = 16 * warp + gr + 8 * r;
        const float hi = sGh[i], lo = sGl[i], bk = sB[i] * sRk[i], rq = d.scale * sRq[i];
        const float g0 = j <= i ? expf((hi - gh.x) + (lo - gl.x)) * rk.x : 0.f;
        const float g1 = j + 1 <= i ? expf((hi - gh.y) + (lo - gl.y)) * rk.y : 0.f;
        kk[t][2 * r] = j < i ? bk * g0 * kk[t][2 * r] : 0.f;
        kk[t][2 * r + 1] = j + 1 < i ? bk * g1 * kk[t][2 * r + 1] : 0.f;
        *reinterpret_cast<uint32_t*>(P + (i & 15) * delta_tri_ld(warp) + j) =
            pack_bf16x2(j <= i ? g0 * rq * qk[t][2 * r] : 0.f, j + 1 <= i ? g1 * rq * qk[t][2 * r + 1] : 0.f);
      }
    }
  }
  if (h % share == 0) {  // fp16 K and Q for all heads that share them
    __half* K16 = reinterpret_cast<__half*>(p.kq + (static_cast<long>(slot) * d.qk_heads + hq) * delta_kq_bytes(DK));
#pragma unroll 4
    for (int e = tid; e < 2 * L * (DK / 8); e += 128) {
      const int r = e / (DK / 8), x = (e % (DK / 8)) * 8;  // rows of K, then of Q
      const uint4 u = *reinterpret_cast<const uint4*>(sK + r * LD + x);
      const float s = r < L ? sKd[r] : sQd[r - L];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = pack_f16x2(__uint_as_float(w[j] << 16) * s, __uint_as_float(w[j] & 0xffff0000u) * s);
      *reinterpret_cast<uint4*>(K16 + r * LD + x) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  __syncthreads();  // K and Q are done with
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    if (t > 2 * warp + 1) break;
#pragma unroll
    for (int r = 0; r < 2; ++r)
      *reinterpret_cast<float2*>(sA + (16 * warp + gr + 8 * r) * 68 + 8 * t + q2) =
          make_float2(kk[t][2 * r], kk[t][2 * r + 1]);
  }
  for (int e = tid; e < L * 17; e += 128) *reinterpret_cast<float4*>(sT + 4 * e) = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
  if (tid < L) {  // diagonal blocks, column tid: x_i = [i = j] - sum_{l < i} A_il x_l
    const int o = tid & ~15, j = tid & 15;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s0 = i == j ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
      for (int l = 0; l < i; ++l) {
        const float a = sA[(o + i) * 68 + o + l];
        if (l & 1)
          s1 = fmaf(-a, x[l], s1);
        else
          s0 = fmaf(-a, x[l], s0);
      }
      x[i] = s0 + s1;
      sT[(o + i) * 68 + tid] = x[i];
    }
  }
  __syncthreads();
  // rows o2 .. o2 + N - 1, columns o1 .. o1 + N - 1 of the inverse, o2 = o1 + N: first A21 T11, then -T22 of it; a
  // thread holds RT rows x 4 columns
  auto merge = [&](auto size, auto rows, int o1, int u) {
    constexpr int N = decltype(size)::value, RT = decltype(rows)::value;
    const int o2 = o1 + N, r = (u / (N / 4)) * RT, x = (u % (N / 4)) * 4;
    float y[RT][4];
    auto product = [&](const float* A, const float* B, auto lower) {  // lower: A's zeros above its diagonal are skipped
#pragma unroll
      for (int i = 0; i < RT; ++i) y[i][0] = y[i][1] = y[i][2] = y[i][3] = 0.f;
#pragma unroll 4
      for (int k = 0; k < (decltype(lower)::value ? r + RT : N); ++k) {
        const float4 b = *reinterpret_cast<const float4*>(B + k * 68 + x);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          if (decltype(lower)::value && k > r + i) continue;
          const float a = A[(r + i) * 68 + k];
          y[i][0] = fmaf(a, b.x, y[i][0]);
          y[i][1] = fmaf(a, b.y, y[i][1]);
          y[i][2] = fmaf(a, b.z, y[i][2]);
          y[i][3] = fmaf(a, b.w, y[i][3]);
        }
      }
    };
    float* to = sT + o2 * 68 + o1;
    product(sA + o2 * 68 + o1, sT + o1 * 68 + o1, std::false_type{});
#pragma unroll
    for (int i = 0; i < RT; ++i)
      *reinterpret_cast<float4*>(to + (r + i) * 68 + x) = make_float4(y[i][0], y[i][1], y[i][2], y[i][3]);
    __syncthreads();
    product(sT + o2 * 68 + o2, to, std::true_type{});
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RT; ++i)
      *reinterpret_cast<float4*>(to + (r + i) * 68 + x) = make_float4(-y[i][0], -y[i][1], -y[i][2], -y[i][3]);
    __syncthreads();
  };
  merge(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{}, 32 * (tid >> 6), tid & 63);
  merge(std::integral_constant<int, 32>{}, std::integral_constant<int, 2>{}, 0, tid);
#pragma unroll
  for (int e = tid; e < L * 8; e += 128) {  // T = inverse diag(beta), 8 values of a row a thread
    const int i = e >> 3, j = (e & 7) * 8, t = i >> 4;
    if (j >= 16 * (t + 1)) continue;
    uint32_t w[4][3];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = j + 2 * k;
      const float2 x = *reinterpret_cast<const float2*>(sT + i * 68 + c), b = *reinterpret_cast<const float2*>(sB + c);
      split_bf16(c <= i ? x.x * b.x : 0.f, c + 1 <= i ? x.y * b.y : 0.f, w[k]);
    }
    __nv_bfloat16* T = reinterpret_cast<__nv_bfloat16*>(blob) + delta_tri_at(t) + (i & 15) * delta_tri_ld(t) + j;
#pragma unroll
    for (int k = 0; k < 3; ++k)
      *reinterpret_cast<uint4*>(T + k * (kDeltaMat / 2)) = make_uint4(w[0][k], w[1][k], w[2][k], w[3][k]);
  }
}

// ---------------------------------------------------------------- chunk after chunk
// cp.async.bulk of contiguous bytes (16-byte aligned) into shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

constexpr int kDeltaCols = 128;  // state columns a block (8 warps)

template <int DK>
struct DeltaChunkCfg {  // two stages of K, Q, a blob and V's columns of `warps` warps
  static constexpr int LD = DK + 8;  // row stride of K, Q
  static constexpr int KQ = delta_kq_bytes(DK);
  static constexpr int stage(int warps) { return KQ + kDeltaBlob + kDeltaL * (16 * warps + 8) * 2; }
  static constexpr int smem(int warps) { return 2 * stage(warps) + 64; }
  static_assert(smem(8) <= 232448, "shared memory");
};

// OUT: the outputs and final states of all columns from the right start states.
// Otherwise: what a part of a sequence adds to the state and does to it, as
// d_v + d_k columns: the columns of V from a zero state, then, with V = 0, the
// unit columns, which become the part's transition matrix.
template <int DK, bool OUT>
__global__ void __launch_bounds__(288, 1) delta_chunk_kernel(const DeltaChunkParams p, int col_blocks) {
  pdl_wait();
  using Cfg = DeltaChunkCfg<DK>;
  constexpr int L = kDeltaL, LD = Cfg::LD, NT = DK / 8;
  const int workers = blockDim.x / 32 - 1;  // warps with 16 columns each; the last warp loads
  const int LDV = 16 * workers + 8, STAGE = Cfg::KQ + kDeltaBlob + L * LDV * 2;
  extern __shared__ __align__(128) uint8_t dsm[];
  uint8_t* sm = dsm;
  const DeltaParams& d = p.d;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + 2 * STAGE);  // [2]
  uint64_t* empty = full + 2;                                     // [2]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + 2);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nthr = blockDim.x;
  const int h = blockIdx.y, hq = h / (d.heads / d.qk_heads);
  const int cb = blockIdx.x % col_blocks, rest = blockIdx.x / col_blocks;
  const int segs = OUT ? p.nseg : p.nseg - 1;
  const int seg = rest % segs, seq = rest / segs;
  const SeqRows sr = seq_rows(d.offsets, seq, static_cast<int>(d.rows));
  const int chunks = (sr.len + L - 1) / L, slot0 = sr.begin / L + seq;
  const int c0 = static_cast<int>(static_cast<long>(chunks) * seg / p.nseg);
  const int c1 = static_cast<int>(static_cast<long>(chunks) * (seg + 1) / p.nseg);
  const int cols = OUT ? d.d_v : d.d_v + d.d_k;  // columns of this call
  const int col0 = cb * kDeltaCols;              // of this block
  const int vcols = min(max(d.d_v - col0, 0), kDeltaCols);  // of them, columns of V
  if (tid == 0) {
    mbar_init(&full[0], 1);
    mbar_init(&full[1], 1);
    mbar_init(&empty[0], workers);
    mbar_init(&empty[1], workers);
    *abort_flag = 0;
    fence_mbar_init();
  }
  for (int s = 0; s < 2; ++s)  // (columns past V's stay zero)
    for (int e = tid; e < L * LDV / 8; e += nthr)
      *reinterpret_cast<uint4*>(sm + s * STAGE + Cfg::KQ + kDeltaBlob + e * 16) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncthreads();

  if (warp == workers) {
    // ------------------------------------------------------------ loads: chunk c into stage c - c0 mod 2
    for (int c = c0; c < c1; ++c) {
      uint8_t* st = sm + ((c - c0) & 1) * STAGE;
      uint64_t* bar = &full[(c - c0) & 1];
      if (!warp_wait(&empty[(c - c0) & 1], (((c - c0) >> 1) & 1) ^ 1, abort_flag, d.status)) {
        let_copies_land();
        break;
      }
      const int n = min(L, sr.len - c * L);
      __nv_bfloat16* v = reinterpret_cast<__nv_bfloat16*>(st + Cfg::KQ + kDeltaBlob);
      for (int r = n; r < L; ++r)  // rows behind the sequence: zeros
        for (int x = lane; x < vcols / 8; x += 32)
          *reinterpret_cast<uint4*>(v + r * LDV + 8 * x) = make_uint4(0u, 0u, 0u, 0u);
      __syncwarp();
      const uint32_t kq = OUT ? Cfg::KQ : Cfg::KQ / 2, bl = OUT ? kDeltaBlob : kDeltaBlob - kDeltaMat;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, kq + bl + n * vcols * 2);
        bulk_load(st, p.kq + (static_cast<long>(slot0 + c) * d.qk_heads + hq) * Cfg::KQ, kq, bar);
        bulk_load(st + Cfg::KQ, p.blobs + (static_cast<long>(slot0 + c) * d.heads + h) * kDeltaBlob, bl, bar);
      }
      __syncwarp();
      if (vcols > 0)
        for (int r = lane; r < n; r += 32)
          bulk_load(v + r * LDV,
                    static_cast<const __nv_bfloat16*>(d.v) + (sr.begin + static_cast<long>(c) * L + r) * d.ldv +
                        h * d.d_v + col0,
                    vcols * 2, bar);
    }
    return;
  }

  // S^T of this warp's 16 columns (rows g and g + 8 of the accumulators), by 8 rows of the state
  const int g = lane >> 2, q2 = 2 * (lane & 3);
  const int my = col0 + 16 * warp;  // first column
  float S[NT][4];
  const long head = static_cast<long>(seq) * d.heads + h;
  const float* start = nullptr;
  if (OUT)
    // (with parts, the first's too: the last part's block may be done with state_out, the same buffer, before the
    // first's begins)
    start = p.nseg > 1 ? p.starts + (head * p.nseg + seg) * d.d_k * d.d_v
                       : (d.state_in ? d.state_in + head * d.d_k * d.d_v : nullptr);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 8 * t + q2 + (e & 1), j = my + g + 8 * (e >> 1);
      if (OUT)
        S[t][e] = start && i < d.d_k && j < d.d_v ? start[static_cast<long>(i) * d.d_v + j] : 0.f;
      else
        S[t][e] = j - d.d_v == i ? 1.f : 0.f;
    }

  // addresses of this lane in ldmatrix's four 8 x 8 blocks
  const int m_row = (lane & 7) + ((lane >> 4) << 3), m_col = ((lane >> 3) & 1) * 8;  // (n, k) blocks of a row-major B
  const int t_row = lane & 15, t_col = (lane >> 4) * 8;                              // (k, n) blocks, transposed
  for (int c = c0; c < c1; ++c) {
    uint8_t* st = sm + ((c - c0) & 1) * STAGE;
    if (!warp_wait(&full[(c - c0) & 1], ((c - c0) >> 1) & 1, abort_flag, d.status)) {
      let_copies_land();
      break;
    }
    const uint32_t sK = smem_u32(st), sQ = sK + Cfg::KQ / 2, sT = sK + Cfg::KQ, sP = sT + 3 * kDeltaMat + kDeltaScal;
    const float* scal = reinterpret_cast<const float*>(st + Cfg::KQ + 3 * kDeltaMat);
    const uint32_t sV = sT + kDeltaBlob + 16 * warp * 2;

    // rows of S^T as fp16 halves; X = K S0 (transposed)
    float mx[2] = {0.f, 0.f}, s_dn[2], s_up[2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], fabsf(S[t][e]));
    auto row_scale = [&](float (&dn)[2], float (&up)[2]) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        pow2_scale(mx[r], dn[r], up[r]);
      }
    };
    row_scale(s_dn, s_up);
    float X[8][4] = {};
#pragma unroll
    for (int k = 0; k < DK / 16; ++k) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int t = 2 * k + (b >> 1), r = b & 1;
        split_f16(S[t][2 * r] * s_dn[r], S[t][2 * r + 1] * s_dn[r], hi[b], lo[b]);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        uint32_t b[4];
        ldsm_x4(sK + ((16 * t + m_row) * LD + 16 * k + m_col) * 2, b);
        mma_f16(X[2 * t], hi, b[0], b[1]);
        mma_f16(X[2 * t + 1], hi, b[2], b[3]);
        mma_f16(X[2 * t], lo, b[0], b[1]);
        mma_f16(X[2 * t + 1], lo, b[2], b[3]);
      }
    }
    // X = V - e^G K^ S0
#pragma unroll
    for (int t = 0; t < 4; ++t) {  // 16 tokens
      uint32_t v[4];
      // blocks: tokens 16 t + 0..7 / 8..15 (rows) x this warp's columns 0..7 / 8..15, transposed
      ldsm_x4_t(sV + ((16 * t + (lane & 7) + ((lane >> 4) << 3)) * LDV + ((lane >> 3) & 1) * 8) * 2, v);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float2 fx = *reinterpret_cast<const float2*>(scal + DS_FX * L + 16 * t + 8 * u + q2);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t w = v[2 * u + r];
          float(&x)[4] = X[2 * t + u];
          x[2 * r] = fmaf(-x[2 * r], s_up[r] * fx.x, __uint_as_float(w << 16));
          x[2 * r + 1] = fmaf(-x[2 * r + 1], s_up[r] * fx.y, __uint_as_float(w & 0xffff0000u));
        }
      }
    }
    // A column's tokens from the first one on that is not finite: cleared for the products, in which it would reach the
    // tokens before it (0 times it, above the diagonals of T and P), and not finite in what comes out. From 2^128 - 2^119
    // on a value is infinite in bf16 and counts as such.
    int cut[2] = {L, L};
    auto odd = [](const float(&m)[8][4]) {
      float z[2] = {0.f, 0.f};
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e & 1] = fmaf(m[t][e], 4.f, z[e & 1]);
      return __any_sync(0xffffffffu, !(fabsf(z[0]) < INFINITY && fabsf(z[1]) < INFINITY)) != 0;  // (or sums past 2^128)
    };
    auto clear = [&](float(&m)[8][4]) {
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!(fabsf(m[t][e]) < 0x1.ffp127f)) cut[e >> 1] = min(cut[e >> 1], 8 * t + q2 + (e & 1));
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        cut[r] = min(cut[r], __shfl_xor_sync(0xffffffffu, cut[r], 1));
        cut[r] = min(cut[r], __shfl_xor_sync(0xffffffffu, cut[r], 2));
      }
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * t + q2 + (e & 1) >= cut[e >> 1]) m[t][e] = 0.f;
    };
    bool bad = odd(X);
    if (bad) clear(X);
    // U = T X, both in three bf16 parts: one scale for the column would round small values beside a large one away, of
    // tokens before it too
    float U[8][4] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t x[3][4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int t = 2 * k + (b >> 1), r = b & 1;
        uint32_t w[3];
        split_bf16(X[t][2 * r], X[t][2 * r + 1], w);
#pragma unroll
        for (int i = 0; i < 3; ++i) x[i][b] = w[i];
      }
#pragma unroll
      for (int t = k; t < 4; ++t)  // rows of T from the diagonal block down
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          uint32_t b[4];
          ldsm_x4(sT + i * kDeltaMat + (delta_tri_at(t) + m_row * delta_tri_ld(t) + 16 * k + m_col) * 2, b);
#pragma unroll
          for (int y = 0; y < 3 - i; ++y) {  // (the products left out are 2^-24 of the whole)
            mma_bf16(U[2 * t], x[y], b[0], b[1]);
            mma_bf16(U[2 * t + 1], x[y], b[2], b[3]);
          }
        }
    }
    if (bad || odd(U)) {
      bad = true;
      clear(U);
    }
    if (OUT) {
      // O = Q^ S0 e^G + P U, rounded to bf16, through this warp's columns of V's tile (Q S0 only now: beside X and U its
      // accumulators do not fit into the registers)
      float O[8][4] = {};
#pragma unroll
      for (int k = 0; k < DK / 16; ++k) {
        uint32_t hi[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int t = 2 * k + (b >> 1), r = b & 1;
          hi[b] = pack_f16x2(S[t][2 * r] * s_dn[r], S[t][2 * r + 1] * s_dn[r]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          uint32_t b[4];
          ldsm_x4(sQ + ((16 * t + m_row) * LD + 16 * k + m_col) * 2, b);
          mma_f16(O[2 * t], hi, b[0], b[1]);
          mma_f16(O[2 * t + 1], hi, b[2], b[3]);
        }
      }
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const float2 fo = *reinterpret_cast<const float2*>(scal + DS_FO * L + 8 * t + q2);
#pragma unroll
        for (int e = 0; e < 4; ++e) O[t][e] *= s_up[e >> 1] * (e & 1 ? fo.y : fo.x);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t a[4], lo[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int t = 2 * k + (b >> 1), r = b & 1;
          a[b] = pack_bf16x2(U[t][2 * r], U[t][2 * r + 1]);
          lo[b] = pack_bf16x2(U[t][2 * r] - __uint_as_float(a[b] << 16),
                              U[t][2 * r + 1] - __uint_as_float(a[b] & 0xffff0000u));
        }
#pragma unroll
        for (int t = k; t < 4; ++t) {
          uint32_t b[4];
          ldsm_x4(sP + (delta_tri_at(t) + m_row * delta_tri_ld(t) + 16 * k + m_col) * 2, b);
          mma_bf16(O[2 * t], a, b[0], b[1]);
          mma_bf16(O[2 * t + 1], a, b[2], b[3]);
          mma_bf16(O[2 * t], lo, b[0], b[1]);
          mma_bf16(O[2 * t + 1], lo, b[2], b[3]);
        }
      }
      if (bad) {
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (8 * t + q2 + (e & 1) >= cut[e >> 1]) O[t][e] = NAN;
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        uint32_t o[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int u = 2 * t + (b >> 1), r = b & 1;
          o[b] = pack_bf16x2(O[u][2 * r], O[u][2 * r + 1]);
        }
        stsm_x4_t(sV + ((16 * t + (lane & 7) + ((lane >> 4) << 3)) * LDV + ((lane >> 3) & 1) * 8) * 2, o);
      }
      __syncwarp();
      const int n = min(L, sr.len - c * L);
      const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(st + Cfg::KQ + kDeltaBlob) + 16 * warp;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(d.out) + (sr.begin + static_cast<long>(c) * L) * d.ldo + h * d.d_v + my;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 16 * e + (lane >> 1), x = (lane & 1) * 8;
        if (r < n && my + x < d.d_v)
          *reinterpret_cast<uint4*>(out + r * d.ldo + x) = *reinterpret_cast<const uint4*>(v + r * LDV + x);
      }
    }
    // S = e^G_64 S + (e^(G_64 - G) K^)^T U
    mx[0] = mx[1] = 0.f;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const float2 f = *reinterpret_cast<const float2*>(scal + DS_W * L + 8 * t + q2);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        U[t][e] *= e & 1 ? f.y : f.x;
        mx[e >> 1] = fmaxf(mx[e >> 1], fabsf(U[t][e]));
      }
    }
    float w_dn[2], w_up[2];
    row_scale(w_dn, w_up);
    uint32_t hi[4][4], lo[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int t = 2 * k + (b >> 1), r = b & 1;
        split_f16(U[t][2 * r] * w_dn[r], U[t][2 * r + 1] * w_dn[r], hi[k][b], lo[k][b]);
      }
    const float a = scal[DS_A * L];
#pragma unroll
    for (int t = 0; t < NT; t += 2) {
      float D[2][4] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t b[4];
        ldsm_x4_t(sK + ((16 * k + t_row) * LD + 8 * t + t_col) * 2, b);
        mma_f16(D[0], hi[k], b[0], b[1]);
        mma_f16(D[1], hi[k], b[2], b[3]);
        mma_f16(D[0], lo[k], b[0], b[1]);
        mma_f16(D[1], lo[k], b[2], b[3]);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[t + u][e] = fmaf(D[u][e], w_up[e >> 1], a * S[t + u][e]);
    }
    if (bad) {  // what is not finite stays in a state
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (cut[e >> 1] < L) S[t][e] = NAN;
    }
    fence_proxy_async_smem();  // (outputs were staged where the next loads go)
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[(c - c0) & 1]);
  }

  float* end = nullptr;
  if (OUT) {
    if (d.state_out && seg == p.nseg - 1) end = d.state_out + head * d.d_k * d.d_v;
  } else {
    end = p.trans + (head * (p.nseg - 1) + seg) * d.d_k * cols;
  }
  if (end) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 8 * t + q2 + (e & 1), j = my + g + 8 * (e >> 1);
        if (i < d.d_k && j < cols) end[static_cast<long>(i) * cols + j] = S[t][e];
      }
  }
}

// The state before each part: starts[0] = state_in, starts[s + 1] = B_s + M_s
// starts[s] (fp32). One block for 16 columns of one (sequence, head); a
// thread sums half of the products of 4 x 4 values (the steps are dependent, so
// their latency is the time: 5.3 us a step with whole sums, 128 x 128); the next
// part's M is fetched while this one's is used.
template <int DK>
struct DeltaJoinCfg {
  static constexpr int LDM = DK + 4;
  static constexpr int SMEM = (2 * DK * LDM + 2 * DK * 16) * 4;
};
template <int DK>
__global__ void __launch_bounds__(2 * DK) delta_join_kernel(const DeltaChunkParams p) {
  pdl_wait();
  constexpr int LDM = DeltaJoinCfg<DK>::LDM;
  extern __shared__ __align__(128) uint8_t dsm[];
  const DeltaParams& d = p.d;
  float* sM = reinterpret_cast<float*>(dsm);  // [2][DK][LDM]
  float* sS = sM + 2 * DK * LDM;              // [DK][16]
  float* sH = sS + DK * 16;                   // [DK][16] sums of the second half
  const int h = blockIdx.y, seq = blockIdx.z, col0 = blockIdx.x * 16;
  const long head = static_cast<long>(seq) * d.heads + h;
  const int cols = d.d_v + d.d_k, tid = threadIdx.x;
  const int half = tid / DK, r0 = ((tid % DK) >> 2) * 4, x0 = (tid & 3) * 4;  // this thread's half, rows and columns
  const bool in = half == 0 && col0 + x0 < d.d_v;
  auto fetch = [&](int s) {  // M_s; rows and columns past d_k are left as they are: their products meet zeros of S
    const float* tr = p.trans + (head * (p.nseg - 1) + s) * d.d_k * cols + d.d_v;
    float* to = sM + (s & 1) * DK * LDM;
    for (int e = tid; e < d.d_k * (d.d_k / 4); e += 2 * DK) {
      const int i = e / (d.d_k / 4), k = (e % (d.d_k / 4)) * 4;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to + i * LDM + k)),
                   "l"(tr + static_cast<long>(i) * cols + k)
                   : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int e = tid; e < 2 * DK * LDM / 4; e += 2 * DK) *reinterpret_cast<float4*>(sM + 4 * e) = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
  fetch(0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (d.state_in && in && r0 + i < d.d_k)
      a = *reinterpret_cast<const float4*>(d.state_in + (head * d.d_k + r0 + i) * d.d_v + col0 + x0);
    if (half == 0) *reinterpret_cast<float4*>(sS + (r0 + i) * 16 + x0) = a;
    if (in && r0 + i < d.d_k)
      *reinterpret_cast<float4*>(p.starts + (head * p.nseg * d.d_k + r0 + i) * d.d_v + col0 + x0) = a;
  }
  for (int s = 0; s + 1 < p.nseg; ++s) {
    const float* tr = p.trans + (head * (p.nseg - 1) + s) * d.d_k * cols + col0 + x0;
    float acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      if (in && r0 + i < d.d_k) a = *reinterpret_cast<const float4*>(tr + static_cast<long>(r0 + i) * cols);
      acc[i][0] = a.x; acc[i][1] = a.y; acc[i][2] = a.z; acc[i][3] = a.w;
    }
    if (s + 2 < p.nseg) {
      fetch(s + 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const float* M = sM + (s & 1) * DK * LDM;
#pragma unroll 2
    for (int k = half * (DK / 2); k < (half + 1) * (DK / 2); k += 4) {
      float4 m[4], v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = *reinterpret_cast<const float4*>(M + (r0 + i) * LDM + k);
        v[i] = *reinterpret_cast<const float4*>(sS + (k + i) * 16 + x0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float mk[4] = {m[i].x, m[i].y, m[i].z, m[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][0] = fmaf(mk[j], v[j].x, acc[i][0]);
          acc[i][1] = fmaf(mk[j], v[j].y, acc[i][1]);
          acc[i][2] = fmaf(mk[j], v[j].z, acc[i][2]);
          acc[i][3] = fmaf(mk[j], v[j].w, acc[i][3]);
        }
      }
    }
    if (half == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(sH + (r0 + i) * 16 + x0) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    }
    __syncthreads();
    float* to = p.starts + (head * p.nseg + s + 1) * d.d_k * d.d_v + col0 + x0;
    if (half == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 b = *reinterpret_cast<const float4*>(sH + (r0 + i) * 16 + x0);
        const float4 a = make_float4(acc[i][0] + b.x, acc[i][1] + b.y, acc[i][2] + b.z, acc[i][3] + b.w);
        *reinterpret_cast<float4*>(sS + (r0 + i) * 16 + x0) = a;
        if (in && r0 + i < d.d_k) *reinterpret_cast<float4*>(to + static_cast<long>(r0 + i) * d.d_v) = a;
      }
    }
  }
}

}  // namespace edit
