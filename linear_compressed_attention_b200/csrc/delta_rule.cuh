// The gated delta rule (edit_delta_rule_forward, edit_delta_rule_step).
#pragma once

#include "packed_seq.cuh"

namespace edit {

// Log decays are limited below here: exp is 0 in fp32 from -104 on, and finite
// sums of them keep differences of sums defined.
constexpr float kMinLogDecay = -200.f;

struct DeltaParams {
  const void *q, *k, *v;
  const float *g, *beta;
  const float* state_in;
  float* state_out;
  void* out;
  const int32_t* offsets;  // nullptr: one row a sequence
  long rows, ldq, ldk, ldv, ldo, ldg, ldb;
  int qk_heads, heads, d_k, d_v, nseq, qk_norm;
  float scale, qk_eps;
  int* status;  // nullptr: none
};

// A NaN passes.
__device__ __forceinline__ float log_decay(float g) { return g < kMinLogDecay ? kMinLogDecay : g; }

template <typename T>
__device__ __forceinline__ void load4(const T* p, float* o) {
  if constexpr (sizeof(T) == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    o[0] = __uint_as_float(u.x << 16);
    o[1] = __uint_as_float(u.x & 0xffff0000u);
    o[2] = __uint_as_float(u.y << 16);
    o[3] = __uint_as_float(u.y & 0xffff0000u);
  } else {
    const float4 a = *reinterpret_cast<const float4*>(p);
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
  }
}

// Token by token, the state in registers. A warp holds 4 CPT columns of one
// (sequence, head)'s state: lane = 8 cg + l keeps columns CPT cg .. and the rows
// 4 (l + 8 m) .. + 3, so that the sums over d_k are three shuffles over 8 lanes.
// CPT is 4 for single tokens (a state row's 16 columns are 64 contiguous bytes;
// they are bound by the state's bytes) and 2 for sequences, where a warp's
// instructions per token are the time (4: 0.37 us a token, d_k = 64). Both
// products with the state, S^T k and S^T q, are taken of the state before the
// token (o = e^g S^T q + (k.q) u), so that a token costs one round of shuffles.
// The state is kept as S / A with A the decay since it was last brought up to
// date (every 16 tokens, or when the log of A leaves +-8): a rounding of every
// value for the decay of every token was most of the state's error (400 fp32
// tokens: 1.1e-6 of its norm).
// STEP: one token of each sequence, straight from memory. Otherwise the block's
// tokens come 16 at a time through shared memory, copied while the 16 before
// them are worked on, and what does not depend on the state (norms, k.q, the
// decays) is found for the 16 at once before the walk (in the walk it was half
// of a token's 0.4 us, which is all latency).
constexpr int kDeltaTokens = 16;

template <bool STEP>
constexpr int kDeltaCpt = STEP ? 4 : 2;  // columns a thread; 16 times that a block

template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float* o) {
  if constexpr (N == 4) {
    load4(p, o);
  } else if constexpr (sizeof(T) == 2) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    o[0] = __uint_as_float(u << 16);
    o[1] = __uint_as_float(u & 0xffff0000u);
  } else {
    const float2 a = *reinterpret_cast<const float2*>(p);
    o[0] = a.x; o[1] = a.y;
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, const float* o) {
  if constexpr (sizeof(T) == 2 && N == 4)
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
  else if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(o[0], o[1]);
  else if constexpr (N == 4)
    *reinterpret_cast<float4*>(p) = make_float4(o[0], o[1], o[2], o[3]);
  else
    *reinterpret_cast<float2*>(p) = make_float2(o[0], o[1]);
}

template <typename T, int DK, int COLS>
struct DeltaTokens {  // one stage
  T q[kDeltaTokens][DK], k[kDeltaTokens][DK], v[kDeltaTokens][COLS];
  float g[kDeltaTokens], beta[kDeltaTokens];
};

struct DeltaScalars {
  float rk, rq;    // 1 / |k| (or 1), scale / |q|
  float kq;        // k . q
  float settle;    // the factor that brings the state up to date before the token, 1 for none
  float A, invA;   // decay held back after it, and its inverse
};

// The decay of the next token joins what is held back; past +-8, or with `all`, everything is settled (a NaN settles).
__device__ __forceinline__ void hold_decay(float& logA, float g, bool all, DeltaScalars& x) {
  logA += log_decay(g);
  x.settle = x.A = x.invA = 1.f;
  if (all || !(fabsf(logA) <= 8.f)) {
    x.settle = expf(logA);
    logA = 0.f;
  }
}

template <int BYTES>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

template <typename T, int DK, bool STEP>
__global__ void __launch_bounds__(128) delta_recurrent_kernel(const DeltaParams p, int col_blocks) {
  pdl_wait();
  if (p.status && blockIdx.x == 0 && blockIdx.y == 0)
    check_offsets(p.offsets, p.rows, nullptr, 0, nullptr, 0, p.nseq, p.status);
  constexpr int RM = DK / 32, CPT = kDeltaCpt<STEP>, COLS = 16 * CPT;
  using Tokens = DeltaTokens<T, DK, COLS>;
  __shared__ __align__(16) Tokens stage[STEP ? 1 : 2];
  __shared__ DeltaScalars scal[kDeltaTokens];
  const int s = blockIdx.x / col_blocks, h = blockIdx.y, tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31, l = lane & 7;
  const int b0 = (blockIdx.x % col_blocks) * COLS, x0 = (warp * 4 + (lane >> 3)) * CPT, c0 = b0 + x0;
  const bool live = c0 < p.d_v;
  const SeqRows sr = STEP ? SeqRows{s, 1} : seq_rows(p.offsets, s, static_cast<int>(p.rows));
  const int hq = h / (p.heads / p.qk_heads);
  const long st_at = (static_cast<long>(s) * p.heads + h) * p.d_k * p.d_v + c0;
  const T* qp = static_cast<const T*>(p.q) + sr.begin * p.ldq + hq * p.d_k;
  const T* kp = static_cast<const T*>(p.k) + sr.begin * p.ldk + hq * p.d_k;
  const T* vp = static_cast<const T*>(p.v) + sr.begin * p.ldv + h * p.d_v;
  const float* gp = p.g + sr.begin * p.ldg + h;
  const float* bp = p.beta + sr.begin * p.ldb + h;
  T* op = static_cast<T*>(p.out) + sr.begin * p.ldo + h * p.d_v + c0;
  auto copy = [&](int t0) {  // tokens t0 .. into their stage
    Tokens& to = stage[STEP ? 0 : (t0 / kDeltaTokens) & 1];
    constexpr int V = 16 / sizeof(T);
    const int n = min(kDeltaTokens, sr.len - t0), ck = p.d_k / V, cv = min(+COLS, p.d_v - b0) / V;
    for (int e = tid; e < n * ck; e += 128) {
      const int r = e / ck, x = (e % ck) * V;
      cp_async<16>(&to.q[r][x], qp + (t0 + r) * p.ldq + x);
      cp_async<16>(&to.k[r][x], kp + (t0 + r) * p.ldk + x);
    }
    for (int e = tid; e < n * cv; e += 128) {
      const int r = e / cv, x = (e % cv) * V;
      cp_async<16>(&to.v[r][x], vp + (t0 + r) * p.ldv + b0 + x);
    }
    if (tid < n) {
      cp_async<4>(&to.g[tid], gp + (t0 + tid) * p.ldg);
      cp_async<4>(&to.beta[tid], bp + (t0 + tid) * p.ldb);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if constexpr (!STEP) {
    if (DK > p.d_k)  // columns past d_k stay zero
      for (int e = tid; e < 2 * kDeltaTokens * DK; e += 128) {
        Tokens& to = stage[e / (kDeltaTokens * DK)];
        (&to.q[0][0])[e % (kDeltaTokens * DK)] = (&to.k[0][0])[e % (kDeltaTokens * DK)] = from_f32<T>(0.f);
      }
    __syncthreads();
    if (sr.len > 0) copy(0);
  }
  float S[RM][4][CPT] = {};
#pragma unroll
  for (int m = 0; m < RM; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * (l + 8 * m) + i;
      if (p.state_in && live && r < p.d_k) load_n<float, CPT>(p.state_in + st_at + static_cast<long>(r) * p.d_v, S[m][i]);
    }
  float logA = 0.f;  // (of the thread that finds the decays)
  float A = 1.f;
  auto settle = [&](float f) {
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < CPT; ++j) S[m][i][j] *= f;
  };
  auto sum8 = [](float v) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  auto norms = [&](float kk, float qq, float kq, DeltaScalars& x) {
    x.rk = p.qk_norm ? rsqrtf(kk + p.qk_eps) : 1.f;
    x.rq = p.scale * (p.qk_norm ? rsqrtf(qq + p.qk_eps) : 1.f);
    x.kq = kq;
  };
  auto token = [&](long t, const float (&q)[RM][4], const float (&k)[RM][4], const float (&v)[CPT], float beta,
                   const DeltaScalars& x) {
    if (x.settle != 1.f) settle(x.settle);
    A = x.A;
    float red[2 * CPT] = {};  // S^T k, S^T q
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
          red[j] = fmaf(S[m][i][j], k[m][i], red[j]);
          red[CPT + j] = fmaf(S[m][i][j], q[m][i], red[CPT + j]);
        }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1)
#pragma unroll
      for (int i = 0; i < 2 * CPT; ++i) red[i] += __shfl_xor_sync(0xffffffffu, red[i], o);
    float u[CPT], o[CPT];
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      u[j] = beta * (v[j] - A * x.rk * red[j]) * x.rk;  // (times 1/|k|: the state adds k u)
      o[j] = x.rq * fmaf(x.kq, u[j], A * red[CPT + j]);
      u[j] *= x.invA;
    }
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < CPT; ++j) S[m][i][j] = fmaf(k[m][i], u[j], S[m][i][j]);
    if (l == 0 && live) store_n<T, CPT>(op + t * p.ldo, o);
  };
  if constexpr (STEP) {
    float q[RM][4], k[RM][4], v[CPT] = {};
#pragma unroll
    for (int m = 0; m < RM; ++m) {
#pragma unroll
      for (int i = 0; i < 4; ++i) q[m][i] = k[m][i] = 0.f;
      if (4 * (l + 8 * m) < p.d_k) {
        load4(qp + 4 * l + 32 * m, q[m]);
        load4(kp + 4 * l + 32 * m, k[m]);
      }
    }
    if (live) load_n<T, CPT>(vp + c0, v);
    float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        kk = fmaf(k[m][i], k[m][i], kk);
        qq = fmaf(q[m][i], q[m][i], qq);
        kq = fmaf(k[m][i], q[m][i], kq);
      }
    DeltaScalars x;
    norms(sum8(kk), sum8(qq), sum8(kq), x);
    hold_decay(logA, gp[0], true, x);
    token(0, q, k, v, bp[0], x);
  } else {
    for (int t0 = 0; t0 < sr.len; t0 += kDeltaTokens) {
      if (t0 + kDeltaTokens < sr.len) {
        copy(t0 + kDeltaTokens);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      __syncthreads();
      const Tokens& in = stage[STEP ? 0 : (t0 / kDeltaTokens) & 1];
      const int n = min(kDeltaTokens, sr.len - t0);
      {  // 8 threads a token
        const int r = tid >> 3;
        float kk = 0.f, qq = 0.f, kq = 0.f;
        if (r < n)
          for (int x = 4 * (tid & 7); x < DK; x += 32) {
            float q[4], k[4];
            load4(&in.q[r][x], q);
            load4(&in.k[r][x], k);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              kk = fmaf(k[i], k[i], kk);
              qq = fmaf(q[i], q[i], qq);
              kq = fmaf(k[i], q[i], kq);
            }
          }
        kk = sum8(kk);
        qq = sum8(qq);
        kq = sum8(kq);
        if (r < n && (tid & 7) == 0) norms(kk, qq, kq, scal[r]);
        if (tid == 127)  // what is held back never passes the 16 tokens
          for (int i = 0; i < n; ++i) {
            hold_decay(logA, in.g[i], i == n - 1, scal[i]);
            scal[i].A = logA;
          }
        __syncthreads();
        if (tid < n) {
          const float a = scal[tid].A;
          scal[tid].A = expf(a);
          scal[tid].invA = expf(-a);
        }
        __syncthreads();
      }
      for (int r = 0; r < n; ++r) {
        float q[RM][4], k[RM][4], v[CPT];
#pragma unroll
        for (int m = 0; m < RM; ++m) {
          load4(&in.q[r][4 * l + 32 * m], q[m]);
          load4(&in.k[r][4 * l + 32 * m], k[m]);
        }
        load_n<T, CPT>(&in.v[r][x0], v);  // (of columns that are not there: whatever it is, they are never stored)
        token(t0 + r, q, k, v, in.beta[r], scal[r]);
      }
      __syncthreads();  // the stage is copied over next
    }
  }
  if (p.state_out && live) {
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * (l + 8 * m) + i;
        if (r < p.d_k) store_n<float, CPT>(p.state_out + st_at + static_cast<long>(r) * p.d_v, S[m][i]);
      }
  }
}

// One token of each of many sequences: a block brings a whole (sequence, head)
// state in with one bulk copy (it is contiguous), keeps its values in registers
// between the two passes over them and sends it back the same way. A thread has
// one column and every RS-th row. Bound by the state's bytes, read and written,
// two blocks of 64 KB an SM (the registers leave room for no third). 64 sequences
// x 32 heads of 128 x 128: 54 us, delta_recurrent_kernel 72, 16-byte copies by all
// threads in place of the bulk copy in, whose wait can give up, 60. If it does, the
// block's out is NaN and its state stays as it was: the call has no status word.
constexpr int kDeltaStepDv = 128;

template <typename T>
__global__ void __launch_bounds__(256) delta_step_kernel(const DeltaParams p) {
  pdl_wait();
  constexpr int DV = kDeltaStepDv, RS = 256 / DV, RPT = 128 / RS;  // row groups; rows a thread at most
  extern __shared__ __align__(128) uint8_t dsm[];
  float* sS = reinterpret_cast<float*>(dsm);  // [d_k][DV]
  __shared__ float sk[128], sq[128], part[8][3], red[RS][2][DV];
  __shared__ __align__(8) uint64_t full;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = tid % DV, rg = tid / DV;
  const int h = blockIdx.y, s = blockIdx.x, hq = h / (p.heads / p.qk_heads);
  const uint32_t bytes = static_cast<uint32_t>(p.d_k) * DV * 4;
  float* state = p.state_out + (static_cast<long>(s) * p.heads + h) * p.d_k * DV;
  if (tid == 0) {
    abort_flag = 0;
    mbar_init(&full, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(&full, bytes);
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(sS)),
                 "l"(state), "r"(bytes), "r"(smem_u32(&full))
                 : "memory");
  }
  float k = 0.f, q = 0.f;
  if (tid < p.d_k) {
    k = to_f32(static_cast<const T*>(p.k)[s * p.ldk + hq * p.d_k + tid]);
    q = to_f32(static_cast<const T*>(p.q)[s * p.ldq + hq * p.d_k + tid]);
  }
  const float v = to_f32(static_cast<const T*>(p.v)[s * p.ldv + h * DV + c]);
  const float a = expf(log_decay(p.g[s * p.ldg + h])), beta = p.beta[s * p.ldb + h];
  if (tid < 128) {
    sk[tid] = k;
    sq[tid] = q;
    const float kk = warp_sum(k * k), qq = warp_sum(q * q), kq = warp_sum(k * q);
    if (lane == 0) {
      part[warp][0] = kk;
      part[warp][1] = qq;
      part[warp][2] = kq;
    }
  }
  __syncthreads();
  float n[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) n[i] = (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
  const float rk = p.qk_norm ? rsqrtf(n[0] + p.qk_eps) : 1.f;
  const float rq = p.scale * (p.qk_norm ? rsqrtf(n[1] + p.qk_eps) : 1.f);
  mbar_wait(&full, 0, &abort_flag, nullptr);
  float S[RPT], r1 = 0.f, r2 = 0.f;
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = rg + RS * i;
    S[i] = r < p.d_k ? a * sS[r * DV + c] : 0.f;
    r1 = fmaf(S[i], sk[r], r1);
    r2 = fmaf(S[i], sq[r], r2);
  }
  red[rg][0][c] = r1;
  red[rg][1][c] = r2;
  __syncthreads();
  r1 = r2 = 0.f;
#pragma unroll
  for (int i = 0; i < RS; ++i) {
    r1 += red[i][0][c];
    r2 += red[i][1][c];
  }
  const bool lost = *static_cast<volatile int*>(&abort_flag) != 0;  // any thread's wait gave up (it was before the barrier)
  const float u = beta * (v - rk * r1) * rk;  // (times 1/|k|: the state adds k u)
  if (rg == 0) static_cast<T*>(p.out)[s * p.ldo + h * DV + c] = from_f32<T>(lost ? NAN : rq * fmaf(n[2], u, r2));
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = rg + RS * i;
    if (r < p.d_k) sS[r * DV + c] = fmaf(sk[r], u, S[i]);
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (lost) {
    let_copies_land();
  } else if (tid == 0) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(state), "r"(smem_u32(sS)), "r"(bytes)
                 : "memory");
    bulk_commit();
    bulk_wait_all();
  }
}

}  // namespace edit
