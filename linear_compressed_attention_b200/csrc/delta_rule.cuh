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

// Token by token, the state in registers. A warp holds 16 columns of one
// (sequence, head)'s state: lane = 8 cg + l keeps columns 4 cg .. 4 cg + 3 and
// the rows 4 (l + 8 m) .. + 3, so that a state row's 16 columns are 64
// contiguous bytes and the sums over d_k are three shuffles over 8 lanes. Both
// products with the state, S^T k and S^T q, are taken of the state before the
// token (o = e^g S^T q + (k.q) u), so that a token costs one round of shuffles.
// The state is kept as S / A with A the decay since it was last brought up to
// date (every 16 tokens, or when the log of A leaves +-8): a rounding of every
// value for the decay of every token was most of the state's error (400 fp32
// tokens: 1.1e-6 of its norm).
template <typename T, int DK>
__global__ void __launch_bounds__(128) delta_recurrent_kernel(const DeltaParams p, int col_blocks) {
  pdl_wait();
  if (p.status && blockIdx.x == 0 && blockIdx.y == 0)
    check_offsets(p.offsets, p.rows, nullptr, 0, nullptr, 0, p.nseq, p.status);
  constexpr int RM = DK / 32;
  const int s = blockIdx.x / col_blocks, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & 7;
  const int c0 = (((blockIdx.x % col_blocks) * 4 + warp) * 4 + (lane >> 3)) * 4;
  if (((blockIdx.x % col_blocks) * 4 + warp) * 16 >= p.d_v) return;  // whole warps
  const bool live = c0 < p.d_v;
  const SeqRows sr = p.offsets ? seq_rows(p.offsets, s, static_cast<int>(p.rows)) : SeqRows{s, 1};
  const int hq = h / (p.heads / p.qk_heads);
  const long st_at = (static_cast<long>(s) * p.heads + h) * p.d_k * p.d_v + c0;
  float S[RM][4][4];
#pragma unroll
  for (int m = 0; m < RM; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * (l + 8 * m) + i;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p.state_in && live && r < p.d_k)
        a = *reinterpret_cast<const float4*>(p.state_in + st_at + static_cast<long>(r) * p.d_v);
      S[m][i][0] = a.x; S[m][i][1] = a.y; S[m][i][2] = a.z; S[m][i][3] = a.w;
    }
  const T* qp = static_cast<const T*>(p.q) + sr.begin * p.ldq + hq * p.d_k + 4 * l;
  const T* kp = static_cast<const T*>(p.k) + sr.begin * p.ldk + hq * p.d_k + 4 * l;
  const T* vp = static_cast<const T*>(p.v) + sr.begin * p.ldv + h * p.d_v + c0;
  const float* gp = p.g + sr.begin * p.ldg + h;
  const float* bp = p.beta + sr.begin * p.ldb + h;
  T* op = static_cast<T*>(p.out) + sr.begin * p.ldo + h * p.d_v + c0;
  float qn[RM][4], kn[RM][4], vn[4], gn = 0.f, bn = 0.f;
  auto fetch = [&](long t) {  // token t into the registers of the next step
#pragma unroll
    for (int m = 0; m < RM; ++m) {
#pragma unroll
      for (int i = 0; i < 4; ++i) qn[m][i] = kn[m][i] = 0.f;
      if (4 * (l + 8 * m) < p.d_k) {
        load4(qp + t * p.ldq + 32 * m, qn[m]);
        load4(kp + t * p.ldk + 32 * m, kn[m]);
      }
    }
    vn[0] = vn[1] = vn[2] = vn[3] = 0.f;
    if (live) load4(vp + t * p.ldv, vn);
    gn = gp[t * p.ldg];
    bn = bp[t * p.ldb];
  };
  float logA = 0.f, A = 1.f, invA = 1.f;
  int held = 0;
  auto settle = [&](float f) {
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) S[m][i][j] *= f;
    logA = 0.f;
    A = invA = 1.f;
    held = 0;
  };
  if (sr.len > 0) fetch(0);
  for (int t = 0; t < sr.len; ++t) {
    float q[RM][4], k[RM][4], v[4];
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[m][i] = qn[m][i];
        k[m][i] = kn[m][i];
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = vn[j];
    const float beta = bn;
    logA += log_decay(gn);
    if (!(fabsf(logA) <= 8.f) || ++held == 16) {  // (a NaN settles, and stays)
      settle(expf(logA));
    } else {
      A = expf(logA);
      invA = expf(-logA);
    }
    if (t + 1 < sr.len) fetch(t + 1);
    float red[11] = {};  // S^T k (4 columns), S^T q (4), |k|^2, |q|^2, k.q
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          red[j] = fmaf(S[m][i][j], k[m][i], red[j]);
          red[4 + j] = fmaf(S[m][i][j], q[m][i], red[4 + j]);
        }
        red[8] = fmaf(k[m][i], k[m][i], red[8]);
        red[9] = fmaf(q[m][i], q[m][i], red[9]);
        red[10] = fmaf(k[m][i], q[m][i], red[10]);
      }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1)
#pragma unroll
      for (int i = 0; i < 11; ++i) red[i] += __shfl_xor_sync(0xffffffffu, red[i], o);
    float rk = 1.f, rq = p.scale;
    if (p.qk_norm) {
      rk = rsqrtf(red[8] + p.qk_eps);
      rq *= rsqrtf(red[9] + p.qk_eps);
    }
    float u[4], o4[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = beta * (v[j] - A * rk * red[j]) * rk;  // (times 1/|k|: the state adds k u)
      o4[j] = rq * fmaf(red[10], u[j], A * red[4 + j]);
      u[j] *= invA;
    }
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) S[m][i][j] = fmaf(k[m][i], u[j], S[m][i][j]);
    if (l == 0 && live) {
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2*>(op + t * p.ldo) = make_uint2(pack_bf16x2(o4[0], o4[1]), pack_bf16x2(o4[2], o4[3]));
      else
        *reinterpret_cast<float4*>(op + t * p.ldo) = make_float4(o4[0], o4[1], o4[2], o4[3]);
    }
  }
  settle(A);
  if (p.state_out && live) {
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * (l + 8 * m) + i;
        if (r < p.d_k)
          *reinterpret_cast<float4*>(p.state_out + st_at + static_cast<long>(r) * p.d_v) =
              make_float4(S[m][i][0], S[m][i][1], S[m][i][2], S[m][i][3]);
      }
  }
}

}  // namespace edit
