// The step between two branches of a block (edit_block_norm_forward), one pass
// over the rows:
//   r = x + rho act(gate) N_post(y),  h = N_pre(r) (1 + scale) + shift
// The row stays in registers between the reads of x, y and the writes of r, h,
// so that both norms cost no memory traffic: 4 C values a row, which bounds it
// (65536 rows of 1152 bf16 are 604 MB, 92 us at the copy rate).
#pragma once

#include "packed_seq.cuh"

namespace edit {

struct BlockNormParams {
  const void *x, *y;
  void *r, *h;
  const void *post_w, *post_b, *pre_w, *pre_b;
  const void *gate0, *scale0, *shift0, *gate, *scale, *shift;
  const int32_t* offsets;
  long rows, rows_per_sample, ldx, ldy, ldr, ldh, ld_mod;
  int C, samples, post, pre, act;
  float eps, rho;
};

// VEC consecutive values as fp32 (VEC 8: 16-byte accesses; VEC 1: any alignment).
template <int VEC, typename T>
__device__ __forceinline__ void bn_load(const T* p, float (&o)[VEC]) {
  if constexpr (VEC == 8 && sizeof(T) == 2) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float(w[i] << 16);
      o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else if constexpr (VEC == 8) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w; o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
  } else {
    o[0] = to_f32(*p);
  }
}

template <int VEC, typename T>
__device__ __forceinline__ void bn_store(T* p, const float (&o)[VEC]) {
  if constexpr (VEC == 8 && sizeof(T) == 2) {
    uint4 u;
    u.x = pack_bf16x2(o[0], o[1]);
    u.y = pack_bf16x2(o[2], o[3]);
    u.z = pack_bf16x2(o[4], o[5]);
    u.w = pack_bf16x2(o[6], o[7]);
    *reinterpret_cast<uint4*>(p) = u;
  } else if constexpr (VEC == 8) {
    *reinterpret_cast<float4*>(p) = make_float4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(o[4], o[5], o[6], o[7]);
  } else {
    *p = from_f32<T>(o[0]);
  }
}

// Sum over the TPR threads of a row (a warp, or a block of TPR threads).
template <int TPR>
__device__ __forceinline__ float row_sum(float v) {
  v = warp_sum(v);
  if constexpr (TPR > 32) {
    __shared__ float part[TPR / 32];
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += part[i];
  }
  return v;
}

// z = N(z) w + b over the row held as NV vectors a thread (vectors past C are 0).
template <typename T, int VEC, int TPR, int NV>
__device__ __forceinline__ void bn_norm(float (&z)[NV][VEC], int kind, float eps, int C, int nv, int t,
                                        const T* w, const T* b) {
  if (kind == EDIT_NORM_NONE) return;
  const float inv = 1.f / static_cast<float>(C);
  float mean = 0.f;
  if (kind == EDIT_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) s += z[k][i];
    mean = row_sum<TPR>(s) * inv;
  }
  float s2 = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (t + TPR * k < nv) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        z[k][i] -= mean;
        s2 = fmaf(z[k][i], z[k][i], s2);
      }
    }
  const float rstd = 1.f / sqrtf(row_sum<TPR>(s2) * inv + eps);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int vi = t + TPR * k;
    if (vi < nv) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) z[k][i] *= rstd;
      if (w) {
        float wv[VEC];
        bn_load<VEC>(w + VEC * vi, wv);
#pragma unroll
        for (int i = 0; i < VEC; ++i) z[k][i] *= wv[i];
      }
      if (b) {
        float bv[VEC];
        bn_load<VEC>(b + VEC * vi, bv);
#pragma unroll
        for (int i = 0; i < VEC; ++i) z[k][i] += bv[i];
      }
    }
  }
}

// The sample's vector plus the common one (0 where missing).
template <typename T, int VEC>
__device__ __forceinline__ void bn_mod(const T* common, const T* own, int at, float (&o)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) o[i] = 0.f;
  if (common) bn_load<VEC>(common + at, o);
  if (own) {
    float a[VEC];
    bn_load<VEC>(own + at, a);
#pragma unroll
    for (int i = 0; i < VEC; ++i) o[i] += a[i];
  }
}

// TPR threads a row, NV vectors of VEC values a thread (C <= TPR * NV * VEC).
template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(256) block_norm_kernel(const BlockNormParams p) {
  pdl_wait();
  constexpr int RPB = 256 / TPR;  // rows a block
  const int t = threadIdx.x % TPR;
  const long row = static_cast<long>(blockIdx.x) * RPB + threadIdx.x / TPR;
  if (row >= p.rows) return;  // (whole warps; whole blocks where TPR is the block)
  long b = 0;
  if (p.offsets) {  // last sample that begins at or before the row
    int lo = 0, n = p.samples;
    while (n > 1) {
      const int half = n / 2;
      if (p.offsets[lo + half] <= row) {
        lo += half;
        n -= half;
      } else {
        n = half;
      }
    }
    if (row < p.offsets[lo] || row >= p.offsets[lo + 1]) return;
    b = lo;
  } else if (p.rows_per_sample > 0) {
    b = row / p.rows_per_sample;
  }
  const int C = p.C, nv = C / VEC;
  const long mod = b * p.ld_mod;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* y = p.y ? static_cast<const T*>(p.y) + row * p.ldy : nullptr;
  auto own = [&](const void* v) { return v ? static_cast<const T*>(v) + mod : nullptr; };
  const T *gate = own(p.gate), *scale = own(p.scale), *shift = own(p.shift);
  const T *gate0 = static_cast<const T*>(p.gate0), *scale0 = static_cast<const T*>(p.scale0),
          *shift0 = static_cast<const T*>(p.shift0);
  float xv[NV][VEC], z[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int vi = t + TPR * k;
#pragma unroll
    for (int i = 0; i < VEC; ++i) xv[k][i] = z[k][i] = 0.f;
    if (vi < nv) {
      bn_load<VEC>(x + VEC * vi, xv[k]);
      if (y) bn_load<VEC>(y + VEC * vi, z[k]);
    }
  }
  if (y) {
    bn_norm<T, VEC, TPR, NV>(z, p.post, p.eps, C, nv, t, static_cast<const T*>(p.post_w),
                             static_cast<const T*>(p.post_b));
    const bool gated = gate || gate0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int vi = t + TPR * k;
      if (vi < nv) {
        float g[VEC];
        if (gated) {
          bn_mod<T, VEC>(gate0, gate, VEC * vi, g);
          if (p.act == EDIT_GATE_TANH) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) g[i] = tanhf(g[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) z[k][i] = fmaf(gated ? p.rho * g[i] : p.rho, z[k][i], xv[k][i]);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) z[k][i] = xv[k][i];
  }
  if (p.r) {
    T* r = static_cast<T*>(p.r) + row * p.ldr;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (t + TPR * k < nv) bn_store<VEC>(r + VEC * (t + TPR * k), z[k]);
  }
  if (!p.h) return;
  bn_norm<T, VEC, TPR, NV>(z, p.pre, p.eps, C, nv, t, static_cast<const T*>(p.pre_w),
                           static_cast<const T*>(p.pre_b));
  T* h = static_cast<T*>(p.h) + row * p.ldh;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int vi = t + TPR * k;
    if (vi < nv) {
      float sc[VEC], sh[VEC];
      bn_mod<T, VEC>(scale0, scale, VEC * vi, sc);
      bn_mod<T, VEC>(shift0, shift, VEC * vi, sh);
#pragma unroll
      for (int i = 0; i < VEC; ++i) z[k][i] = fmaf(z[k][i], 1.f + sc[i], sh[i]);
      bn_store<VEC>(h + VEC * vi, z[k]);
    }
  }
}

}  // namespace edit
