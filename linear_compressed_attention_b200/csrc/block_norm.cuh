// The step between two branches of a block (edit_block_norm_forward), one pass
// over the rows:
//   r = x + rho act(gate) N_post(y),  h = N_pre(r) (1 + scale) + shift
// The row stays in registers between the reads of x, y and the writes of r, h,
// so that both norms cost no memory traffic: 4 C values a row, which bounds it
// (65536 rows of 1152 bf16 are 604 MB, 92 us at the copy rate; it takes 108).
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

// 8 consecutive values, as loaded (16-byte accesses) or one (any alignment).
template <typename T, int VEC>
struct BnRaw {
  static constexpr int W = VEC == 8 ? 8 * sizeof(T) / 4 : 1;
  uint32_t w[W];
};
// STREAM: read once, not kept in L1 (which holds the samples' vectors).
template <bool STREAM, typename T, int VEC>
__device__ __forceinline__ BnRaw<T, VEC> bn_load(const T* p) {
  BnRaw<T, VEC> r;
  if constexpr (VEC == 8) {
#pragma unroll
    for (int i = 0; i < BnRaw<T, VEC>::W; i += 4) {
      const uint4* q = reinterpret_cast<const uint4*>(p) + i / 4;
      const uint4 u = STREAM ? __ldcs(q) : *q;
      r.w[i] = u.x; r.w[i + 1] = u.y; r.w[i + 2] = u.z; r.w[i + 3] = u.w;
    }
  } else if constexpr (sizeof(T) == 2) {
    r.w[0] = *reinterpret_cast<const uint16_t*>(p);
  } else {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
  return r;
}
template <typename T, int VEC>
__device__ __forceinline__ float bn_get(const BnRaw<T, VEC>& r, int i) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(r.w[i]);
  if constexpr (VEC == 1) return __uint_as_float(r.w[0] << 16);
  return __uint_as_float(i & 1 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
}
template <int VEC, typename T>
__device__ __forceinline__ void bn_store(T* p, const float (&o)[VEC]) {
  if constexpr (VEC == 8 && sizeof(T) == 2) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]),
                                                   pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])));
  } else if constexpr (VEC == 8) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(o[0], o[1], o[2], o[3]));
    __stcs(reinterpret_cast<float4*>(p + 4), make_float4(o[4], o[5], o[6], o[7]));
  } else {
    *p = from_f32<T>(o[0]);
  }
}

// Sum over the TPR threads of a row: a warp, or TPR / 32 warps of the block,
// which meet at a barrier of their own (another row's threads may be gone).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = warp_sum(v);
  if constexpr (TPR > 32) {
    const int group = threadIdx.x / TPR;
    float* mine = part + group * (TPR / 32);
    named_bar_sync(1 + group, TPR);  // (the last sum has been read)
    if ((threadIdx.x & 31) == 0) mine[(threadIdx.x % TPR) >> 5] = v;
    named_bar_sync(1 + group, TPR);
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += mine[i];
  }
  return v;
}

// z = N(z) w + b over the row held as NV vectors a thread (vectors past C are 0).
template <typename T, int VEC, int TPR, int NV>
__device__ __forceinline__ void bn_norm(float (&z)[NV][VEC], int kind, float eps, int C, int nv, int t,
                                        const T* w, const T* b, float* part) {
  if (kind == EDIT_NORM_NONE) return;
  const float inv = 1.f / static_cast<float>(C);
  float mean = 0.f;
  if (kind == EDIT_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) s += z[k][i];
    mean = row_sum<TPR>(s, part) * inv;
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
  const float rstd = 1.f / sqrtf(row_sum<TPR>(s2, part) * inv + eps);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int vi = t + TPR * k;
    if (vi < nv) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) z[k][i] *= rstd;
      if (w) {
        const auto wv = bn_load<false, T, VEC>(w + VEC * vi);
#pragma unroll
        for (int i = 0; i < VEC; ++i) z[k][i] *= bn_get(wv, i);
      }
      if (b) {
        const auto bv = bn_load<false, T, VEC>(b + VEC * vi);
#pragma unroll
        for (int i = 0; i < VEC; ++i) z[k][i] += bn_get(bv, i);
      }
    }
  }
}

// The sample's vector plus the common one (0 where missing).
template <typename T, int VEC>
__device__ __forceinline__ void bn_mod(const T* common, const T* own, int at, float (&o)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) o[i] = 0.f;
  if (common) {
    const auto a = bn_load<false, T, VEC>(common + at);
#pragma unroll
    for (int i = 0; i < VEC; ++i) o[i] = bn_get(a, i);
  }
  if (own) {
    const auto a = bn_load<false, T, VEC>(own + at);
#pragma unroll
    for (int i = 0; i < VEC; ++i) o[i] += bn_get(a, i);
  }
}

// Rows of up to kBnNarrow values: a block takes rows_per_block consecutive rows
// and, for each sample among them, first folds everything that is the same for the
// sample's rows into fp32 vectors in shared memory,
//   r = x + n_y a + b,  h = n_r c + d  (n_y, n_r the bare norms)
//   a = rho act(gate) post_w, b = rho act(gate) post_b, c = pre_w (1 + scale), d = pre_b (1 + scale) + shift,
// so that a value costs some 20 instructions whatever is given (with the vectors
// read and combined for every row it was 50, and the instructions, not the memory,
// bounded it: 184 us for 65536 rows of 1152 bf16).
constexpr int kBnNarrow = 2048;

template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(256, 3) block_norm_rows_kernel(const BlockNormParams p, int rows_per_block) {
  pdl_wait();
  constexpr int RPB = 256 / TPR;
  // a, b, c, d: C values each (rounded up to 4); with VEC 8 the first four of every eight, then the last four, so
  // that a warp's 16-byte reads are contiguous
  extern __shared__ __align__(16) float bn_vec[];
  __shared__ float part[256 / 32];
  const int C = p.C, nv = C / VEC, Cp = (C + 3) & ~3, t = threadIdx.x % TPR, mine = threadIdx.x / TPR;
  float *va = bn_vec, *vb = va + Cp, *vc = vb + Cp, *vd = vc + Cp;
  const long first = static_cast<long>(blockIdx.x) * rows_per_block;
  const long last = min(first + rows_per_block, p.rows);
  long at = first;
  int b = 0;
  if (p.offsets) {  // last sample that begins at or before the first row
    int n = p.samples;
    while (n > 1) {
      const int half = n / 2;
      if (p.offsets[b + half] <= first) {
        b += half;
        n -= half;
      } else {
        n = half;
      }
    }
  } else {
    b = static_cast<int>(first / p.rows_per_sample);
  }
  for (; at < last && b < p.samples; ++b) {
    // the rows of sample b among this block's (offsets that run backwards give none)
    const long s0 = p.offsets ? p.offsets[b] : b * p.rows_per_sample;
    const long s1 = p.offsets ? p.offsets[b + 1] : s0 + p.rows_per_sample;
    const long r0 = max(at, s0), r1 = min(last, s1);
    if (r1 <= r0) continue;
    at = r1;
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += 256) {
      auto get = [&](const void* v, long i) { return to_f32(static_cast<const T*>(v)[i]); };
      const long m = b * p.ld_mod + c;
      float g = p.rho;
      if (p.gate || p.gate0) {
        g = (p.gate0 ? get(p.gate0, c) : 0.f) + (p.gate ? get(p.gate, m) : 0.f);
        g = p.rho * (p.act == EDIT_GATE_TANH ? tanhf(g) : g);
      }
      const float sc = 1.f + ((p.scale0 ? get(p.scale0, c) : 0.f) + (p.scale ? get(p.scale, m) : 0.f));
      const float sh = (p.shift0 ? get(p.shift0, c) : 0.f) + (p.shift ? get(p.shift, m) : 0.f);
      const int to = VEC == 8 ? (c & 4 ? C / 2 : 0) + (c >> 3) * 4 + (c & 3) : c;
      va[to] = p.post_w ? g * get(p.post_w, c) : g;
      vb[to] = p.post_b ? g * get(p.post_b, c) : 0.f;
      vc[to] = p.pre_w ? sc * get(p.pre_w, c) : sc;
      vd[to] = p.pre_b ? fmaf(sc, get(p.pre_b, c), sh) : sh;
    }
    __syncthreads();
    auto vec = [&](const float* v, int vi, float (&o)[VEC]) {
      if constexpr (VEC == 8) {
        const float4 u = *reinterpret_cast<const float4*>(v + 4 * vi);
        const float4 w = *reinterpret_cast<const float4*>(v + C / 2 + 4 * vi);
        o[0] = u.x; o[1] = u.y; o[2] = u.z; o[3] = u.w; o[4] = w.x; o[5] = w.y; o[6] = w.z; o[7] = w.w;
      } else {
        o[0] = v[vi];
      }
    };
    // the bare norm's factor; z becomes z - mean
    auto norm = [&](float (&z)[NV][VEC], int kind) {
      if (kind == EDIT_NORM_NONE) return 1.f;
      const float inv = 1.f / static_cast<float>(C);
      if (kind == EDIT_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < VEC; ++i) s += z[k][i];
        const float mean = row_sum<TPR>(s, part) * inv;
#pragma unroll
        for (int k = 0; k < NV; ++k)
          if (t + TPR * k < nv) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) z[k][i] -= mean;
          }
      }
      float s2 = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) s2 = fmaf(z[k][i], z[k][i], s2);
      return 1.f / sqrtf(row_sum<TPR>(s2, part) * inv + p.eps);
    };
    for (long row = r0 + mine; row < r1; row += RPB) {
      BnRaw<T, VEC> xr[NV] = {}, yr[NV] = {};
      const T* x = static_cast<const T*>(p.x) + row * p.ldx;
      const T* y = p.y ? static_cast<const T*>(p.y) + row * p.ldy : nullptr;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int vi = t + TPR * k;
        if (vi < nv) {
          if (y) yr[k] = bn_load<true, T, VEC>(y + VEC * vi);
          xr[k] = bn_load<true, T, VEC>(x + VEC * vi);
        }
      }
      float z[NV][VEC];
      if (y) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < VEC; ++i) z[k][i] = bn_get(yr[k], i);
        const float f = norm(z, p.post);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int vi = t + TPR * k;
          if (vi < nv) {
            float a[VEC];
            vec(va, vi, a);
#pragma unroll
            for (int i = 0; i < VEC; ++i) z[k][i] = fmaf(z[k][i] * f, a[i], bn_get(xr[k], i));
            if (p.post_b) {
              vec(vb, vi, a);
#pragma unroll
              for (int i = 0; i < VEC; ++i) z[k][i] += a[i];
            }
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < VEC; ++i) z[k][i] = bn_get(xr[k], i);
      }
      if (p.r) {
        T* r = static_cast<T*>(p.r) + row * p.ldr;
#pragma unroll
        for (int k = 0; k < NV; ++k)
          if (t + TPR * k < nv) bn_store<VEC>(r + VEC * (t + TPR * k), z[k]);
      }
      if (!p.h) continue;
      const float f = norm(z, p.pre);
      T* h = static_cast<T*>(p.h) + row * p.ldh;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int vi = t + TPR * k;
        if (vi < nv) {
          float c[VEC], d[VEC];
          vec(vc, vi, c);
          vec(vd, vi, d);
#pragma unroll
          for (int i = 0; i < VEC; ++i) z[k][i] = fmaf(z[k][i] * f, c[i], d[i]);
          bn_store<VEC>(h + VEC * vi, z[k]);
        }
      }
    }
  }
}

// Wider rows: TPR threads a row, NV vectors of VEC values a thread (C <= TPR *
// NV * VEC), the samples' vectors read for every row.
template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(256) block_norm_kernel(const BlockNormParams p) {
  pdl_wait();
  constexpr int RPB = 256 / TPR;  // rows a block
  __shared__ float part[256 / 32];
  const int t = threadIdx.x % TPR;
  const long row = static_cast<long>(blockIdx.x) * RPB + threadIdx.x / TPR;
  if (row >= p.rows) return;  // (all threads of the row)
  const int C = p.C, nv = C / VEC;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* y = p.y ? static_cast<const T*>(p.y) + row * p.ldy : nullptr;
  BnRaw<T, VEC> xr[NV] = {}, yr[NV] = {};
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int vi = t + TPR * k;
    if (vi < nv) {
      xr[k] = bn_load<true, T, VEC>(x + VEC * vi);
      if (y) yr[k] = bn_load<true, T, VEC>(y + VEC * vi);
    }
  }
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
  const long mod = b * p.ld_mod;
  auto own = [&](const void* v) { return v ? static_cast<const T*>(v) + mod : nullptr; };
  float z[NV][VEC];
  if (y) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) z[k][i] = bn_get(yr[k], i);
    bn_norm<T, VEC, TPR, NV>(z, p.post, p.eps, C, nv, t, static_cast<const T*>(p.post_w),
                             static_cast<const T*>(p.post_b), part);
    const T *gate = own(p.gate), *gate0 = static_cast<const T*>(p.gate0);
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
        for (int i = 0; i < VEC; ++i) z[k][i] = fmaf(gated ? p.rho * g[i] : p.rho, z[k][i], bn_get(xr[k], i));
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i) z[k][i] = bn_get(xr[k], i);
  }
  if (p.r) {
    T* r = static_cast<T*>(p.r) + row * p.ldr;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (t + TPR * k < nv) bn_store<VEC>(r + VEC * (t + TPR * k), z[k]);
  }
  if (!p.h) return;
  bn_norm<T, VEC, TPR, NV>(z, p.pre, p.eps, C, nv, t, static_cast<const T*>(p.pre_w),
                           static_cast<const T*>(p.pre_b), part);
  T* h = static_cast<T*>(p.h) + row * p.ldh;
  const T *scale = own(p.scale), *shift = own(p.shift);
  const T *scale0 = static_cast<const T*>(p.scale0), *shift0 = static_cast<const T*>(p.shift0);
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
