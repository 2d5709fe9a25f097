// Softmax attention over packed sequences (edit_packed_attention_forward):
// what all its kernels share, the CUDA-core kernel of fp32 calls, and the join
// of a key list that was split over blocks.
//
// The G = heads / kv_heads query heads that share a key/value head are packed
// into the rows of one tile, row r = (query token r / G, head r % G), so that a
// key tile is read once for all of them and a single new token still fills G
// rows. Softmax runs over the key tiles with a running maximum and sum,
// exponents in base 2.
#pragma once

#include "packed_seq.cuh"

namespace edit {

struct PackedAttnParams {
  const void *q, *k, *v;
  void* out;
  const int32_t *q_offsets, *k_offsets, *k_lens;
  long ldq, ldk, ldv, ldo;
  int rows_q, rows_k;
  int heads, kv_heads, d, nseq, causal, max_k;
  float scale;
  int slots;     // row tiles (see seq_of_slot)
  int nsplit;    // parts of a key list (1: the tile writes its rows itself)
  float* part_o;   // [nsplit][rows_q][heads][d]: unnormalised, relative to part_ml's maximum
  float2* part_ml; // [nsplit][rows_q][heads]: (maximum in base-2 units, sum); sum 0: no keys, part_o not written
  int* status;
};

struct AttnItem {
  int q0, lq;      // the sequence's query rows
  int k0, lk;      // its keys
  int tok0, ntok;  // this tile's tokens within the sequence
  int kbeg, kend;  // key range of this tile and split (kend: what its last row sees), whole tiles of KT but the last
};

// The keys of sequence s, within the rows given and max_k.
__device__ __forceinline__ SeqRows seq_keys(const PackedAttnParams& p, int s) {
  SeqRows r = seq_rows(p.k_offsets, s, p.rows_k);
  if (p.k_lens) r.len = clamp_int(p.k_lens[s], 0, r.len);
  r.len = min(r.len, p.max_k);
  return r;
}

// Work of one block: row tile `slot` of R tokens, part `split` of its keys in
// tiles of KT. Returns false for an empty slot. All 32 lanes call.
template <int KT>
__device__ __forceinline__ bool attn_item(const PackedAttnParams& p, int slot, int split, int R, AttnItem& it) {
  const int s = seq_of_slot(p.q_offsets, p.nseq, p.rows_q, R, slot);
  const SeqRows q = seq_rows(p.q_offsets, s, p.rows_q), k = seq_keys(p, s);
  const int tile = slot - (q.begin / R + s);
  if (tile < 0 || tile * static_cast<long>(R) >= q.len) return false;
  it.q0 = q.begin;
  it.lq = q.len;
  it.k0 = k.begin;
  it.lk = k.len;
  it.tok0 = tile * R;
  it.ntok = min(R, q.len - it.tok0);
  int kend = k.len;
  if (p.causal) kend = clamp_int(it.tok0 + it.ntok + k.len - q.len, 0, k.len);
  const int nt = (kend + KT - 1) / KT;
  it.kbeg = static_cast<int>(static_cast<long>(nt) * split / p.nsplit) * KT;
  it.kend = min(kend, static_cast<int>(static_cast<long>(nt) * (split + 1) / p.nsplit) * KT);
  return true;
}

// ---------------------------------------------------------------- CUDA cores
// 64 packed rows against 64 keys at a time; a thread holds 4 rows x 4 keys of
// the scores and 4 rows x DP / 16 columns of the output. K and V rows past the
// visible keys are zeros in shared memory, and a masked key skips its product, so
// that nothing behind a mask reaches a row (a key that is seen never does: a weight
// of 0 times what is not finite is NaN, whichever tile the key lies in).
template <typename T, int DP>
__global__ void __launch_bounds__(256) packed_attn_simt_kernel(const PackedAttnParams p) {
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
    check_offsets(p.q_offsets, p.rows_q, p.k_offsets, p.rows_k, p.k_lens, p.max_k, p.nseq, p.status);
  constexpr int LD = DP + 4, NC = DP / 64 > 0 ? DP / 64 : 1, CW = DP / 16 < 4 ? DP / 16 : 4;
  extern __shared__ float sm[];
  float* sq = sm;             // [64][LD]
  float* sk = sq + 64 * LD;   // [64][LD]
  float* sv = sk + 64 * LD;   // [64][DP]
  float* sp = sv + 64 * DP;   // [64 keys][68]: weights, by key
  const int G = p.heads / p.kv_heads, R = 64 / G, hk = blockIdx.y;
  AttnItem it;
  if (!attn_item<64>(p, p.slots - 1 - blockIdx.x, blockIdx.z, R, it)) return;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const float c = p.scale * 1.4426950408889634f;
  const T* qg = static_cast<const T*>(p.q) + (it.q0 + static_cast<long>(it.tok0)) * p.ldq + hk * G * p.d;
  for (int e = tid; e < 64 * (DP / 4); e += 256) {
    const int r = e / (DP / 4), x = (e % (DP / 4)) * 4;
    const int t = r / G;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < it.ntok && r < R * G && x < p.d) {
      const T* s = qg + t * p.ldq + (r % G) * p.d + x;
      a = make_float4(to_f32(s[0]), to_f32(s[1]), to_f32(s[2]), to_f32(s[3]));
    }
    *reinterpret_cast<float4*>(sq + r * LD + x) = a;
  }
  // keys a row sees: 0 .. see[i] - 1
  int see[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = it.tok0 + (4 * ty + i) / G;
    see[i] = p.causal ? clamp_int(t + 1 + it.lk - it.lq, 0, it.lk) : it.lk;
  }
  float m[4], l[4], o[4][NC][CW];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int w = 0; w < CW; ++w) o[i][j][w] = 0.f;
  }
  for (int key0 = it.kbeg; key0 < it.kend; key0 += 64) {
    const int nk = min(64, it.kend - key0);
    __syncthreads();
    const T* kg = static_cast<const T*>(p.k) + (it.k0 + static_cast<long>(key0)) * p.ldk + hk * p.d;
    const T* vg = static_cast<const T*>(p.v) + (it.k0 + static_cast<long>(key0)) * p.ldv + hk * p.d;
    for (int e = tid; e < 64 * (DP / 4); e += 256) {
      const int r = e / (DP / 4), x = (e % (DP / 4)) * 4;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
      if (r < nk && x < p.d) {
        const T *s = kg + r * p.ldk + x, *u = vg + r * p.ldv + x;
        a = make_float4(to_f32(s[0]), to_f32(s[1]), to_f32(s[2]), to_f32(s[3]));
        b = make_float4(to_f32(u[0]), to_f32(u[1]), to_f32(u[2]), to_f32(u[3]));
      }
      *reinterpret_cast<float4*>(sk + r * LD + x) = a;
      *reinterpret_cast<float4*>(sv + r * DP + x) = b;
    }
    __syncthreads();
    float s[4][4] = {};
#pragma unroll 4
    for (int x = 0; x < DP; x += 4) {
      float4 qv[4], kv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4*>(sq + (4 * ty + i) * LD + x);
#pragma unroll
      for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * LD + x);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = fmaf(qv[i].x, kv[j].x,
                         fmaf(qv[i].y, kv[j].y, fmaf(qv[i].z, kv[j].z, fmaf(qv[i].w, kv[j].w, s[i][j]))));
    }
    bool masked = nk < 64;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = see[i] - key0;  // visible keys of this tile
      masked |= n < 64;
      float mt = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (tx + 16 * j < n) mt = fmaxf(mt, s[i][j] * c);
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, w));
      const float mn = fmaxf(m[i], mt), base = mn == -INFINITY ? 0.f : mn;
      const float alpha = exp2f(m[i] - base);
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = tx + 16 * j < n ? exp2f(s[i][j] * c - base) : 0.f;
        sum += e;
        sp[(tx + 16 * j) * 68 + 4 * ty + i] = e;
      }
      l[i] = fmaf(l[i], alpha, sum);  // (this thread's keys; summed over the row at the end)
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int w = 0; w < CW; ++w) o[i][j][w] *= alpha;
    }
    masked = __syncthreads_or(masked);
    int n[4];  // visible keys of this tile
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i] = see[i] - key0;
    auto accumulate = [&](auto skip) {
#pragma unroll 4
      for (int key = 0; key < nk; ++key) {
        const float4 pv = *reinterpret_cast<const float4*>(sp + key * 68 + 4 * ty);
        const float pr[4] = {pv.x, pv.y, pv.z, pv.w};
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int w = 0; w < CW; ++w) {
            const float x = sv[key * DP + 64 * j + tx * CW + w];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!decltype(skip)::value || key < n[i]) o[i][j][w] = fmaf(pr[i], x, o[i][j][w]);
          }
      }
    };
    if (masked)
      accumulate(std::true_type{});
    else
      accumulate(std::false_type{});
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float sum = l[i];
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    const int r = 4 * ty + i, t = r / G;
    if (r >= R * G || t >= it.ntok) continue;
    const long row = it.q0 + static_cast<long>(it.tok0) + t;
    const int h = hk * G + r % G;
    const float inv = p.nsplit > 1 ? 1.f : (sum > 0.f || sum != sum ? 1.f / sum : 0.f);
    const long at = (blockIdx.z * static_cast<long>(p.rows_q) + row) * p.heads + h;
    if (p.nsplit > 1 && tx == 0) p.part_ml[at] = make_float2(m[i], sum);
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int w = 0; w < CW; ++w) {
        const int x = 64 * j + tx * CW + w;
        if (x >= p.d) continue;
        if (p.nsplit > 1)
          p.part_o[at * p.d + x] = o[i][j][w];
        else
          static_cast<T*>(p.out)[row * p.ldo + h * p.d + x] = from_f32<T>(o[i][j][w] * inv);
      }
  }
}

// Joins the parts of split key lists, in the order of the parts: one warp for
// each (row, head). Rows in no sequence stay as they are.
template <typename T>
__global__ void __launch_bounds__(128) packed_attn_join_kernel(const PackedAttnParams p) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long item = static_cast<long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (item >= static_cast<long>(p.rows_q) * p.heads) return;
  const long row = item / p.heads;
  const int h = static_cast<int>(item % p.heads);
  if (row < p.q_offsets[0] || row >= p.q_offsets[p.nseq]) return;
  const long step = static_cast<long>(p.rows_q) * p.heads;
  float m = -INFINITY;
  for (int s = lane; s < p.nsplit; s += 32) {
    const float2 ml = p.part_ml[s * step + item];
    if (ml.y != 0.f) m = fmaxf(m, ml.x);
  }
  m = warp_max(m);
  if (m == -INFINITY) m = 0.f;
  float l = 0.f, o[4] = {};
  for (int s = 0; s < p.nsplit; ++s) {
    const float2 ml = p.part_ml[s * step + item];
    if (ml.y == 0.f) continue;
    const float w = exp2f(ml.x - m);
    l = fmaf(w, ml.y, l);
    if (4 * lane < p.d) {
      const float4 a = *reinterpret_cast<const float4*>(p.part_o + (s * step + item) * p.d + 4 * lane);
      o[0] = fmaf(w, a.x, o[0]);
      o[1] = fmaf(w, a.y, o[1]);
      o[2] = fmaf(w, a.z, o[2]);
      o[3] = fmaf(w, a.w, o[3]);
    }
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  if (4 * lane < p.d) {
    T* out = static_cast<T*>(p.out) + row * p.ldo + h * p.d + 4 * lane;
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    else
      *reinterpret_cast<float4*>(out) = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
  }
}

}  // namespace edit
