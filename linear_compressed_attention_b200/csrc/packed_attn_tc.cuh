// Packed softmax attention on the 5th-generation tensor cores (bf16 calls of
// edit_packed_attention_forward).
//
// A block takes one or two row tiles of 128 packed rows (NQ; see
// packed_attn.cuh for the packing) of one key/value head and streams the keys
// in tiles of 128. With two row tiles each K and V tile read into shared memory
// serves 256 rows, and while the softmax of one row tile runs, the tensor
// cores work for the other.
//   warps 0-3, 4-7  softmax of row tile 0, 1: one thread a row (its TMEM lane).
//   then            one warp each: TMA producer, MMA issuer, V guard, idle.
// S = Q K^T (128 x 128 fp32) is read from TMEM into registers, P = 2^(c S - m)
// is rounded to bf16 (half a step, 2^-8 of a weight: the product with V takes
// bf16) and written back over S, and O += P V takes P from TMEM and V from
// shared memory as it was loaded (MN-major operand, no transposed copy). The row
// sum uses the unrounded weights.
// Running maximum: O and the sum are only rescaled when a row's maximum has
// grown by more than 2^8 since the last rescale (weights stay below 2^8, and a
// weight's bf16 error is relative); the wait for the product before it and the
// pass over O are then rare.
// V guard: in tiles with masked keys the rows behind the last visible key are
// cleared in shared memory (0 times what a cache holds there could be NaN), and
// among the keys that only some rows see, values that are not finite are
// cleared and added at the end to the rows that do see them.
#pragma once

#include "packed_attn.cuh"
#include "sdpa_tc.cuh"

namespace edit {

template <int DP, int NQ>
struct AttnTcCfg {
  static_assert(DP == 64 || DP == 80 || DP == 128, "padded head width");
  static constexpr int NBX = DP > 64 ? 2 : 1;       // 64-column boxes of a row
  static constexpr int BOX = 128 * 128;             // 128 rows x 128 bytes
  static constexpr int TILE = NBX * BOX;            // one Q, K or V tile
  static constexpr int SLOTS = NQ == 1 ? (DP == 64 ? 4 : 2) : (DP == 64 ? 8 : 5);  // ring of K and V tiles
  static constexpr int V_PERIOD = SLOTS % 2 ? SLOTS : SLOTS / 2;  // key tiles between two uses of a slot for V
  static constexpr int BARS = NQ * 4 + 4 * SLOTS;
  static constexpr int SMEM = 1024 + (NQ + SLOTS) * TILE + BARS * 8 + 16 + 96;
  static_assert(SMEM * (NQ == 1 ? 2 : 1) + (NQ == 1 ? 2048 : 0) <= 232448 + 1024, "shared memory");
  // two row tiles: launched with 168 registers a thread, 200 for the softmax warps and 104 for the others (256 x 200 +
  // 128 x 104 = 384 x 168)
  static constexpr int THREADS = NQ * 128 + 128;
  static constexpr int TMEM = NQ * 256;             // S of tile i at 128 i, O behind them
  static constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 128);
  static constexpr uint32_t IDESC_O = idesc_bf16_f32(128, DP) | IDESC_B_MN;
};

template <int NQ>
struct AttnBlock {
  bool some;        // the slot has rows
  AttnItem it;
  int tiles[NQ];    // key tiles of each row tile
  int most;         // the most of them
  int all_see;      // keys that every row sees: 0 .. all_see - 1; V tiles reaching beyond have masked keys
  int clean;        // key tiles before the first of those
};

template <int R>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// mbar_wait / warp_wait without a function call: ptxas allocates no registers
// beyond a call in a kernel that moves registers between its warps.
__device__ __forceinline__ bool attn_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > EDIT_WAIT_TIMEOUT_NS) {
      *abort_flag = 1;
      record_status(status, EDIT_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool attn_warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  return __all_sync(0xffffffffu, attn_wait(bar, parity, abort_flag, status));  // (every lane polls)
}

template <int DP, int NQ>
__global__ void __launch_bounds__(NQ * 128 + 128, NQ == 1 ? 2 : 1)
    packed_attn_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                          const __grid_constant__ CUtensorMap mv, const PackedAttnParams p) {
  using Cfg = AttnTcCfg<DP, NQ>;
  constexpr int NBX = Cfg::NBX, BOX = Cfg::BOX, TILE = Cfg::TILE, SLOTS = Cfg::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sQ = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sKV = sQ + NQ * TILE;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sKV + SLOTS * TILE);  // [NQ]
  uint64_t* s_full = q_full + NQ;    // [NQ] scores of a key tile
  uint64_t* p_full = s_full + NQ;    // [NQ] weights of a key tile
  uint64_t* o_full = p_full + NQ;    // [NQ] O includes a key tile
  uint64_t* kv_full = o_full + NQ;   // [SLOTS]
  uint64_t* kv_empty = kv_full + SLOTS;
  uint64_t* v_ok = kv_empty + SLOTS;  // [SLOTS] V tile with masked keys made safe
  uint64_t* v_load = v_ok + SLOTS;    // [SLOTS] such a tile's load has been issued
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(v_load + SLOTS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* odd_values = abort_flag + 1;  // the guard cleared values that are not finite
  AttnBlock<NQ>* work = reinterpret_cast<AttnBlock<NQ>*>(tmem_slot + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int W_TMA = NQ * 4, W_MMA = W_TMA + 1, W_GUARD = W_TMA + 2;
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
    check_offsets(p.q_offsets, p.rows_q, p.k_offsets, p.rows_k, p.k_lens, p.max_k, p.nseq, p.status);
  // the block's work, found by one warp; every warp takes what it needs from shared memory after the roles part
  // (held in registers across them, it costs the softmax warps theirs)
  if (warp == 0) {
    const int G = p.heads / p.kv_heads, R = 128 / G;  // R tokens a row tile
    AttnBlock<NQ> w;
    w.some = attn_item<128>(p, p.slots - 1 - blockIdx.x, blockIdx.z, NQ * R, w.it);
    w.most = 0;
    if (w.some) {
      // key tiles of each row tile: those its last row sees (within this split)
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int n = min(w.it.ntok - i * R, R);  // tokens
        int kend = w.it.kend;
        if (p.causal) kend = min(kend, w.it.tok0 + i * R + n + w.it.lk - w.it.lq);
        w.tiles[i] = n > 0 && kend > w.it.kbeg ? (kend - w.it.kbeg + 127) / 128 : 0;
        w.most = max(w.most, w.tiles[i]);
      }
      w.all_see = min(w.it.kend, p.causal ? clamp_int(w.it.tok0 + 1 + w.it.lk - w.it.lq, 0, w.it.lk) : w.it.lk);
      w.clean = max(0, min(w.most, (w.all_see - w.it.kbeg) / 128));
    }
    if (lane == 0) *work = w;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);  // one arrival a softmax warp
      mbar_init(&o_full[i], 1);
    }
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
      mbar_init(&v_ok[s], 1);
      mbar_init(&v_load[s], 1);
    }
    *abort_flag = 0;
    *odd_values = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (!work->some) return;
  if (warp == W_MMA) tmem_alloc(tmem_slot, Cfg::TMEM);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp >= W_TMA) {
    if constexpr (NQ == 2) regs_dec<104>();
    if (warp == W_TMA && lane == 0) {
      // ---------------------------------------------------------- producer: Q, then K_0 V_0 K_1 V_1 ...
      const AttnItem it = work->it;
      const int most = work->most, clean = work->clean, hk = blockIdx.y;
      const int G = p.heads / p.kv_heads, R = 128 / G;
      bool ok = true;
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        if (work->tiles[i] == 0) continue;
        mbar_arrive_expect_tx(&q_full[i], NBX * R * G * 128);
#pragma unroll
        for (int b = 0; b < NBX; ++b)
          tma_load_4d(&mq, &q_full[i], sQ + i * TILE + b * BOX, 64 * b, 0, hk, it.q0 + it.tok0 + i * R);
      }
      for (int t = 0; t < 2 * most && ok; ++t) {
        const int s = t % SLOTS;
        if (!attn_wait(&kv_empty[s], ((t / SLOTS) & 1) ^ 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&kv_full[s], TILE);
#pragma unroll
        for (int b = 0; b < NBX; ++b)
          tma_load_3d(t & 1 ? &mv : &mk, &kv_full[s], sKV + s * TILE + b * BOX, 64 * b, hk,
                      it.k0 + it.kbeg + (t >> 1) * 128);
        if ((t & 1) && (t >> 1) >= clean) mbar_arrive(&v_load[s]);
      }
      if (*abort_flag) {  // let copies already issued land before the block exits
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
      }
    } else if (warp == W_MMA && lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t tmem = *tmem_slot;
      const int most = work->most, clean = work->clean;
      int tiles[NQ];
#pragma unroll
      for (int i = 0; i < NQ; ++i) tiles[i] = work->tiles[i];
      auto wait = [&](uint64_t* bar, uint32_t parity) { return attn_wait(bar, parity, abort_flag, p.status); };
      auto scores = [&](int i, int t) {  // S_i = Q_i K_t^T
        const uint64_t qd = sdesc_kmajor_sw128(smem_u32(sQ + i * TILE));
        const uint64_t kd = sdesc_kmajor_sw128(smem_u32(sKV + ((2 * t) % SLOTS) * TILE));
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint64_t step = ((k >> 2) * BOX + (k & 3) * 32) >> 4;
          umma_bf16(tmem + 128 * i, qd + step, kd + step, Cfg::IDESC_S, k > 0 ? 1u : 0u);
        }
        umma_commit(&s_full[i]);
      };
      auto weigh = [&](int i, int t) {  // O_i += P_i V_t
        const uint64_t vd = sdesc_mnmajor_sw128(smem_u32(sKV + ((2 * t + 1) % SLOTS) * TILE), BOX);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_bf16_ts(tmem + NQ * 128 + DP * i, tmem + 128 * i + 8 * k, vd + (2048 >> 4) * k, Cfg::IDESC_O,
                       (t > 0 || k > 0) ? 1u : 0u);
        umma_commit(&o_full[i]);
      };
      bool ok = true;
      for (int i = 0; i < NQ && ok; ++i) {
        if (tiles[i] == 0) continue;
        ok = wait(&q_full[i], 0) && wait(&kv_full[0], 0);
        if (!ok) break;
        tc_fence_after();
        scores(i, 0);
      }
      if (most > 0 && ok) umma_commit(&kv_empty[0]);
      for (int t = 0; t < most && ok; ++t) {
        const int vs = (2 * t + 1) % SLOTS, ks = (2 * t + 2) % SLOTS;
        ok = wait(&kv_full[vs], ((2 * t + 1) / SLOTS) & 1);
        if (ok && t >= clean) ok = wait(&v_ok[vs], ((t - clean) / Cfg::V_PERIOD) & 1);
        bool key_waited = false;
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          if (!ok || t >= tiles[i]) continue;
          ok = wait(&p_full[i], t & 1);
          if (!ok) break;
          tc_fence_after();
          weigh(i, t);
          if (t + 1 < tiles[i]) {
            if (!key_waited) {
              ok = wait(&kv_full[ks], ((2 * t + 2) / SLOTS) & 1);
              if (!ok) break;
              key_waited = true;
              tc_fence_after();
            }
            scores(i, t + 1);
          }
        }
        if (!ok) break;
        umma_commit(&kv_empty[vs]);
        if (t + 1 < most) umma_commit(&kv_empty[ks]);
      }
    } else if (warp == W_GUARD) {
      // ---------------------------------------------------------- V guard
      const int most = work->most, clean = work->clean, all_see = work->all_see;
      const int kbeg = work->it.kbeg, kend = work->it.kend;
      for (int t = clean; t < most; ++t) {
        const int s = (2 * t + 1) % SLOTS, key0 = kbeg + t * 128;
        // (the load's issue first: before it, kv_full's parity could be that of a use two back)
        if (!attn_warp_wait(&v_load[s], ((t - clean) / Cfg::V_PERIOD) & 1, abort_flag, p.status) ||
            !attn_warp_wait(&kv_full[s], ((2 * t + 1) / SLOTS) & 1, abort_flag, p.status))
          break;
        uint8_t* v = sKV + s * TILE;
        const int nk = min(128, kend - key0);             // rows behind are cleared
        const int from = clamp_int(all_see - key0, 0, nk);  // rows before are seen by all
#pragma unroll 1
        for (int e = lane; e < NBX * (128 - from) * 8; e += 32) {
          const int b = e / ((128 - from) * 8), x = e % ((128 - from) * 8), r = from + (x >> 3);
          uint4* c = reinterpret_cast<uint4*>(v + b * BOX + r * 128 + (x & 7) * 16);
          if (r >= nk) {
            *c = make_uint4(0u, 0u, 0u, 0u);
            continue;
          }
          uint4 u = *c;
          uint32_t w[4] = {u.x, u.y, u.z, u.w};
          bool odd = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if ((w[i] & 0x7f80u) == 0x7f80u) {
              w[i] &= 0xffff0000u;
              odd = true;
            }
            if ((w[i] & 0x7f800000u) == 0x7f800000u) {
              w[i] &= 0xffffu;
              odd = true;
            }
          }
          if (odd) {
            *c = make_uint4(w[0], w[1], w[2], w[3]);
            *odd_values = 1;
          }
        }
        fence_proxy_async_smem();  // the tensor cores read V through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_ok[s]);
      }
    }
    __syncwarp();
  } else {
    constexpr bool HOLD = NQ == 2;
    if constexpr (NQ == 2) regs_inc<200>();
    // ------------------------------------------------------------ softmax, output
    const int i = NQ == 2 ? warp >> 2 : 0;
    const int q4 = warp & 3, r = q4 * 32 + lane;
    const uint32_t tmem = *tmem_slot;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
    const uint32_t tS = t_lane + 128 * i, tO = t_lane + NQ * 128 + DP * i;
    const int T = work->tiles[i], kbeg = work->it.kbeg;
    const int G = p.heads / p.kv_heads, R = 128 / G;
    const int tok = work->it.tok0 + i * R + r / G;  // of the sequence
    const bool real = r < R * G && tok < work->it.lq;
    const bool any = __any_sync(0xffffffffu, real);  // a warp without rows only keeps the barriers going
    int see = work->it.kend;
    if (p.causal) see = min(see, tok + 1 + work->it.lk - work->it.lq);
    const float c = p.scale * 1.4426950408889634f;
    float m = -INFINITY, l = 0.f;  // maximum (of c S) that O and l refer to
    bool ok = true;
    for (int t = 0; t < T; ++t) {
      if (!attn_warp_wait(&s_full[i], t & 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (any) {
        // S of the row, 64 keys at a time: held in registers with two row tiles, read
        // twice with one (which leaves registers for a second block on the SM)
        float s[HOLD ? 2 : 1][64];
        const int n = see - (kbeg + t * 128);  // visible keys of this tile
        const bool masked = __any_sync(0xffffffffu, n < 128);
        auto fetch = [&](int half) {
          float(&v)[64] = s[HOLD ? half : 0];
          tmem_ld2x32(tS + 64 * half, v);
          if (masked) {
#pragma unroll
            for (int x = 0; x < 64; ++x)
              if (64 * half + x >= n) v[x] = -INFINITY;
          }
        };
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          fetch(half);
#pragma unroll
          for (int x = 0; x < 64; x += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx[k] = fmaxf(mx[k], fmaxf(s[HOLD ? half : 0][x + k], s[HOLD ? half : 0][x + 4 + k]));
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        const bool grow = top > m + 8.f || (m == -INFINITY && top > m);
        if (__any_sync(0xffffffffu, grow)) {
          const float mn = grow ? top : m;
          if (t > 0) {
            const float alpha = grow ? ex2_approx(m - mn) : 1.f;
            l *= alpha;
            if (!attn_warp_wait(&o_full[i], (t - 1) & 1, abort_flag, p.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < DP; x += 16) {
              float o[16];
              tmem_ld16(tO + x, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= alpha;
              tmem_st16(tO + x, o);
            }
          }
          m = mn;
        }
        const float base = m == -INFINITY ? 0.f : m;
        float sum[4] = {};
#pragma unroll
        for (int x0 = 0; x0 < 128; x0 += 32) {
          if (!HOLD && (x0 & 63) == 0) fetch(x0 >> 6);  // (P lies over columns of S already read)
          const float(&v)[64] = s[HOLD ? x0 >> 6 : 0];
          uint32_t w[16];
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const int y = (x0 & 63) + x;
            const float a = ex2_approx(fmaf(v[y], c, -base)), b = ex2_approx(fmaf(v[y + 1], c, -base));
            sum[x & 2] += a;
            sum[(x & 2) + 1] += b;
            w[x >> 1] = pack_bf16x2(a, b);
          }
          tmem_st16(tS + x0 / 2, w);
        }
        tmem_st_wait();
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[i]);
    }
    if (ok && T > 0) ok = attn_warp_wait(&o_full[i], (T - 1) & 1, abort_flag, p.status);
    if (ok && any) {
      tc_fence_after();
      const long row = work->it.q0 + static_cast<long>(tok);
      const int hk = blockIdx.y, h = hk * G + r % G;
      const long at = (blockIdx.z * static_cast<long>(p.rows_q) + row) * p.heads + h;
      const float inv = p.nsplit > 1 ? 1.f : (l > 0.f || l != l ? 1.f / l : 0.f);
      const bool odd = *odd_values;
      if (p.nsplit > 1 && real) p.part_ml[at] = make_float2(m, l);
#pragma unroll
      for (int x = 0; x < DP; x += 16) {
        float o[16];
        if (T > 0) {
          tmem_ld16(tO + x, o);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = 0.f;
        }
        if (odd && real) {  // values the guard cleared, for the rows that see them
          for (int j = max(work->all_see, kbeg + work->clean * 128); j < see; ++j) {
            const __nv_bfloat16* vj = static_cast<const __nv_bfloat16*>(p.v) +
                                      (work->it.k0 + static_cast<long>(j)) * p.ldv + hk * p.d + x;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              if (x + k >= p.d) continue;
              const float f = to_f32(vj[k]);
              if (!isfinite(f)) o[k] += f;
            }
          }
        }
        if (!real) continue;
        if (p.nsplit > 1) {
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            if (x + k < p.d)
              *reinterpret_cast<float4*>(p.part_o + at * p.d + x + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        } else {
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row * p.ldo + h * p.d + x;
#pragma unroll
          for (int k = 0; k < 16; k += 8)
            if (x + k < p.d) {
              uint4 u;
              u.x = pack_bf16x2(o[k] * inv, o[k + 1] * inv);
              u.y = pack_bf16x2(o[k + 2] * inv, o[k + 3] * inv);
              u.z = pack_bf16x2(o[k + 4] * inv, o[k + 5] * inv);
              u.w = pack_bf16x2(o[k + 6] * inv, o[k + 7] * inv);
              *reinterpret_cast<uint4*>(out + k) = u;
            }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, Cfg::TMEM);
  }
}

}  // namespace edit
