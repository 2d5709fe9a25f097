// Packed softmax attention on the 5th-generation tensor cores (bf16 calls of
// edit_packed_attention_forward).
//
// Persistent blocks. An item is one or two row tiles of 128 packed rows (NQ; see
// packed_attn.cuh for the packing) of one key/value head, whose keys are streamed
// in tiles of 128. With two row tiles each K and V tile read into shared memory
// serves 256 rows, and while the softmax of one row tile runs, the tensor
// cores work for the other.
//   warps 0-3, 4-7  softmax of row tile 0, 1: one thread a row (its TMEM lane).
//   then            one warp each: TMA producer, MMA issuer; two warps: V guard.
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
// What bounds it: a row tile's round of scores, softmax, product is 3430 cycles for
// 1024 of tensor work (d = 128), and two row tiles overlap only in part, since S
// and O of two fill TMEM and P takes the place of S: 602 us for 5 causal prompts of
// up to 4100 tokens, 32 / 8 heads of 128 (890 TFLOP/s). One new token of 32 requests
// over 8K caches is the keys' bytes: 120 us, 4.5 TB/s.
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
  static constexpr int BARS = NQ * 5 + 4 * SLOTS;
  static constexpr int BATCH = 24;                  // items whose work is found at a time
  static constexpr int SMEM = 1024 + (NQ + SLOTS) * TILE + BARS * 8 + 16 + BATCH * 64;
  static_assert(SMEM * (NQ == 1 ? 2 : 1) + (NQ == 1 ? 2048 : 0) <= 232448 + 1024, "shared memory");
  // two row tiles: launched with 168 registers a thread, 200 for the softmax warps and 104 for the others (256 x 200 +
  // 128 x 104 = 384 x 168)
  static constexpr int THREADS = NQ * 128 + 128;
  static constexpr int TMEM = NQ * 256;             // S of tile i at 128 i, O behind them
  static constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 128);
  static constexpr uint32_t IDESC_O = idesc_bf16_f32(128, DP) | IDESC_B_MN;
};

// One item of a block's work: row tile(s) of a slot, a key/value head and a part
// of the keys.
template <int NQ>
struct AttnWork {
  int q_row, ntok;  // first row of q, tokens (0: an empty slot)
  int k_row;        // row of k of the first key, kbeg
  int kbeg, kend;   // key range within the sequence (kend: what the item's last row sees)
  int see0;         // keys that the item's first row sees (below 1: none)
  int hk, split;
  int tiles[NQ];    // key tiles of each row tile
  int most;         // the most of them
  int clean;        // key tiles all of whose keys every row sees; V tiles from there on have masked keys
};
template <int NQ>
__device__ __forceinline__ void attn_work(const PackedAttnParams& p, int item, int G, AttnWork<NQ>& w) {
  const int R = 128 / G;  // tokens a row tile
  w.split = 0;
  if (p.nsplit > 1) {
    w.split = item % p.nsplit;
    item /= p.nsplit;
  }
  const int slot = p.slots - 1 - item / p.kv_heads;  // last slots first: in a causal sequence they see the most keys
  w.hk = item % p.kv_heads;
  // the slot's sequence: the last one whose first slot is at or before it (see seq_of_slot)
  int s = 0;
  for (int n = p.nseq; n > 1;) {
    const int half = n / 2, first = clamp_int(p.q_offsets[s + half], 0, p.rows_q) / (NQ * R) + s + half;
    s += first <= slot ? half : 0;
    n = first <= slot ? n - half : half;
  }
  const SeqRows q = seq_rows(p.q_offsets, s, p.rows_q), k = seq_keys(p, s);
  const int tile = slot - (q.begin / (NQ * R) + s);
  w.ntok = tile < 0 || tile > (q.len - 1) / (NQ * R) || q.len == 0 ? 0 : min(NQ * R, q.len - tile * NQ * R);
  w.most = w.clean = 0;
#pragma unroll
  for (int i = 0; i < NQ; ++i) w.tiles[i] = 0;
  if (w.ntok == 0) return;
  const int tok0 = tile * NQ * R, shift = k.len - q.len;
  w.q_row = q.begin + tok0;
  w.kbeg = 0;
  w.kend = p.causal ? clamp_int(tok0 + w.ntok + shift, 0, k.len) : k.len;
  w.see0 = p.causal ? tok0 + 1 + shift : k.len;
  if (p.nsplit > 1) {  // whole tiles but the last
    const long nt = (w.kend + 127) / 128;
    w.kbeg = static_cast<int>(nt * w.split / p.nsplit) * 128;
    w.kend = min(w.kend, static_cast<int>(nt * (w.split + 1) / p.nsplit) * 128);
  }
  w.k_row = k.begin + w.kbeg;
#pragma unroll
  for (int i = 0; i < NQ; ++i) {  // those that the tile's last row sees (within this part)
    const int n = min(w.ntok - i * R, R);  // tokens
    const int kend = p.causal ? min(w.kend, tok0 + i * R + n + shift) : w.kend;
    w.tiles[i] = n > 0 && kend > w.kbeg ? (kend - w.kbeg + 127) / 128 : 0;
    w.most = max(w.most, w.tiles[i]);
  }
  w.clean = max(0, min(w.most, (min(w.kend, w.see0) - w.kbeg) / 128));
}

template <int R>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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
                          const __grid_constant__ CUtensorMap mv, const PackedAttnParams p, const int items) {
  using Cfg = AttnTcCfg<DP, NQ>;
  constexpr int NBX = Cfg::NBX, BOX = Cfg::BOX, TILE = Cfg::TILE, SLOTS = Cfg::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sQ = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sKV = sQ + NQ * TILE;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sKV + SLOTS * TILE);  // [NQ]
  uint64_t* q_empty = q_full + NQ;   // [NQ]
  uint64_t* s_full = q_empty + NQ;   // [NQ] scores of a key tile
  uint64_t* p_full = s_full + NQ;    // [NQ] weights of a key tile
  uint64_t* o_full = p_full + NQ;    // [NQ] O includes a key tile
  uint64_t* kv_full = o_full + NQ;   // [SLOTS]
  uint64_t* kv_empty = kv_full + SLOTS;
  uint64_t* v_ok = kv_empty + SLOTS;  // [SLOTS] V tile with masked keys made safe
  uint64_t* v_load = v_ok + SLOTS;    // [SLOTS] such a tile's load has been issued
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(v_load + SLOTS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* odd_values = abort_flag + 1;  // the guard cleared values that are not finite (in any item so far)

  AttnWork<NQ>* work = reinterpret_cast<AttnWork<NQ>*>(tmem_slot + 4);  // [BATCH]
  static_assert(sizeof(AttnWork<NQ>) <= 64, "work");

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  constexpr int W_TMA = NQ * 4, W_MMA = W_TMA + 1, W_GUARD = W_TMA + 2;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);  // one arrival a softmax warp
      mbar_init(&o_full[i], 1);
    }
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
      mbar_init(&v_ok[s], 2);  // one arrival a guard warp
      mbar_init(&v_load[s], 1);
    }
    *abort_flag = 0;
    *odd_values = 0;
    fence_mbar_init();
  }
  if (warp == W_TMA && lane == 0) {
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
  }
  if (warp == W_MMA) tmem_alloc(tmem_slot, Cfg::TMEM);
  pdl_wait();
  if (blockIdx.x == 0)
    check_offsets(p.q_offsets, p.rows_q, p.k_offsets, p.rows_k, p.k_lens, p.max_k, p.nseq, p.status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  // Each role walks the block's items by itself, so that the loads and the first scores of an item run under the
  // end of the one before. What the items are is found for a batch of them at once, one thread each (found by every
  // role for every item it took 8 us an item, a chain of loads and divisions).
  const int G = p.heads / p.kv_heads, R = 128 / G;
  auto batch = [&](int first) {  // all threads of the block; returns the items of the batch
    named_bar_sync(1, Cfg::THREADS);  // the last batch is done with
    const int item = first + static_cast<int>(threadIdx.x * gridDim.x);
    if (threadIdx.x < Cfg::BATCH && item < items) attn_work<NQ>(p, item, G, work[threadIdx.x]);
    named_bar_sync(1, Cfg::THREADS);
    return min(+Cfg::BATCH, (items - first + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x));
  };
  const int stride = Cfg::BATCH * static_cast<int>(gridDim.x);
  if (warp >= W_TMA) {
    if constexpr (NQ == 2) regs_dec<104>();
    bool ok = true;
    uint32_t guarded = 0;  // bit s: parity of v_ok / v_load of slot s
    if (warp == W_TMA) {
      // ---------------------------------------------------------- producer: Q, then K_0 V_0 K_1 V_1 ...
      int s = 0;                     // slot of the next load
      uint32_t empty = 1, qe = ~0u;  // parities to wait for
      for (int first = blockIdx.x; first < items; first += stride)
        for (int left = batch(first), e = 0; e < left; ++e) {
        const AttnWork<NQ> w = work[e];
        if (lane == 0 && ok) {
#pragma unroll
          for (int i = 0; i < NQ; ++i) {
            if (w.tiles[i] == 0 || !ok) continue;
            ok = attn_wait(&q_empty[i], (qe >> i) & 1, abort_flag, p.status);
            if (!ok) break;
            qe ^= 1u << i;
            mbar_arrive_expect_tx(&q_full[i], NBX * R * G * 128);
#pragma unroll
            for (int b = 0; b < NBX; ++b)
              tma_load_4d(&mq, &q_full[i], sQ + i * TILE + b * BOX, 64 * b, 0, w.hk, w.q_row + i * R);
          }
          for (int t = 0; t < 2 * w.most && ok; ++t) {
            ok = attn_wait(&kv_empty[s], empty, abort_flag, p.status);
            if (!ok) break;
            mbar_arrive_expect_tx(&kv_full[s], TILE);
#pragma unroll
            for (int b = 0; b < NBX; ++b)
              tma_load_3d(t & 1 ? &mv : &mk, &kv_full[s], sKV + s * TILE + b * BOX, 64 * b, w.hk,
                          w.k_row + (t >> 1) * 128);
            if ((t & 1) && (t >> 1) >= w.clean) mbar_arrive(&v_load[s]);
            if (++s == SLOTS) {
              s = 0;
              empty ^= 1;
            }
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (lane == 0 && *abort_flag) let_copies_land();
    } else if (warp == W_MMA) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t tmem = *tmem_slot;
      // the whole warp walks along, one lane issues (see umma_bf16_by)
      const uint32_t leader = elect_one();
      auto wait = [&](uint64_t* bar, uint32_t parity) { return attn_warp_wait(bar, parity, abort_flag, p.status); };
      auto scores = [&](int i, int slot) {  // S_i = Q_i K^T
        const uint64_t qd = sdesc_kmajor_sw128(smem_u32(sQ + i * TILE));
        const uint64_t kd = sdesc_kmajor_sw128(smem_u32(sKV + slot * TILE));
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint64_t step = ((k >> 2) * BOX + (k & 3) * 32) >> 4;
          umma_bf16_by(leader, tmem + 128 * i, qd + step, kd + step, Cfg::IDESC_S, k > 0 ? 1u : 0u);
        }
        umma_commit_by(leader, &s_full[i]);
      };
      auto weigh = [&](int i, int slot, bool first) {  // O_i += P_i V
        const uint64_t vd = sdesc_mnmajor_sw128(smem_u32(sKV + slot * TILE), BOX);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_bf16_ts_by(leader, tmem + NQ * 128 + DP * i, tmem + 128 * i + 8 * k, vd + (2048 >> 4) * k, Cfg::IDESC_O,
                       (!first || k > 0) ? 1u : 0u);
        umma_commit_by(leader, &o_full[i]);
      };
      int s = 0;          // slot of the next tile to use
      uint32_t full = 0;  // its parity
      uint32_t qf = 0, pf = 0;  // parities of q_full, p_full by row tile
      auto next = [&](int& slot, uint32_t& par) {
        if (++slot == SLOTS) {
          slot = 0;
          par ^= 1;
        }
      };
      for (int first = blockIdx.x; first < items; first += stride)
        for (int left = batch(first), e = 0; e < left; ++e) {
        const AttnWork<NQ> w = work[e];
        if (w.most == 0 || !ok) continue;
        ok = wait(&kv_full[s], full);
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          if (w.tiles[i] == 0 || !ok) continue;
          ok = wait(&q_full[i], (qf >> i) & 1);
          if (!ok) break;
          qf ^= 1u << i;
          tc_fence_after();
          scores(i, s);
          if (w.tiles[i] == 1) umma_commit_by(leader, &q_empty[i]);
        }
        if (ok) umma_commit_by(leader, &kv_empty[s]);
        next(s, full);
        for (int t = 0; t < w.most && ok; ++t) {
          const int vs = s;
          ok = wait(&kv_full[vs], full);
          if (ok && t >= w.clean) {
            ok = wait(&v_ok[vs], (guarded >> vs) & 1);
            guarded ^= 1u << vs;
          }
          next(s, full);  // now the next K
          bool key_waited = false;
#pragma unroll
          for (int i = 0; i < NQ; ++i) {
            if (!ok || t >= w.tiles[i]) continue;
            ok = wait(&p_full[i], (pf >> i) & 1);
            if (!ok) break;
            pf ^= 1u << i;
            tc_fence_after();
            weigh(i, vs, t == 0);
            if (t + 1 < w.tiles[i]) {
              if (!key_waited) {
                ok = wait(&kv_full[s], full);
                if (!ok) break;
                key_waited = true;
                tc_fence_after();
              }
              scores(i, s);
              if (t + 2 == w.tiles[i]) umma_commit_by(leader, &q_empty[i]);  // the item's last reads of its Q
            }
          }
          if (!ok) break;
          umma_commit_by(leader, &kv_empty[vs]);
          if (t + 1 < w.most) {
            umma_commit_by(leader, &kv_empty[s]);
            next(s, full);
          }
        }
      }
    } else {
      // ---------------------------------------------------------- V guard, two warps
      int n = 0;  // tiles loaded before this item
      for (int first = blockIdx.x; first < items; first += stride)
        for (int left = batch(first), e = 0; e < left && ok; ++e) {
        const AttnWork<NQ> w = work[e];
        const int n0 = n;
        n += 2 * w.most;
        for (int t = w.clean; t < w.most; ++t) {
          const int nv = n0 + 2 * t + 1, s = nv % SLOTS, key0 = w.kbeg + t * 128;
          // (the load's issue first: before it, kv_full's parity could be that of a use two back)
          if (!attn_warp_wait(&v_load[s], (guarded >> s) & 1, abort_flag, p.status) ||
              !attn_warp_wait(&kv_full[s], (nv / SLOTS) & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          guarded ^= 1u << s;
          uint8_t* v = sKV + s * TILE;
          const int nk = min(128, w.kend - key0);               // rows behind are cleared
          const int from = clamp_int(w.see0 - key0, 0, nk);     // rows before are seen by all
          // a warp takes 4 of every 8 rows, 16 bytes a lane
          const int r0 = 4 * (warp - W_GUARD) + (lane >> 3);
          uint8_t* mine = v + (lane & 7) * 16;
          for (int r = (from & ~7) + r0; r < 128; r += 8) {
            if (r < from) continue;
#pragma unroll
            for (int b = 0; b < NBX; ++b) {
              uint4* c = reinterpret_cast<uint4*>(mine + b * BOX + r * 128);
              const uint4 u = r < nk ? *c : make_uint4(0u, 0u, 0u, 0u);
              if (r < nk) {  // exponents of all ones in either half of a word
                auto odd2 = [](uint32_t x) { return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
                if (odd2(u.x) | odd2(u.y) | odd2(u.z) | odd2(u.w)) {
                  auto clear = [&](uint32_t x) {
                    const uint32_t o = odd2(x);
                    return x & ((o & 0x8000u ? 0u : 0xffffu) | (o & 0x80000000u ? 0u : 0xffff0000u));
                  };
                  *c = make_uint4(clear(u.x), clear(u.y), clear(u.z), clear(u.w));
                  *odd_values = 1;
                }
              } else {
                *c = u;
              }
            }
          }
          fence_proxy_async_smem();  // the tensor cores read V through the async proxy
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_ok[s]);
        }
      }
    }
    __syncwarp();
  } else {
    if constexpr (NQ == 2) regs_inc<200>();
    constexpr bool HOLD = NQ == 2;
    // ------------------------------------------------------------ softmax, output
    const int i = NQ == 2 ? warp >> 2 : 0;
    const int q4 = warp & 3, r = q4 * 32 + lane;
    const uint32_t t_lane = *tmem_slot + (static_cast<uint32_t>(q4 * 32) << 16);
    const uint32_t tS = t_lane + 128 * i, tO = t_lane + NQ * 128 + DP * i;
    const float c = p.scale * 1.4426950408889634f;
    uint32_t n_par = 0;  // parity of this row tile's next key tile
    bool ok = true;
    const int r_tok = i * R + r / G, r_head = r % G;  // this row's token of an item and head of a group
    for (int first = blockIdx.x; first < items; first += stride)
      for (int left = batch(first), e = 0; e < left; ++e) {
      const AttnWork<NQ>& w = work[e];
      if (w.ntok == 0 || !ok) continue;
      const int T = w.tiles[i], kbeg = w.kbeg;
      const bool real = r < R * G && r_tok < w.ntok;
      const bool any = __any_sync(0xffffffffu, real);  // a warp without rows only keeps the barriers going
      const int see = p.causal ? min(w.kend, w.see0 + r_tok) : w.kend;  // keys this row sees
      float m = -INFINITY, l = 0.f;  // maximum (of c S) that O and l refer to
      for (int t = 0; t < T; ++t, n_par ^= 1) {
        if (!attn_warp_wait(&s_full[i], n_par, abort_flag, p.status)) {
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
                mx[k] = max3(mx[k], s[HOLD ? half : 0][x + 2 * k], s[HOLD ? half : 0][x + 2 * k + 1]);
          }
          const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * c;
          const bool grow = top > m + 8.f || (m == -INFINITY && top > m);
          if (__any_sync(0xffffffffu, grow)) {
            const float mn = grow ? top : m;
            if (t > 0) {
              const float alpha = grow ? ex2_approx(m - mn) : 1.f;
              l *= alpha;
              if (!attn_warp_wait(&o_full[i], n_par ^ 1, abort_flag, p.status)) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll
              for (int x = 0; x < DP; x += 16) {
                float o[16];
                uint32_t u[16];
                tmem_ld16(tO + x, o);
#pragma unroll
                for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(o[k] * alpha);
                tmem_st16(tO + x, u);
              }
            }
            m = mn;
          }
          const float base = m == -INFINITY ? 0.f : m;
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const float2 c2 = make_float2(c, c), b2 = make_float2(-base, -base);
#pragma unroll
          for (int x0 = 0; x0 < 128; x0 += 32) {
            if (!HOLD && (x0 & 63) == 0) fetch(x0 >> 6);  // (P lies over columns of S already read)
            const float(&v)[64] = s[HOLD ? x0 >> 6 : 0];
            uint32_t u[16];
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              const int y = (x0 & 63) + x;
              float2 e = fma2(make_float2(v[y], v[y + 1]), c2, b2);
              e.x = ex2_approx(e.x);
              e.y = ex2_approx(e.y);
              sum[(x >> 1) & 1] = add2(sum[(x >> 1) & 1], e);
              u[x >> 1] = pack_bf16x2(e.x, e.y);
            }
            tmem_st16(tS + x0 / 2, u);
          }
          tmem_st_wait();
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[i]);
      }
      if (ok && T > 0) ok = attn_warp_wait(&o_full[i], n_par ^ 1, abort_flag, p.status);
      if (!ok || !any) continue;
      tc_fence_after();
      const long row = w.q_row + static_cast<long>(r_tok);
      const int h = w.hk * G + r_head;
      const long at = (w.split * static_cast<long>(p.rows_q) + row) * p.heads + h;
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
          for (int j = max(w.see0, kbeg + w.clean * 128); j < see; ++j) {
            const __nv_bfloat16* vj = static_cast<const __nv_bfloat16*>(p.v) +
                                      (w.k_row - kbeg + static_cast<long>(j)) * p.ldv + w.hk * p.d + x;
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
      tc_fence_before();  // O has been read: the next item's first weights may be announced
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
