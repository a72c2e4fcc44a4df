// attn_cache.cu -- attention of chunks of new tokens over the paged key/value
// cache (hia_attn_cache_fwd), bf16 and fp16, head dimension 64 and 128.
//
// Definition: row (t, h) of sequence b, bound e: O = sum_{j <= e} p_j v_j / l,
// p_j = exp(scale q . k_j - m), l = sum p_j, lse = m + log l, with the running
// maximum m and sum l of an online softmax in fp32.
//
// Two kernels, for the two things that bound this operator:
//   attn_cache_rows   few rows per sequence (single tokens): the time is that
//                     of reading K and V once.  Warp-private streams of key
//                     steps, mma.sync on 16 rows.
//   attn_cache_tiles  many rows: the products bound it.  tcgen05 on 2 x 128
//                     rows per CTA, one CTA per SM.
// Both cut their work by the same device-side plan: an item is (sequence, row
// tile, kv head); an item with more than C units of 128 keys is split into
// equal pieces over the keys, whose normalised partials attn_cache_join adds
// in piece order.  The lengths are only known on the device (they change
// between replays of a captured graph), so every CTA computes the plan from
// the arrays of the chunk.
#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "cache.cuh"
#include "devctx.h"

namespace hia {
namespace {

constexpr int kUnit = 128;  // keys per unit of the plan
constexpr uint64_t kTimeoutNs = 2000000000ull;

struct CacheAttn {
  ChunkDev chunk;
  const void* q;  // rows kernel only (the tiles kernel has a tensor map)
  int64_t q_ss, q_sh, q_sq;
  void* o;
  int64_t o_ss, o_sh, o_sq;
  float* lse;            // [Hq][T], or nullptr
  const int32_t* bound;  // [T], or nullptr: causal
  float scale_log2;
  int Hkv, g;
  int tpt;           // tiles kernel: tokens per 128-row tile; 0: rows kernel
  int cta_slots;     // CTAs resident on the device at a time
  int max_slots;     // partial slots in the workspace
  float piece_cost;  // fixed cost of a piece, in units
  float* part;       // [max_slots][rows of a tile][D], normalised
  float* part_lse;   // [max_slots][rows of a tile], log2
};

// Rows of an item: the rows kernel takes 16 consecutive (token, head of the
// group) rows, the tiles kernel 2 x tpt tokens with all g heads each.
constexpr int kRowsM = 16;
constexpr int kTilesM = 256;

__device__ __forceinline__ int item_tiles(const CacheAttn& p, int n) {
  if (p.tpt) return (n + 2 * p.tpt - 1) / (2 * p.tpt);
  return int((int64_t(n) * p.g + kRowsM - 1) / kRowsM);
}

// ---------------------------------------------------------------- plan
struct Work {
  int b, row0, n, past;  // the sequence
  int tile, hkv, piece, pieces;
  int slot;              // partial slot of this piece (pieces > 1)
};

constexpr int kCand = 5;

template <int NT>
struct PlanSmem {
  long long sum[NT / 32][2 * kCand];
  int top[NT / 32];
  int scan[NT / 32][3];
  int C;
  int found;
  Work work;
};

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Pieces of an item of `units` units.
__device__ __forceinline__ int pieces_of(int units, int C) { return units > C ? (units + C - 1) / C : 1; }

// The most units of a piece.  Candidates: no split, and splits that give
// about 1, 2, 3, 4 pieces per CTA slot; the estimate of each is that of a
// list schedule, work per slot plus half of the longest piece (all in one
// wave: the longest piece), each piece with a fixed cost.
template <int NT>
__device__ int plan_units(const CacheAttn& p, PlanSmem<NT>& sm) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  long long w = 0;
  int top = 0;
  for (int b = tid; b < p.chunk.B; b += NT) {
    const Seq s = chunk_seq(p.chunk, b);
    if (!s.n) continue;
    const int units = (s.past + s.n + kUnit - 1) / kUnit;
    w += (long long)item_tiles(p, s.n) * units;
    top = max(top, units);
  }
  w = warp_sum(w);
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) {
    sm.sum[warp][0] = w;
    sm.top[warp] = top;
  }
  __syncthreads();
  w = 0;
  top = 0;
  for (int i = 0; i < NT / 32; ++i) {
    w += sm.sum[i][0];
    top = max(top, sm.top[i]);
  }
  w *= p.Hkv;
  if (top <= 1) return 1;
  int C[kCand];
  long long n[kCand], ns[kCand];
#pragma unroll
  for (int k = 0; k < kCand; ++k) {
    const long long per = k ? (w + (long long)p.cta_slots * k - 1) / ((long long)p.cta_slots * k) : top;
    C[k] = int(per < top ? per : top);
    n[k] = ns[k] = 0;
  }
  for (int b = tid; b < p.chunk.B; b += NT) {
    const Seq s = chunk_seq(p.chunk, b);
    if (!s.n) continue;
    const int units = (s.past + s.n + kUnit - 1) / kUnit;
    const long long tiles = item_tiles(p, s.n);
#pragma unroll
    for (int k = 0; k < kCand; ++k) {
      const int P = pieces_of(units, C[k]);
      n[k] += tiles * P;
      if (P > 1) ns[k] += tiles * P;
    }
  }
  __syncthreads();  // sum[][0] has been read
#pragma unroll
  for (int k = 0; k < kCand; ++k) {
    const long long a = warp_sum(n[k]), c = warp_sum(ns[k]);
    if (lane == 0) {
      sm.sum[warp][k] = a;
      sm.sum[warp][kCand + k] = c;
    }
  }
  __syncthreads();
  if (tid == 0) {
    float best = 0.f;
    int pick = top;
#pragma unroll
    for (int k = 0; k < kCand; ++k) {
      long long a = 0, c = 0;
      for (int i = 0; i < NT / 32; ++i) {
        a += sm.sum[i][k];
        c += sm.sum[i][kCand + k];
      }
      a *= p.Hkv;
      c *= p.Hkv;
      if (k && c > p.max_slots) continue;
      const float piece = C[k] + p.piece_cost;
      const float est = a <= p.cta_slots ? piece : (w + a * p.piece_cost) / p.cta_slots + 0.5f * piece;
      if (k == 0 || est < best) {
        best = est;
        pick = C[k];
      }
    }
    sm.C = pick;
  }
  __syncthreads();
  return sm.C;
}

// Piece `target` of the plan (JOIN: split item `target`).  Every thread of the
// block calls it; false past the last one.
template <int NT, bool JOIN>
__device__ bool plan_find(const CacheAttn& p, PlanSmem<NT>& sm, int target) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) sm.found = 0;
  const int C = plan_units<NT>(p, sm);
  // thread i owns the sequences [i K, (i+1) K): exclusive scan over the
  // threads of their pieces (JOIN: split items) and partial slots
  const int K = (p.chunk.B + NT - 1) / NT;
  const int b0 = tid * K, b1 = min(b0 + K, p.chunk.B);
  int cnt = 0, slots = 0;
  const auto count = [&](const Seq& s, int& units, int& P, int& c, int& sl) {
    units = (s.past + s.n + kUnit - 1) / kUnit;
    P = pieces_of(units, C);
    const int items = s.n ? item_tiles(p, s.n) * p.Hkv : 0;
    sl = P > 1 ? items * P : 0;
    c = JOIN ? (P > 1 ? items : 0) : items * P;
  };
  for (int b = b0; b < b1; ++b) {
    int u, P, c, sl;
    count(chunk_seq(p.chunk, b), u, P, c, sl);
    cnt += c;
    slots += sl;
  }
  int ic = cnt, is = slots;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, ic, o), y = __shfl_up_sync(0xffffffffu, is, o);
    if (lane >= o) {
      ic += x;
      is += y;
    }
  }
  if (lane == 31) {
    sm.scan[warp][0] = ic;
    sm.scan[warp][1] = is;
  }
  __syncthreads();
  int at = ic - cnt, slot0 = is - slots;
  for (int i = 0; i < warp; ++i) {
    at += sm.scan[i][0];
    slot0 += sm.scan[i][1];
  }
  if (target >= at && target < at + cnt) {
    for (int b = b0; b < b1; ++b) {
      const Seq s = chunk_seq(p.chunk, b);
      int u, P, c, sl;
      count(s, u, P, c, sl);
      if (target < at + c) {
        // within a sequence: last tiles (the longest, when causal) first
        int i = target - at;
        Work w{b, s.row0, s.n, s.past, 0, 0, 0, P, 0};
        w.hkv = i % p.Hkv;
        i /= p.Hkv;
        if (!JOIN) {
          w.piece = i % P;
          i /= P;
        }
        w.tile = item_tiles(p, s.n) - 1 - i;
        w.slot = slot0 + (i * P + w.piece) * p.Hkv + w.hkv;  // slots of an item: Hkv apart
        sm.work = w;
        sm.found = 1;
        break;
      }
      at += c;
      slot0 += sl;
    }
  }
  __syncthreads();
  return sm.found != 0;
}

// Last visible position of the row of token i, -1 for none.
__device__ __forceinline__ int row_limit(const CacheAttn& p, const Work& w, int i) {
  const int e = p.bound ? __ldg(p.bound + w.row0 + i) : w.past + i;
  return max(min(e, w.past + w.n - 1), -1);
}

// Units of the piece: an equal share of the units that the tile sees.
__device__ __forceinline__ void piece_range(const Work& w, int units, int& u0, int& u1) {
  u0 = int((long long)units * w.piece / w.pieces);
  u1 = int((long long)units * (w.piece + 1) / w.pieces);
}

template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  return pack_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---------------------------------------------------------------- few rows
constexpr int kRWarps = 4;
constexpr int kRThreads = kRWarps * 32;
template <int D>
struct RowsCfg {
  static constexpr int kKeys = 16;                 // keys of a step
  static constexpr int kStages = D == 128 ? 3 : 6;  // steps in flight per warp
};

template <int D>
struct RowsSmem {
  static constexpr int kHalf = RowsCfg<D>::kKeys * 64;  // elements: keys x 64 columns, 128-byte rows, swizzled
  // [stage][K, V][64-wide column block]
  alignas(1024) uint16_t kv[kRWarps][RowsCfg<D>::kStages][2][D / 64][kHalf];
  uint64_t full[kRWarps][RowsCfg<D>::kStages];
  float m[kRWarps][kRowsM], l[kRWarps][kRowsM];
  int abort_flag;
  PlanSmem<kRThreads> plan;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <class T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A warp streams its own key steps (every fourth of the piece) through its own
// ring of TMA tiles with its own running maximum, sum and output; the four
// warps meet once, at the end.  Row r of the tile is row tile*16 + r of the
// sequence's n*g (token, head of the group) rows.
template <class T, int D>
__global__ void __launch_bounds__(kRThreads)
    attn_cache_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const CacheAttn p) {
  constexpr int kKeys = RowsCfg<D>::kKeys, kStages = RowsCfg<D>::kStages;
  extern __shared__ uint8_t smem_raw[];
  RowsSmem<D>& sm = *reinterpret_cast<RowsSmem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int w = 0; w < kRWarps; ++w)
      for (int i = 0; i < kStages; ++i) mbar_init(&sm.full[w][i], 1);
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (!plan_find<kRThreads, false>(p, sm.plan, blockIdx.x)) return;  // ends with __syncthreads
  const Work w = sm.plan.work;
  const WaitCtx wc{&sm.abort_flag, p.chunk.status, kTimeoutNs};

  // this thread's rows: lane / 4 and lane / 4 + 8
  const int64_t n_rows = int64_t(w.n) * p.g;
  int lim[2];
  uint32_t qf[D / 16][4];
  int end = 0, low = 0x7fffffff;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t r = int64_t(w.tile) * kRowsM + (lane >> 2) + 8 * i;
    lim[i] = -1;
    if (r < n_rows) {
      const int tok = int(r / p.g), h = int(r % p.g);
      lim[i] = row_limit(p, w, tok);
      end = max(end, lim[i] + 1);
      low = min(low, lim[i]);
      const uint16_t* q = static_cast<const uint16_t*>(p.q) + int64_t(w.row0 + tok) * p.q_ss + int64_t(w.hkv) * p.q_sh +
                          int64_t(h) * p.q_sq;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          qf[ks][i + 2 * j] = __ldg(reinterpret_cast<const uint32_t*>(q + ks * 16 + j * 8 + (lane & 3) * 2));
    } else {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) qf[ks][i] = qf[ks][i + 2] = 0u;
    }
  }
  end = __reduce_max_sync(0xffffffffu, end);
  low = __reduce_min_sync(0xffffffffu, low);

  int u0, u1;
  piece_range(w, (end + kUnit - 1) / kUnit, u0, u1);
  const int key0 = u0 * kUnit, key1 = min(u1 * kUnit, end);
  const int steps = key1 > key0 ? (key1 - key0 + kKeys - 1) / kKeys : 0;
  const int mine = steps > warp ? (steps - warp + kRWarps - 1) / kRWarps : 0;  // steps warp, warp + 4, ...

  // one lane issues the copies of step i: one box per (K or V, column block);
  // a step never crosses a page (pages hold a multiple of 16 slots)
  int page_reg = 0;  // page of step (i & ~31) + lane
  const auto load_pages = [&](int i0) {
    const int i = i0 + lane;
    if (i < mine) page_reg = chunk_page(p.chunk, w.b, (key0 + (warp + i * kRWarps) * kKeys) >> p.chunk.page_shift);
  };
  const auto issue = [&](int i) {
    if ((i & 31) == 0) load_pages(i);
    const int page = __shfl_sync(0xffffffffu, page_reg, i & 31);
    if (lane == 0) {
      const int s = i % kStages;
      const int slot = (key0 + (warp + i * kRWarps) * kKeys) & ((1 << p.chunk.page_shift) - 1);
      mbar_arrive_expect_tx(&sm.full[warp][s], 2 * D * kKeys * 2);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        tma_load_4d(sm.kv[warp][s][0][c], &tm_k, &sm.full[warp][s], c * 64, slot, w.hkv, page);
        tma_load_4d(sm.kv[warp][s][1][c], &tm_v, &sm.full[warp][s], c * 64, slot, w.hkv, page);
      }
    }
  };
  int issued = 0;
  for (; issued < min(mine, kStages); ++issued) issue(issued);

  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const float cs = p.scale_log2;

  for (int i = 0; i < mine; ++i) {
    const int s = i % kStages;
    if (!__all_sync(0xffffffffu, mbar_wait(&sm.full[warp][s], (i / kStages) & 1, wc))) break;
    const uint32_t kb = smem_u32(sm.kv[warp][s][0]), vb = smem_u32(sm.kv[warp][s][1]);
    float acc[kKeys / 8][4];
#pragma unroll
    for (int n = 0; n < kKeys / 8; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int np = 0; np < kKeys / 16; ++np) {
        const int key = np * 16 + ((lane >> 4) << 3) + (lane & 7), ch = ks * 2 + ((lane >> 3) & 1);
        uint32_t b[4];
        ldsm4(b, kb + uint32_t(ch >> 3) * (kKeys * 128) + sw128_offset(key, ch & 7));
        mma16816<T>(acc[2 * np], qf[ks], b[0], b[1]);
        mma16816<T>(acc[2 * np + 1], qf[ks], b[2], b[3]);
      }
    const int k0 = key0 + (warp + i * kRWarps) * kKeys;
    if (k0 + kKeys - 1 > low) {
#pragma unroll
      for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (k0 + n * 8 + (lane & 3) * 2 + (e & 1) > lim[e >> 1]) acc[n][e] = -INFINITY;
    }
    uint32_t pf[kKeys / 16][4];
    float f[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float x = -INFINITY;
#pragma unroll
      for (int n = 0; n < kKeys / 8; ++n) x = fmaxf(x, fmaxf(acc[n][2 * r], acc[n][2 * r + 1]));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
      const float mn = fmaxf(m[r], x * cs);
      const float sub = mn == -INFINITY ? 0.f : mn;  // a row that has seen no key yet
      f[r] = ex2_approx(m[r] - sub);
      m[r] = mn;
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float pv = ex2_approx(fmaf(acc[n][2 * r + e], cs, -sub));
          acc[n][2 * r + e] = pv;
          sum += pv;
        }
      l[r] = l[r] * f[r] + sum;
    }
#pragma unroll
    for (int kp = 0; kp < kKeys / 16; ++kp) {
      pf[kp][0] = pack2<T>(acc[2 * kp][0], acc[2 * kp][1]);
      pf[kp][1] = pack2<T>(acc[2 * kp][2], acc[2 * kp][3]);
      pf[kp][2] = pack2<T>(acc[2 * kp + 1][0], acc[2 * kp + 1][1]);
      pf[kp][3] = pack2<T>(acc[2 * kp + 1][2], acc[2 * kp + 1][3]);
    }
    if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][0] *= f[0];
        o[n][1] *= f[0];
        o[n][2] *= f[1];
        o[n][3] *= f[1];
      }
    }
    // slots at or past the tile's last visible key may hold anything: a weight
    // of zero does not silence a NaN, so their values are cleared
    const bool tail = k0 + kKeys > end;
#pragma unroll
    for (int kp = 0; kp < kKeys / 16; ++kp) {
      uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
      if (tail) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int key = k0 + kp * 16 + j * 8 + (lane & 3) * 2;
          keep[j] = (key < end ? 0xffffu : 0u) | (key + 1 < end ? 0xffff0000u : 0u);
        }
      }
#pragma unroll
      for (int dp = 0; dp < D / 16; ++dp) {
        const int key = kp * 16 + (((lane >> 3) & 1) << 3) + (lane & 7), ch = dp * 2 + (lane >> 4);
        uint32_t b[4];
        ldsm4_t(b, vb + uint32_t(ch >> 3) * (kKeys * 128) + sw128_offset(key, ch & 7));
        if (tail) {
          b[0] &= keep[0];
          b[1] &= keep[1];
          b[2] &= keep[0];
          b[3] &= keep[1];
        }
        mma16816<T>(o[2 * dp], pf[kp], b[0], b[1]);
        mma16816<T>(o[2 * dp + 1], pf[kp], b[2], b[3]);
      }
    }
    __syncwarp();
    if (issued < mine) {
      issue(issued);
      ++issued;
    }
  }
  // every copy issued must land before the shared memory is reused or released
  for (int i = max(issued - kStages, 0); i < issued; ++i)
    mbar_wait_hw(&sm.full[warp][i % kStages], (i / kStages) & 1, wc);

  // ---- the warps meet: output rows [16][D] fp32 in each warp's own ring
  static_assert(sizeof(sm.kv[0]) >= kRowsM * D * 4, "a warp's ring holds its output rows");
  __syncwarp();
  float* om = reinterpret_cast<float*>(sm.kv[warp]);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    const int row = (lane >> 2) + 8 * r;
    if ((lane & 3) == 0) {
      sm.m[warp][row] = m[r];
      sm.l[warp][row] = l[r];
    }
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<float2*>(om + row * D + ((n * 8 + (lane & 3) * 2) ^ ((row & 3) * 8))) =
          make_float2(o[n][2 * r], o[n][2 * r + 1]);
  }
  __syncthreads();
  const int row = threadIdx.x >> 3, sub = threadIdx.x & 7;  // 8 threads a row
  const int64_t flat = int64_t(w.tile) * kRowsM + row;
  if (flat >= n_rows) return;
  float top = -INFINITY, sum = 0.f, wt[kRWarps];
#pragma unroll
  for (int i = 0; i < kRWarps; ++i) top = fmaxf(top, sm.m[i][row]);
#pragma unroll
  for (int i = 0; i < kRWarps; ++i) {
    wt[i] = top == -INFINITY ? 0.f : ex2_approx(sm.m[i][row] - top);
    sum += sm.l[i][row] * wt[i];
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int tok = int(flat / p.g), h = int(flat % p.g);
  const float lse2 = sum > 0.f ? top + __log2f(sum) : -INFINITY;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    const int d = c * 64 + sub * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kRWarps; ++i) {
      const float4* x = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm.kv[i]) + row * D + (d ^ ((row & 3) * 8)));
      const float4 a = x[0], b = x[1];
      v[0] = fmaf(a.x, wt[i], v[0]); v[1] = fmaf(a.y, wt[i], v[1]);
      v[2] = fmaf(a.z, wt[i], v[2]); v[3] = fmaf(a.w, wt[i], v[3]);
      v[4] = fmaf(b.x, wt[i], v[4]); v[5] = fmaf(b.y, wt[i], v[5]);
      v[6] = fmaf(b.z, wt[i], v[6]); v[7] = fmaf(b.w, wt[i], v[7]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= inv;
    if (w.pieces > 1) {
      float4* dst = reinterpret_cast<float4*>(p.part + (int64_t(w.slot) * kRowsM + row) * D + d);
      dst[0] = make_float4(v[0], v[1], v[2], v[3]);
      dst[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint16_t* dst = static_cast<uint16_t*>(p.o) + int64_t(w.row0 + tok) * p.o_ss + int64_t(w.hkv) * p.o_sh +
                      int64_t(h) * p.o_sq + d;
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]),
                                                  pack2<T>(v[6], v[7]));
    }
  }
  if (sub == 0) {
    if (w.pieces > 1)
      p.part_lse[int64_t(w.slot) * kRowsM + row] = lse2;
    else if (p.lse)
      p.lse[int64_t(w.hkv * p.g + h) * p.chunk.T + w.row0 + tok] = lse2 * 0.69314718055994531f;
  }
}

// ---------------------------------------------------------------- many rows
// The forward kernel's pipeline (attn_fwd.cu) over pages: warp 0 TMA producer
// (Q once, K and V rings), warp 1 MMA issuer, warps 4-7 and 8-11 softmax and
// epilogue of the two 128-row tiles.  A tile's rows are tpt = 128 / g tokens
// times the g heads of one kv head, token-major, so a short chunk fills its
// rows with heads and every K/V tile feeds all heads that share it.
constexpr int kTThreads = 384;
constexpr int kLaunchRegs = 168;           // 128*72 + 256*216 = 384*168 after setmaxnreg
constexpr float kRescaleThreshold = 8.0f;  // log2 units: rescale O only if the max grows by > 2^8
constexpr int kFmaExpPairs = 5;            // of every 16 column pairs, this many use exp2_fma2
constexpr int kKStages = 3;
constexpr int kVStages = 2;

template <int D>
struct TilesSmem {
  static constexpr int kTileElems = 128 * D;
  alignas(1024) uint16_t q[2][kTileElems];
  alignas(1024) uint16_t k[kKStages][kTileElems];
  alignas(1024) uint16_t v[kVStages][kTileElems];
  uint64_t bar_q;
  uint64_t bar_k_full[kKStages];
  uint64_t bar_k_empty[kKStages];
  uint64_t bar_v_full[kVStages];
  uint64_t bar_v_empty[kVStages];
  uint64_t bar_s_full[2];
  uint64_t bar_p_half[2];
  uint64_t bar_p_ready[2];
  uint64_t bar_o_final[2];
  uint32_t tmem_base;
  int abort_flag;
  int end;
  PlanSmem<kTThreads> plan;
};

// Instruction descriptor of kind::f16 with fp16 (type bits 0) or bf16 inputs.
template <class T>
__host__ __device__ constexpr uint32_t idesc16(int M, int N, int a_mn, int b_mn) {
  return idesc_bf16_f32(M, N, a_mn, b_mn) & ~(std::is_same<T, __half>::value ? (1u << 7) | (1u << 10) : 0u);
}

template <class T, int D>
__device__ __forceinline__ void issue_qk(uint32_t tS, uint64_t qdesc, uint64_t kdesc) {
  constexpr uint32_t idesc = idesc16<T>(128, 128, 0, 0);
  constexpr KMajorSteps<D / 16> st(16384);
  mma_chain_ss_w<D / 16>(tS, qdesc, st.v, kdesc, st.v, idesc, 0u);
}

template <class T, int D>
__device__ __forceinline__ void issue_pv_half(uint32_t tO, uint32_t tP, uint64_t vdesc, int half, bool accumulate) {
  constexpr uint32_t idesc = idesc16<T>(128, D, 0, 1);
  constexpr MNMajorSteps<4> st;
  mma_chain_ts_w<4>(tO, tP + uint32_t(half * 32), 8u, vdesc + uint64_t(half * (4 * 2048 >> 4)), st.v, idesc,
                    accumulate ? 1u : 0u);
}

template <class T, bool kFma, int C0, int C1>
__device__ __forceinline__ void exp_pack(const uint32_t (&sr)[128], float2 cs2, float2 nm2, uint32_t (&pk)[64],
                                         float2 (&ls)[2]) {
#pragma unroll
  for (int c = C0; c < C1; ++c) {
    const float2 x = __ffma2_rn(make_float2(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1])), cs2, nm2);
    const float2 pv = (kFma && (c & 15) < kFmaExpPairs) ? exp2_fma2(x)
                                                        : make_float2(ex2_approx(x.x), ex2_approx(x.y));
    ls[c & 1] = __fadd2_rn(ls[c & 1], pv);
    pk[c] = pack2<T>(pv.x, pv.y);
  }
}

template <class T, int D>
__global__ void __launch_bounds__(kTThreads, 1)
    attn_cache_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const CacheAttn p) {
  extern __shared__ uint8_t smem_raw[];
  TilesSmem<D>& sm =
      *reinterpret_cast<TilesSmem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&sm.bar_q, 1);
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&sm.bar_k_full[i], 1);
      mbar_init(&sm.bar_k_empty[i], 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&sm.bar_v_full[i], 1);
      mbar_init(&sm.bar_v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.bar_s_full[i], 1);
      mbar_init(&sm.bar_p_half[i], 4);   // one arrival per softmax warp
      mbar_init(&sm.bar_p_ready[i], 4);
      mbar_init(&sm.bar_o_final[i], 1);
    }
    sm.abort_flag = 0;
    sm.end = 0;
    fence_barrier_init();
  }
  if (!plan_find<kTThreads, false>(p, sm.plan, blockIdx.x)) return;  // ends with __syncthreads
  const Work w = sm.plan.work;
  const int tok0 = w.tile * 2 * p.tpt;
  const int n_tiles = w.n - tok0 > p.tpt ? 2 : 1;
  // the row of a softmax thread: its last visible position (rows that are no
  // row of the sequence count as seeing everything, and are never stored)
  const int t = warp >= 8 ? 1 : 0, quarter = warp & 3, r = quarter * 32 + lane;
  int tok = 0, head = 0;
  bool valid = false;
  int lim = 0x7fffffff;
  if (warp >= 4) {
    tok = tok0 + t * p.tpt + r / p.g;
    head = r % p.g;
    valid = r < p.tpt * p.g && tok < w.n;
    if (valid) lim = row_limit(p, w, tok);
    const int e = __reduce_max_sync(0xffffffffu, valid ? lim + 1 : 0);
    if (lane == 0) atomicMax(&sm.end, e);
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const int end = sm.end;  // the tile's keys are [0, end)
  int u0, n_vis;
  piece_range(w, (end + kUnit - 1) / kUnit, u0, n_vis);
  n_vis -= u0;
  const WaitCtx wc{&sm.abort_flag, p.chunk.status, kTimeoutNs};

  if (warp < 4) {
    regs_dec<72>();
    if (warp == 0) {
      // =============================== TMA producer: lane l copies box l of a
      // tile, (64-wide column block l % (D/64)) of page l / (D/64)
      if (n_vis > 0) {
        const int box = min(1 << p.chunk.page_shift, 128), n_box = 128 / box;
        const int col = lane % (D / 64), pg = lane / (D / 64);
        if (lane == 0) {
          tma_prefetch_desc(&tm_q);
          tma_prefetch_desc(&tm_k);
          tma_prefetch_desc(&tm_v);
          mbar_arrive_expect_tx(&sm.bar_q, uint32_t(p.tpt * p.g) * D * 2 * n_tiles);
          for (int i = 0; i < n_tiles; ++i)
            for (int c = 0; c < D / 64; ++c)
              tma_load_4d(&sm.q[i][c * 128 * 64], &tm_q, &sm.bar_q, c * 64, 0, w.hkv, w.row0 + tok0 + i * p.tpt);
        }
        int kiss = 0, viss = 0;
        for (int j = 0; j < n_vis; ++j) {
          const int ks = j % kKStages, vs = j % kVStages;
          const int key = (u0 + j) * 128 + pg * box;  // first key of this lane's box
          const bool mine = pg < n_box && key < end;
          const int page = mine ? chunk_page(p.chunk, w.b, key >> p.chunk.page_shift) : 0;
          const int slot = key & ((1 << p.chunk.page_shift) - 1);
          const uint32_t bytes = uint32_t(min(n_box, (end - (u0 + j) * 128 + box - 1) / box)) * box * D * 2;
          if (j >= kKStages &&
              !__all_sync(0xffffffffu, mbar_wait(&sm.bar_k_empty[ks], ((j / kKStages) - 1) & 1, wc)))
            break;
          if (lane == 0) mbar_arrive_expect_tx(&sm.bar_k_full[ks], bytes);
          __syncwarp();
          if (mine)
            tma_load_4d(&sm.k[ks][col * 128 * 64 + pg * box * 64], &tm_k, &sm.bar_k_full[ks], col * 64, slot, w.hkv,
                        page);
          kiss = j + 1;
          if (j >= kVStages &&
              !__all_sync(0xffffffffu, mbar_wait(&sm.bar_v_empty[vs], ((j / kVStages) - 1) & 1, wc)))
            break;
          if (lane == 0) mbar_arrive_expect_tx(&sm.bar_v_full[vs], bytes);
          __syncwarp();
          if (mine)
            tma_load_4d(&sm.v[vs][col * 128 * 64 + pg * box * 64], &tm_v, &sm.bar_v_full[vs], col * 64, slot, w.hkv,
                        page);
          viss = j + 1;
        }
        __syncwarp();
        // Drain: the copies this CTA issued must land before its shared memory
        // can be released, whatever the consumers did.
        mbar_wait_hw(&sm.bar_q, 0, wc);
        for (int j = max(kiss - kKStages, 0); j < kiss; ++j)
          mbar_wait_hw(&sm.bar_k_full[j % kKStages], (j / kKStages) & 1, wc);
        for (int j = max(viss - kVStages, 0); j < viss; ++j)
          mbar_wait_hw(&sm.bar_v_full[j % kVStages], (j / kVStages) & 1, wc);
      }
    } else if (warp == 1) {
      // =============================== MMA issuer (order as in attn_fwd.cu)
      if (n_vis > 0) {
        const uint32_t tS[2] = {tmem, tmem + 128};
        const uint32_t tO[2] = {tmem + 256, tmem + 256 + D};
        const uint64_t qd[2] = {sdesc_sw128(smem_u32(sm.q[0]), 16, 1024), sdesc_sw128(smem_u32(sm.q[1]), 16, 1024)};
        const uint64_t kd0 = sdesc_sw128(smem_u32(sm.k[0]), 16, 1024);
        const uint64_t vd0 = sdesc_sw128(smem_u32(sm.v[0]), 16384, 1024);
        constexpr uint32_t kStageStep = (128u * D * 2u) >> 4;
        bool ok = __all_sync(0xffffffffu, mbar_wait(&sm.bar_q, 0, wc) && mbar_wait(&sm.bar_k_full[0], 0, wc));
        if (ok) {
          for (int i = 0; i < n_tiles; ++i) {
            issue_qk<T, D>(tS[i], qd[i], kd0);
            tc_commit_w(&sm.bar_s_full[i]);
          }
          tc_commit_w(&sm.bar_k_empty[0]);
        }
        for (int j = 0; ok && j < n_vis; ++j) {
          const int vs = j % kVStages, ks1 = (j + 1) % kKStages;
          const bool more = j + 1 < n_vis;
          for (int i = 0; i < n_tiles; ++i) {
            if (i == 0) {
              ok = __all_sync(0xffffffffu, mbar_wait(&sm.bar_v_full[vs], (j / kVStages) & 1, wc) &&
                                               (!more || mbar_wait(&sm.bar_k_full[ks1], ((j + 1) / kKStages) & 1, wc)));
              if (!ok) break;
              // Values at or past the tile's last visible key (the rest of the
              // sequence's last page, pages that were not loaded) may be
              // anything, and a weight of zero does not silence a NaN: clear them.
              const int held = end - (u0 + j) * 128;
              if (held < 128) {
                for (int c = held * 8 + lane; c < 128 * 8; c += 32)
#pragma unroll
                  for (int h = 0; h < D / 64; ++h)
                    *reinterpret_cast<uint4*>(&sm.v[vs][h * 128 * 64 + c * 8]) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
              }
            }
            if (!__all_sync(0xffffffffu, mbar_wait(&sm.bar_p_half[i], j & 1, wc))) { ok = false; break; }
            tc_fence_after();
            issue_pv_half<T, D>(tO[i], tS[i], vd0 + uint32_t(vs) * kStageStep, 0, j > 0);
            if (!__all_sync(0xffffffffu, mbar_wait(&sm.bar_p_ready[i], j & 1, wc))) { ok = false; break; }
            tc_fence_after();
            issue_pv_half<T, D>(tO[i], tS[i], vd0 + uint32_t(vs) * kStageStep, 1, true);
            if (more) {
              issue_qk<T, D>(tS[i], qd[i], kd0 + uint32_t(ks1) * kStageStep);
              tc_commit_w(&sm.bar_s_full[i]);
            }
          }
          if (!ok) break;
          tc_commit_w(&sm.bar_v_empty[vs]);
          if (more) tc_commit_w(&sm.bar_k_empty[ks1]);
        }
        for (int i = 0; i < 2; ++i) tc_commit_w(&sm.bar_o_final[i]);
        mbar_wait_hw(&sm.bar_o_final[0], 0, wc);
      }
    }
  } else {
    regs_inc<216>();
    // =============================== softmax / epilogue; tcgen05.ld/st are
    // warp-collective: every branch around them is warp-uniform
    const bool active = t < n_tiles;
    const uint32_t lane_off = uint32_t(quarter * 32) << 16;
    const uint32_t tS = tmem + uint32_t(t * 128) + lane_off;
    const uint32_t tO = tmem + 256u + uint32_t(t * D) + lane_off;
    const int low = __reduce_min_sync(0xffffffffu, lim);  // every row of the warp sees the keys <= low
    const float cs = p.scale_log2;
    float m = -INFINITY, l = 0.f;
    bool ok = active;
    for (int j = 0; ok && j < n_vis; ++j) {
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.bar_s_full[t], j & 1, wc));
      if (!ok) break;
      tc_fence_after();
      uint32_t sr[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
      tmem_ld_wait_regs(sr);
      const int k0 = (u0 + j) * 128;
      const bool full = k0 + 127 <= low && k0 + 128 <= end;
      if (!full) {
        const int last = min(lim, end - 1) - k0;  // key k0 + c is visible iff c <= last
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c > last) sr[c] = __float_as_uint(-INFINITY);
      }
      __syncwarp();
      float mp[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) mp[c] = __uint_as_float(sr[c]);
#pragma unroll
      for (int c = 8; c < 128; c += 16)
#pragma unroll
        for (int k = 0; k < 8; ++k) mp[k] = fmax3(mp[k], __uint_as_float(sr[c + k]), __uint_as_float(sr[c + 8 + k]));
      const float xmax = fmaxf(fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])),
                               fmaxf(fmaxf(mp[4], mp[5]), fmaxf(mp[6], mp[7]))) * cs;
      // Lazy rescale of O, by selects.  A row that has seen no key yet has m =
      // -inf: its O and l are 0 and any first maximum "grows" it with f = 0.
      float f = 1.f;
      bool rescale = false;
      if (j == 0) {
        m = xmax;
      } else {
        const bool grow = xmax > m + kRescaleThreshold;
        rescale = __any_sync(0xffffffffu, grow);
        const float fg = ex2_approx(m - xmax);
        f = grow ? fg : 1.f;
        m = grow ? xmax : m;
      }
      const float sub = m == -INFINITY ? 0.f : m;
      uint32_t pk[64];
      float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      const float2 cs2 = make_float2(cs, cs), nm2 = make_float2(-sub, -sub);
      if (full)
        exp_pack<T, true, 0, 32>(sr, cs2, nm2, pk, ls);
      else
        exp_pack<T, false, 0, 32>(sr, cs2, nm2, pk, ls);
      tmem_st32(tS, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
      if (rescale) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32(tO + c * 32, ov);
          tmem_ld_wait_regs(ov);
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * f);
          tmem_st32(tO + c * 32, ov);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.bar_p_half[t]);
      if (full)
        exp_pack<T, true, 32, 64>(sr, cs2, nm2, pk, ls);
      else
        exp_pack<T, false, 32, 64>(sr, cs2, nm2, pk, ls);
      l = l * f + ((ls[0].x + ls[1].x) + (ls[0].y + ls[1].y));
      tmem_st32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.bar_p_ready[t]);
    }
    // ---- epilogue
    if (active) {
      bool have = n_vis > 0 && ok;
      if (have) have = __all_sync(0xffffffffu, mbar_wait(&sm.bar_o_final[t], 0, wc));
      if (have) tc_fence_after();
      const bool some = have && l > 0.f;
      const float inv = some ? 1.f / l : 0.f;
      const float lse2 = some ? m + __log2f(l) : -INFINITY;
      if (w.pieces > 1) {  // normalised partial row, fp32
        const int64_t row = int64_t(w.slot) * kTilesM + t * 128 + r;
        float* dst = p.part + row * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          if (have) {
            tmem_ld32(tO + c * 32, ov);
            tmem_ld_wait_regs(ov);
          }
          if (valid) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<float4*>(dst + c * 32)[i] =
                  some ? make_float4(__uint_as_float(ov[4 * i]) * inv, __uint_as_float(ov[4 * i + 1]) * inv,
                                     __uint_as_float(ov[4 * i + 2]) * inv, __uint_as_float(ov[4 * i + 3]) * inv)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
        if (valid) p.part_lse[row] = lse2;
      } else {
        // bf16 / fp16 rows staged in this tile's Q buffer (every MMA has
        // finished), 16-byte chunks XOR-swizzled by row, then written whole
        constexpr int CPR = D / 8;
        uint8_t* tile = reinterpret_cast<uint8_t*>(sm.q[t]);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          if (have) {
            tmem_ld32(tO + c * 32, ov);
            tmem_ld_wait_regs(ov);
          }
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            pk[i] = some ? pack2<T>(__uint_as_float(ov[2 * i]) * inv, __uint_as_float(ov[2 * i + 1]) * inv) : 0u;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int ch = (c * 4 + i) ^ (r & (CPR - 1));
            *reinterpret_cast<uint4*>(tile + r * (D * 2) + ch * 16) =
                make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
          }
        }
        __syncwarp();
        constexpr int RPI = 32 / CPR;  // rows per warp store
        const int ch = lane % CPR;
#pragma unroll 4
        for (int rr = 0; rr < 32; rr += RPI) {
          const int row = quarter * 32 + rr + lane / CPR;
          const int tk = tok0 + t * p.tpt + row / p.g;
          if (row < p.tpt * p.g && tk < w.n) {
            const uint4 x = *reinterpret_cast<const uint4*>(tile + row * (D * 2) + ((ch ^ (row & (CPR - 1))) * 16));
            uint16_t* dst = static_cast<uint16_t*>(p.o) + int64_t(w.row0 + tk) * p.o_ss + int64_t(w.hkv) * p.o_sh +
                            int64_t(row % p.g) * p.o_sq + ch * 8;
            *reinterpret_cast<uint4*>(dst) = x;
          }
        }
        if (valid && p.lse)
          p.lse[int64_t(w.hkv * p.g + head) * p.chunk.T + w.row0 + tok] = lse2 * 0.69314718055994531f;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- join
// Row of a split item: O = sum_i O_i 2^(lse_i - max) / sum_i 2^(lse_i - max)
// over its pieces, in piece order.  A block takes 16 rows of one split item,
// 8 threads a row.
template <class T, int D>
__global__ void __launch_bounds__(128) attn_cache_join_kernel(const CacheAttn p) {
  __shared__ PlanSmem<128> plan;
  if (!plan_find<128, true>(p, plan, blockIdx.x)) return;
  const Work w = plan.work;
  const int tile_rows = p.tpt ? kTilesM : kRowsM;
  const int r = blockIdx.y * 16 + (threadIdx.x >> 3), sub = threadIdx.x & 7;
  int tok, head;
  if (p.tpt) {
    tok = w.tile * 2 * p.tpt + (r >> 7) * p.tpt + (r & 127) / p.g;
    head = (r & 127) % p.g;
    if ((r & 127) >= p.tpt * p.g || tok >= w.n) return;
  } else {
    const int64_t flat = int64_t(w.tile) * kRowsM + r;
    if (flat >= int64_t(w.n) * p.g) return;
    tok = int(flat / p.g);
    head = int(flat % p.g);
  }
  float top = -INFINITY;
  for (int i = 0; i < w.pieces; ++i)
    top = fmaxf(top, __ldcg(p.part_lse + int64_t(w.slot + i * p.Hkv) * tile_rows + r));
  float sum = 0.f, v[D / 8];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) v[i] = 0.f;
  if (top != -INFINITY) {
    for (int i = 0; i < w.pieces; ++i) {
      const int64_t row = int64_t(w.slot + i * p.Hkv) * tile_rows + r;
      const float wt = ex2_approx(__ldcg(p.part_lse + row) - top);
      sum += wt;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const float4* x = reinterpret_cast<const float4*>(p.part + row * D + c * 64 + sub * 8);
        const float4 a = __ldcg(x), b = __ldcg(x + 1);
        float* o = v + c * 8;
        o[0] = fmaf(a.x, wt, o[0]); o[1] = fmaf(a.y, wt, o[1]); o[2] = fmaf(a.z, wt, o[2]); o[3] = fmaf(a.w, wt, o[3]);
        o[4] = fmaf(b.x, wt, o[4]); o[5] = fmaf(b.y, wt, o[5]); o[6] = fmaf(b.z, wt, o[6]); o[7] = fmaf(b.w, wt, o[7]);
      }
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    const float* o = v + c * 8;
    uint16_t* dst = static_cast<uint16_t*>(p.o) + int64_t(w.row0 + tok) * p.o_ss + int64_t(w.hkv) * p.o_sh +
                    int64_t(head) * p.o_sq + c * 64 + sub * 8;
    *reinterpret_cast<uint4*>(dst) =
        make_uint4(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv),
                   pack2<T>(o[4] * inv, o[5] * inv), pack2<T>(o[6] * inv, o[7] * inv));
  }
  if (sub == 0 && p.lse)
    p.lse[int64_t(w.hkv * p.g + head) * p.chunk.T + w.row0 + tok] =
        sum > 0.f ? (top + __log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

// ---------------------------------------------------------------- host side
size_t a256(size_t x) { return (x + 255) & ~size_t(255); }

int sm_count() {
  static PerContext<int> cache;
  int n = 0;
  if (cache.get(&n, [](int* out) {
        int dev = 0;
        const cudaError_t e = cudaGetDevice(&dev);
        return e != cudaSuccess ? e : cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
      }) != cudaSuccess)
    return 148;
  return n;
}

struct Launch {
  bool tiles;       // attn_cache_tiles, or attn_cache_rows
  int cta_slots, max_slots, rows;
  int64_t items;    // upper bound
  size_t part, lse, total;
};

// The tiles kernel when an average chunk has more than 16 rows per kv head.
Launch plan_launch(const hia_cache& c, const hia_cache_chunk& k, int64_t T, int g) {
  Launch L{};
  const int n_sm = sm_count();
  const int64_t B = std::max<int64_t>(1, std::min<int64_t>(k.B, T));
  L.tiles = T * g > 16 * B;
  L.rows = L.tiles ? kTilesM : kRowsM;
  L.cta_slots = L.tiles ? n_sm : 2 * n_sm;
  L.max_slots = 2 * L.cta_slots;
  const int tpt = 128 / g;
  L.items = (L.tiles ? T / (2 * tpt) + B : T * g / kRowsM + B) * c.Hkv;
  L.part = 0;
  L.lse = a256(size_t(L.max_slots) * L.rows * c.D * 4);
  L.total = L.lse + a256(size_t(L.max_slots) * L.rows * 4);
  return L;
}

bool attn_args_ok(const hia_cache* c, const hia_cache_chunk* k, int64_t T, int Hq, int* rc) {
  *rc = cache_check(c, k, T, Hq);
  if (*rc == HIA_OK && Hq / c->Hkv > 128) *rc = HIA_ERR_UNSUPPORTED;
  return *rc == HIA_OK;
}

template <class K>
cudaError_t smem_optin(PerContext<int>& c, K kernel, size_t bytes, int regs) {
  int done = 0;
  return c.get(&done, [&](int* out) {
    *out = 1;
    if (regs) {  // the setmaxnreg split assumes this register count
      cudaFuncAttributes fa{};
      const cudaError_t e = cudaFuncGetAttributes(&fa, reinterpret_cast<const void*>(kernel));
      if (e != cudaSuccess) return e;
      if (fa.numRegs != regs) return cudaErrorInvalidConfiguration;
    }
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                int(bytes));
  });
}

template <class T, int D>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CacheAttn& p,
                   const Launch& L, cudaStream_t st) {
  const int64_t grid = L.items + L.max_slots;
  if (L.tiles) {
    static_assert(sizeof(TilesSmem<D>) + 1024 <= 232448, "shared memory budget");
    constexpr size_t smem = sizeof(TilesSmem<D>) + 1024;
    static PerContext<int> ready;
    const cudaError_t e = smem_optin(ready, attn_cache_tiles_kernel<T, D>, smem, kLaunchRegs);
    if (e != cudaSuccess) return e;
    prof_begin(kAttnCacheTiles, st);
    attn_cache_tiles_kernel<T, D><<<int(grid), kTThreads, smem, st>>>(tq, tk, tv, p);
    prof_end(kAttnCacheTiles, st);
  } else {
    static_assert(2 * (sizeof(RowsSmem<D>) + 1024 + 1024) <= 233472, "two blocks an SM");
    constexpr size_t smem = sizeof(RowsSmem<D>) + 1024;
    static PerContext<int> ready;
    const cudaError_t e = smem_optin(ready, attn_cache_rows_kernel<T, D>, smem, 0);
    if (e != cudaSuccess) return e;
    prof_begin(kAttnCacheRows, st);
    attn_cache_rows_kernel<T, D><<<int(grid), kRThreads, smem, st>>>(tk, tv, p);
    prof_end(kAttnCacheRows, st);
  }
  prof_begin(kAttnCacheJoin, st);
  attn_cache_join_kernel<T, D><<<dim3(L.max_slots / 2, L.rows / 16), 128, 0, st>>>(p);
  prof_end(kAttnCacheJoin, st);
  return cudaGetLastError();
}

}  // namespace
}  // namespace hia

extern "C" size_t hia_attn_cache_workspace_bytes(const hia_cache* c, const hia_cache_chunk* k, int64_t T, int Hq) {
  int rc;
  if (!hia::attn_args_ok(c, k, T, Hq, &rc)) return 0;
  return hia::plan_launch(*c, *k, T, Hq / c->Hkv).total;
}

extern "C" int hia_attn_cache_fwd(const hia_cache* c, const hia_cache_chunk* k, int64_t T, int Hq, hia_tensor q,
                                  const int32_t* bound, float scale, hia_tensor o, float* lse, void* ws,
                                  size_t ws_bytes, void* stream) {
  using namespace hia;
  int rc;
  if (!attn_args_ok(c, k, T, Hq, &rc)) return rc;
  if (!std::isfinite(scale) || !(scale > 0.f)) return HIA_ERR_INVALID_ARG;
  if (T == 0 || k->B == 0) return HIA_OK;
  if (!q.ptr || !o.ptr || !ws) return HIA_ERR_INVALID_ARG;
  const int g = Hq / c->Hkv, D = c->D;
  if ((rc = rows_check(q, true, g, 2)) || (rc = rows_check(o, true, g, 2))) return rc;
  if (!aligned_to(bound, 4) || !aligned_to(lse, 4)) return HIA_ERR_UNSUPPORTED;
  const Launch L = plan_launch(*c, *k, T, g);
  if (ws_bytes < L.total || !aligned_to(ws, 256)) return HIA_ERR_INVALID_ARG;
  if (L.items + L.max_slots >= (int64_t(1) << 31)) return HIA_ERR_UNSUPPORTED;
  int* status = device_status_word();
  if (!status) return HIA_ERR_CUDA;
  CacheAttn p{};
  p.chunk = chunk_dev(*c, *k, T, status);
  p.q = q.ptr;
  p.q_ss = q.stride_s;
  p.q_sh = q.stride_hkv;
  p.q_sq = q.stride_hq;
  p.o = o.ptr;
  p.o_ss = o.stride_s;
  p.o_sh = o.stride_hkv;
  p.o_sq = o.stride_hq;
  p.lse = lse;
  p.bound = bound;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.Hkv = c->Hkv;
  p.g = g;
  p.tpt = L.tiles ? 128 / g : 0;
  p.cta_slots = L.cta_slots;
  p.max_slots = L.max_slots;
  p.piece_cost = L.tiles ? 2.f : 1.f;
  p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + L.part);
  p.part_lse = reinterpret_cast<float*>(static_cast<char*>(ws) + L.lse);

  // pages as (D, page_size, Hkv, n_pages); a box is 64 columns of the rows of
  // one page that a step or tile takes
  const uint32_t box_rows = uint32_t(std::min(c->page_size, L.tiles ? 128 : 16));
  CUtensorMap tq{}, tk, tv;
  const uint64_t kd[4] = {uint64_t(D), uint64_t(c->page_size), uint64_t(c->Hkv), uint64_t(c->n_pages)};
  const uint64_t ks[3] = {uint64_t(c->stride_s) * 2, uint64_t(c->Hkv > 1 ? c->stride_h : D) * 2,
                          uint64_t(c->n_pages > 1 ? c->stride_page : D) * 2};
  const uint32_t kbox[4] = {64, box_rows, 1, 1};
  if (!make_map_nd(&tk, c->k, 4, kd, ks, kbox) || !make_map_nd(&tv, c->v, 4, kd, ks, kbox)) return HIA_ERR_UNSUPPORTED;
  if (L.tiles) {
    const uint64_t qd[4] = {uint64_t(D), uint64_t(g), uint64_t(c->Hkv), uint64_t(T)};
    const uint64_t qs[3] = {uint64_t(g > 1 ? q.stride_hq : D) * 2, uint64_t(c->Hkv > 1 ? q.stride_hkv : D) * 2,
                            uint64_t(T > 1 ? q.stride_s : D) * 2};
    const uint32_t qbox[4] = {64, uint32_t(g), 1, uint32_t(p.tpt)};
    if (!make_map_nd(&tq, q.ptr, 4, qd, qs, qbox)) return HIA_ERR_UNSUPPORTED;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (c->dtype == HIA_BF16)
    e = D == 128 ? launch<__nv_bfloat16, 128>(tq, tk, tv, p, L, st) : launch<__nv_bfloat16, 64>(tq, tk, tv, p, L, st);
  else
    e = D == 128 ? launch<__half, 128>(tq, tk, tv, p, L, st) : launch<__half, 64>(tq, tk, tv, p, L, st);
  return e == cudaSuccess ? HIA_OK : HIA_ERR_CUDA;
}
