// attn_cache.cu -- attention of chunks of new tokens over the paged key/value
// cache (hia_attn_cache_fwd), bf16 and fp16, head dimension 64 and 128.
//
// Definition: row (t, h) of sequence b, bound e: O = sum_{j <= e} p_j v_j / l,
// p_j = exp(scale q . k_j - m), l = sum p_j, lse = m + log l, with the running
// maximum m and sum l of an online softmax in fp32.  Scores, statistics, outputs
// and the partials of split items stay in fp32.  Two roundings to 16 bits: the
// weights p_j, because the products with V take their operands in the cache's type
// (each off by half a step, against sums of the unrounded ones), and O at the end.
// fp16 has no exponents for weights far below the largest, and a long cache can
// hold many of them, so its m is kept some powers of two below the maximum
// (Fp16Weights): weights go up to 2^15, the factor cancels in O / l and in m + log l, and
// half a step holds down to 2^-25 (few rows: 2^-28) of a row's largest weight; below,
// the error is at most half a step there, 2^-36 (2^-39) of the largest weight.
//
// Two kernels, for the two things that bound this operator:
//   attn_cache_rows   few rows per sequence (single tokens): the time is that
//                     of reading K and V once.  Warp-private streams of key
//                     steps, mma.sync on 16 rows.
//   attn_cache_tiles  many rows: the products bound it.  tcgen05 on two
//                     128-row tiles, one persistent CTA per SM.
// attn_cache_plan, one block, goes before either.  The lengths and bounds are
// only known on the device (they change between replays of a captured graph),
// so it lists the row tiles with the keys each sees, and cuts the line of all
// items (sequence, kv head, row tile) into one equal stretch of work per
// resident CTA.  An item that a cut falls into is computed in pieces: each
// writes a normalised fp32 partial, and whichever piece finishes last
// (attn_cache_rows) or attn_cache_join (for attn_cache_tiles) adds them in key
// order: the result is the same at every run.
#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "cache.cuh"
#include "devctx.h"

namespace hia {
namespace {

constexpr int kUnit = 128;  // keys per unit of work
constexpr uint64_t kTimeoutNs = 2000000000ull;

// Rows of an item: the rows kernel takes 16 consecutive (token, head of the
// group) rows, the tiles kernel 2 x tpt tokens with all g heads each.
constexpr int kRowsM = 16;
constexpr int kTilesM = 256;

// A row tile of one sequence, for every kv head: the keys [0, end) it sees.
struct Tile {
  int b, tile, row0, n, past, end;
  int nt, low;  // row tiles it reaches (tiles kernel); every row of it sees the keys [0, low]
};

// The start of a CTA's stretch of the line: unit u of item (tile index tau, kv
// head hkv).  owner: if u > 0, the CTA that has the item's first piece.
struct Cut {
  int tau, hkv, u, owner;
};

// A split item: its pieces (1: there is none), and whose rows they are.
struct Join {
  int pieces, hkv, tile, row0, n, pad0, pad1, pad2;
};

struct PlanWs {  // device workspace written by attn_cache_plan
  int* head;           // [2]: whole items that each CTA takes first; row tiles
  Cut* cuts;           // [ctas + 1]
  Join* joins;         // [ctas]: the split item whose first piece is this CTA's last one
  int* arrived;        // [ctas]: pieces of it that are written (zeroed by the plan)
  int* first;          // [B + 1]: first tile index of each sequence
  Tile* tiles;         // [max_tiles]
  long long* cum;      // [max_tiles + 1]: cost of all tiles before this one, for one kv head
};

struct CacheAttn {
  ChunkDev chunk;
  PlanWs ws;
  const void* q;  // rows kernel only (the tiles kernel has a tensor map)
  int64_t q_ss, q_sh, q_sq;
  const void* v;  // tiles kernel: pages, for values that are not finite
  int64_t v_sp, v_ss, v_sh;
  void* o;
  int64_t o_ss, o_sh, o_sq;
  float* lse;            // [Hq][T], or nullptr
  const int32_t* bound;  // [T], or nullptr: causal
  float scale_log2;
  int Hkv, g;
  int tpt;         // tiles kernel: tokens per 128-row tile; 0: rows kernel
  int ctas;        // resident CTAs: stretches of the plan
  int max_tiles;
  int item_cost;   // fixed cost of an item, in positions (rows kernel: units)
  int wide_o;      // o rows are 32-byte aligned
  float* part;     // [2 * ctas][rows of a tile][D]: normalised partials; CTA c: slot 2c the piece its stretch starts in, 2c + 1 the one it ends in
  // [2 * ctas][rows of a tile]: their m and l (apart: m + log l in one fp32 would
  // lose the share of a piece where |m| is large)
  float2* part_ml;
};

__device__ __forceinline__ long long seq_tiles(const CacheAttn& p, int n) {
  if (p.tpt) return (n + 2 * p.tpt - 1) / (2 * p.tpt);
  return (int64_t(n) * p.g + kRowsM - 1) / kRowsM;
}

// Units of a tile's keys; a tile that sees nothing still counts one, without
// keys, in which its empty rows are written.
__device__ __forceinline__ int units_of(int end) { return max(1, (end + kUnit - 1) / kUnit); }

// Last visible position of the row of token i (of the sequence at row0), -1 for none.
__device__ __forceinline__ int row_limit(const CacheAttn& p, int row0, int n, int past, int i) {
  const int e = p.bound ? __ldg(p.bound + row0 + i) : past + i;
  return max(min(e, past + n - 1), -1);
}

// The factor of O (0) of a row without weights (l = 0): such a row sees no key and is empty, or
// all its scores are -inf and exp(-inf - -inf) leaves none: NaN by the formula.  (In
// a piece of a split item it is the other pieces that count, so this is settled
// where a row is written for good.)
__device__ __forceinline__ float no_weights(bool sees) { return sees ? __uint_as_float(0x7fffffffu) : 0.f; }

// ---------------------------------------------------------------- plan
constexpr int kPlanThreads = 512;

// Exclusive scan over the block; *total receives the sum.
__device__ long long block_scan(long long v, long long* total, long long (&warp_s)[kPlanThreads / 32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_s[warp] = x;
  __syncthreads();
  long long w = lane < kPlanThreads / 32 ? warp_s[lane] : 0, z = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, z, o);
    if (lane >= o) z += y;
  }
  *total = __shfl_sync(0xffffffffu, z, 31);
  return x - v + __shfl_sync(0xffffffffu, z - w, warp);
}

// Largest i in [lo, hi) with a[i] <= x (a non-decreasing, a[lo] <= x).
template <class A>
__device__ __forceinline__ int last_at_most(const A* a, int lo, int hi, A x) {
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (a[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// First index in [lo, hi) whose key is at least x (keys in order), or hi.
__device__ __forceinline__ int first_at_least(const long long* key, int lo, int hi, long long x) {
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (key[mid] < x)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

// The line of work: items (hkv, tile) with hkv the slower index, each costing
// its positions (units times row tiles) and a fixed item_cost.  CTA c takes
// whole items c, c + ctas, ... first (head[0] of them; the CTAs that share keys
// then read them at the same time) and then its stretch of the rest of the
// line, which makes all shares of the cost equal.  Whole items first only where
// they are even enough to leave every CTA a stretch; few items are all
// stretches.  One block: its time is latency (loads, scans, searches; 7 us for 48
// sequences, 5 for one), so the tables stay in shared memory while they fit.  (A
// plan inside the kernels, worked out by every CTA for itself, cost each 4 to 6 us;
// here the prologue of the next kernel hides part of it.)
__global__ void __launch_bounds__(kPlanThreads) attn_cache_plan_kernel(const __grid_constant__ CacheAttn p) {
  __shared__ long long warp_s[kPlanThreads / 32];
  __shared__ long long key_s[kPlanThreads + 1];
  __shared__ long long cum_s[kPlanThreads + 1];
  __shared__ int4 seq_s[kPlanThreads];  // row0, n, past, first tile
  __shared__ int4 span_s[kPlanThreads];  // first row of a tile's bounds, their number, the sequence's last position
  __shared__ int2 end_s[kPlanThreads];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31;
  const PlanWs& ws = p.ws;
  const bool cached = p.chunk.B <= kPlanThreads;

  // the tiles of every sequence, one after the other
  long long carry = 0, sum;
  for (int b0 = 0; b0 < p.chunk.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    const Seq s = b < p.chunk.B ? chunk_seq(p.chunk, b) : Seq{0, 0, 0};
    const long long at = carry + block_scan(seq_tiles(p, s.n), &sum, warp_s);
    const int f = int(at < p.max_tiles ? at : p.max_tiles);
    if (cached)
      seq_s[tid] = make_int4(s.row0, s.n, s.past, f);
    else if (b < p.chunk.B)
      ws.first[b] = f;
    carry += sum;
  }
  // (more tiles than rows allow: only with rows that do not fit, and reported)
  const int n_tiles = int(carry < p.max_tiles ? carry : p.max_tiles);
  __syncthreads();

  // the keys that each tile sees, and the cost of the tiles before it
  long long* cum = n_tiles <= kPlanThreads ? cum_s : ws.cum;
  carry = 0;
  for (int i0 = 0; i0 < n_tiles; i0 += kPlanThreads) {
    const int i = i0 + tid;
    Tile t{};
    if (i < n_tiles) {
      int lo = 0, hi = p.chunk.B;  // the last sequence that begins at or before tile i
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((cached ? seq_s[mid].w : ws.first[mid]) <= i)
          lo = mid;
        else
          hi = mid;
      }
      Seq s;
      int f;
      if (cached) {
        const int4 x = seq_s[lo];
        s = Seq{x.x, x.y, x.z};
        f = x.w;
      } else {
        s = chunk_seq(p.chunk, lo);
        f = ws.first[lo];
      }
      int t0, t1;  // its tokens
      if (p.tpt) {
        t0 = (i - f) * 2 * p.tpt;
        t1 = min(t0 + 2 * p.tpt, s.n);
      } else {
        const int64_t r = int64_t(i - f) * kRowsM;
        t0 = int(r / p.g);
        t1 = int(min(int64_t(s.n), (r + kRowsM - 1) / p.g + 1));
      }
      t = Tile{lo, i - f, s.row0, s.n, s.past, s.past + t1, p.tpt && t1 - t0 > p.tpt ? 2 : 1, s.past + t0};
      span_s[tid] = make_int4(s.row0 + t0, t1 - t0, s.past + s.n - 1, 0);
    }
    if (p.bound) {  // 8 lanes read a tile's bounds
      __syncthreads();
      for (int k = tid >> 3; k < min(kPlanThreads, n_tiles - i0); k += kPlanThreads / 8) {
        const int4 x = span_s[k];
        int e = -1, low = x.z;
#pragma unroll 8
        for (int j = lane & 7; j < x.y; j += 8) {
          const int v = max(min(__ldg(p.bound + x.x + j), x.z), -1);
          e = max(e, v);
          low = min(low, v);
        }
        e = __reduce_max_sync(0xffu << (lane & 24), e);
        low = __reduce_min_sync(0xffu << (lane & 24), low);
        if ((lane & 7) == 0) end_s[k] = make_int2(e + 1, low);
      }
      __syncthreads();
      if (i < n_tiles) {
        t.end = end_s[tid].x;
        t.low = end_s[tid].y;
      }
    }
    const long long cost = i < n_tiles ? units_of(t.end) * t.nt + p.item_cost : 0;
    const long long at = carry + block_scan(cost, &sum, warp_s);
    if (i < n_tiles) {
      cum[i] = at;
      ws.tiles[i] = t;
    }
    carry += sum;
  }
  if (tid == 0) cum[n_tiles] = carry;
  __syncthreads();

  // whole items first: rounds of one item per CTA, while no CTA's are worth
  // more than an equal share (less the least stretch)
  const long long head_cost = carry, all = head_cost * p.Hkv, least = p.item_cost + 2;
  const bool small = all < (1ll << 31);  // 32-bit divisions
  const int n_cta = int(all < least * p.ctas ? max(1, int(all) / int(least)) : p.ctas);
  const long long share = small ? unsigned(all) / unsigned(n_cta) : all / n_cta;
  const int over = int(all - share * n_cta);  // the first `over` shares are one larger
  long long mine = 0;                         // the cost of this thread's CTA's whole items
  int rounds = 0;
  if (p.tpt && n_tiles > 0) {
    rounds = int(max(0ll, min((long long)n_tiles * p.Hkv / p.ctas - 1, 1ll << 29)));
    const int step = p.ctas % n_tiles;
    while (rounds > 0) {
      mine = 0;
      if (tid < p.ctas) {
        int tau = tid % n_tiles;
        for (int k = 0; k < rounds; ++k) {
          mine += cum[tau + 1] - cum[tau];
          tau += step;
          if (tau >= n_tiles) tau -= n_tiles;
        }
      }
      if (!__syncthreads_or(mine > share - least)) break;
      rounds >>= 1;
      mine = 0;
    }
  }
  long long before = 0, base_cost = 0;  // cost of the whole items of the CTAs before; of all
  if (rounds > 0) {
    before = block_scan(mine, &base_cost, warp_s);
    // the line's cost up to the first item of the stretches is that of all whole items
  }

  // the cuts: equal shares
  Cut k{0, p.Hkv, 0, -1};  // the end of the line
  if (tid < n_cta && n_tiles > 0) {
    const long long s = base_cost + share * tid + min(tid, over) - before;
    k.hkv = int(small ? unsigned(s) / unsigned(head_cost) : s / head_cost);
    const long long y = s - head_cost * k.hkv;
    if (k.hkv < p.Hkv) {
      k.tau = last_at_most(cum, 0, n_tiles, y);
      const long long x = y - cum[k.tau] - p.item_cost;  // positions of the item before the cut
      k.u = int(max(0ll, x) / (p.tpt ? ws.tiles[k.tau].nt : 1));
    }
  }
  if (tid <= p.ctas) key_s[tid] = (((long long)k.hkv * n_tiles + k.tau) << 24) | k.u;
  if (tid == 0) {
    ws.head[0] = rounds;
    ws.head[1] = n_tiles;
  }
  __syncthreads();
  if (tid < p.ctas) {
    // owner of a cut inside an item: the CTA before the item's first such cut
    // (cuts inside one item differ: they are `least` apart)
    const long long item = key_s[tid] >> 24, next = key_s[tid + 1] >> 24;
    if (k.u > 0) k.owner = first_at_least(key_s, 0, tid, (item << 24) + 1) - 1;
    ws.cuts[tid] = k;
    ws.arrived[tid] = 0;
    // the item that CTA tid begins and does not end
    Join j{1, 0, 0, 0, 0, 0, 0, 0};
    if ((key_s[tid + 1] & 0xffffff) > 0 && key_s[tid] <= (next << 24)) {
      j.pieces = first_at_least(key_s, tid + 1, p.ctas + 1, (next + 1) << 24) - tid;
      j.hkv = int(next / n_tiles);
      const Tile t = ws.tiles[next - (long long)j.hkv * n_tiles];
      j.tile = t.tile;
      j.row0 = t.row0;
      j.n = t.n;
    }
    ws.joins[tid] = j;
  }
  if (tid == p.ctas) ws.cuts[p.ctas] = k;
}

// A CTA's way through its items, piece by piece.
struct Walk {
  int tau, hkv, u0, u1;   // the piece: units [u0, u1)
  int e_tau, e_hkv, e_u;  // the end of the stretch
  int left;               // whole items before the stretch, this one included
  int n_tiles;
  Tile t;

  __device__ __forceinline__ int units() const { return units_of(t.end); }
  __device__ __forceinline__ void load(const CacheAttn& p) {
    const int4* x = reinterpret_cast<const int4*>(p.ws.tiles + tau);
    const int4 a = __ldcg(x);
    const int4 b = __ldcg(x + 1);
    t = Tile{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  }
  __device__ __forceinline__ bool stretch(const CacheAttn& p) {
    const bool at_end = tau == e_tau && hkv == e_hkv;
    if (at_end && e_u <= u0) return false;
    load(p);
    u1 = at_end ? e_u : units();
    return true;
  }
  __device__ __forceinline__ bool start_stretch(const CacheAttn& p) {
    const int4 s = __ldcg(reinterpret_cast<const int4*>(p.ws.cuts + blockIdx.x));
    const int4 e = __ldcg(reinterpret_cast<const int4*>(p.ws.cuts + blockIdx.x + 1));
    tau = s.x;
    hkv = s.y;
    u0 = s.z;
    e_tau = e.x;
    e_hkv = e.y;
    e_u = e.z;
    return stretch(p);
  }
  __device__ __forceinline__ bool item(const CacheAttn& p) {
    while (tau >= n_tiles) {
      tau -= n_tiles;
      ++hkv;
    }
    u0 = 0;
    load(p);
    u1 = units();
    return true;
  }
  __device__ __forceinline__ bool begin(const CacheAttn& p) {
    const int2 h = __ldcg(reinterpret_cast<const int2*>(p.ws.head));
    left = h.x;
    n_tiles = h.y;
    if (left == 0) return start_stretch(p);
    tau = blockIdx.x;
    hkv = 0;
    return item(p);
  }
  __device__ __forceinline__ bool next(const CacheAttn& p) {
    if (left > 0) {
      if (--left == 0) return start_stretch(p);
      tau += gridDim.x;
      return item(p);
    }
    if (tau == e_tau && hkv == e_hkv) return false;  // that was the piece the stretch ends in
    u0 = 0;
    if (++tau == n_tiles) {
      tau = 0;
      ++hkv;
    }
    return stretch(p);
  }
  __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == units(); }
  __device__ __forceinline__ int slot() const { return 2 * blockIdx.x + (u0 > 0 ? 0 : 1); }
};

// A partial of this CTA is written (by the `threads` that meet at barrier
// `bar`): true in all of them if it was the item's last one.
__device__ __forceinline__ bool piece_arrive(const CacheAttn& p, const Walk& w, int bar, int threads, bool one, int* flag,
                                             int* owner, int* pieces) {
  *owner = w.u0 > 0 ? __ldcg(&p.ws.cuts[blockIdx.x].owner) : int(blockIdx.x);
  *pieces = __ldcg(&p.ws.joins[*owner].pieces);
  __threadfence();
  named_bar_sync(bar, threads);
  if (one) *flag = atomicAdd(p.ws.arrived + *owner, 1) == *pieces - 1;
  named_bar_sync(bar, threads);
  __threadfence();
  return *reinterpret_cast<volatile int*>(flag) != 0;
}

template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);

// Row r (of rows_per tile rows) of a split item: O = sum_i O_i w_i / sum_i w_i with
// w_i = l_i 2^(m_i - max) over its pieces in key order; piece i was written by
// CTA owner + i.  8 neighbouring lanes (sub) share a row; (row, head): where it
// goes.
template <class T, int D>
__device__ __forceinline__ void join_row(const CacheAttn& p, int hkv, int owner, int pieces, int rows_per, int r, int sub,
                                      int row, int head) {
  const unsigned group = 0xffu << (threadIdx.x & 24);
  const auto at = [&](int i) { return int64_t(i == 0 ? 2 * owner + 1 : 2 * (owner + i)) * rows_per + r; };
  float top = -INFINITY;
  for (int i = sub; i < pieces; i += 8) top = fmaxf(top, __ldcg(p.part_ml + at(i)).x);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(group, top, o));
  if (top == -INFINITY) top = 0.f;  // no piece has a key, or all are NaN
  float sum = 0.f, v[D / 8];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) v[i] = 0.f;
  for (int i0 = 0; i0 < pieces; i0 += 8) {
    float mine = 0.f;
    if (i0 + sub < pieces) {
      const float2 ml = __ldcg(p.part_ml + at(i0 + sub));
      mine = ex2_approx(ml.x - top) * ml.y;
    }
#pragma unroll
    for (int k0 = 0; k0 < 8; k0 += 4) {
      if (i0 + k0 >= pieces) break;
      float4 x[4][D / 32];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i0 + k0 + k < pieces) {
          const float4* src = reinterpret_cast<const float4*>(p.part + at(i0 + k0 + k) * D + sub * 8);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            x[k][2 * c] = __ldcg(src + c * 16);
            x[k][2 * c + 1] = __ldcg(src + c * 16 + 1);
          }
        }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float wt = __shfl_sync(group, mine, k0 + k, 8);
        if (i0 + k0 + k >= pieces) continue;
        sum += wt;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float* o = v + c * 4;
          o[0] = fmaf(x[k][c].x, wt, o[0]);
          o[1] = fmaf(x[k][c].y, wt, o[1]);
          o[2] = fmaf(x[k][c].z, wt, o[2]);
          o[3] = fmaf(x[k][c].w, wt, o[3]);
        }
      }
    }
  }
  const float none = sum != 0.f ? 0.f : no_weights(!p.bound || __ldg(p.bound + row) >= 0);
  const float inv = sum != 0.f ? 1.f / sum : none;
#pragma unroll
  for (int k = 0; k < D / 64; ++k) {
    const float* o = v + k * 8;
    uint16_t* dst = static_cast<uint16_t*>(p.o) + int64_t(row) * p.o_ss + int64_t(hkv) * p.o_sh +
                    int64_t(head) * p.o_sq + k * 64 + sub * 8;
    *reinterpret_cast<uint4*>(dst) =
        make_uint4(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv),
                   pack2<T>(o[4] * inv, o[5] * inv), pack2<T>(o[6] * inv, o[7] * inv));
  }
  if (sub == 0 && p.lse)
    p.lse[int64_t(hkv * p.g + head) * p.chunk.T + row] =
        sum != 0.f ? (top + __log2f(sum)) * 0.69314718055994531f : none - INFINITY;
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

// fp16 weights: how far below a row's maximum score (log2 units) its m is kept.  In
// the tiles kernel those bits and the lag of the lazy maximum make the 15 that fp16
// has above 1; the rows kernel's m does not lag, and one bit is left for rounding.
// (A lag of 8 would leave 7 bits: weights 2^-23 of the largest off by up to 4 half
// steps.  The shorter lag costs nothing that shows: 2 x 4098 fp16 rows over 5122 keys
// take 698 us back to back, 706 with m at the maximum and a lag of 8.)  Scores in the
// millions, where m is rounded by a unit or more, go without.  bf16 has the exponents
// of fp32 and needs none of it.
template <class T>
struct Fp16Weights {
  static constexpr bool kOn = std::is_same<T, __half>::value;
  static constexpr float kRows = 14.f, kTiles = 11.f;
  static constexpr float kLag = kOn ? 4.f : 8.f;  // rescale O only if the maximum grows by more
  // m of a maximum of x
  static __device__ __forceinline__ float below(float x, float bits) {
    return kOn ? x - (fabsf(x) < 4194304.f ? bits : 0.f) : x;
  }
};

// Two packed elements: as fp32; whether one of them is infinite or a NaN.
template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t x) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
}
template <class T>
__device__ __forceinline__ bool not_finite2(uint32_t x) {
  constexpr uint32_t e = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
  return (x & e) == e || (x & (e << 16)) == (e << 16);
}
// w v for a weight that is positive, though it may have underflowed to 0.
__device__ __forceinline__ float weighted(float w, float v) { return w == 0.f && !isfinite(v) ? v : w * v; }

// ---------------------------------------------------------------- few rows
// What bounds it is reading K and V once: 48 sequences of 64 to 32768 keys, one
// token each (957 MB), take 171 us with the plan, 5.6 TB/s of 6.5.  Two CTAs of
// four warps an SM, each warp with its own ring: 192 KB in flight an SM, and
// neither a barrier nor a wait for another warp inside a piece.  (Stretches that
// CTAs take as they come free, 55 to 80% of the work dealt out first, cost more in
// pieces than the even ends gave: 177 to 209 against 175 us.)
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
  int joins;
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
// warps meet once per piece.  Row r of the tile is row tile*16 + r of the
// sequence's n*g (token, head of the group) rows.
template <class T, int D>
__global__ void __launch_bounds__(kRThreads)
    attn_cache_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ CacheAttn p) {
  constexpr int kKeys = RowsCfg<D>::kKeys, kStages = RowsCfg<D>::kStages;
  extern __shared__ uint8_t smem_raw[];
  RowsSmem<D>& sm = *reinterpret_cast<RowsSmem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    for (int w = 0; w < kRWarps; ++w)
      for (int i = 0; i < kStages; ++i) mbar_init(&sm.full[w][i], 1);
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const WaitCtx wc{&sm.abort_flag, p.chunk.status, kTimeoutNs};
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan is written
  int it = 0;  // key steps of this warp over all pieces: stage it % kStages, phase it / kStages
  Walk w;
  for (bool more = w.begin(p); more; more = w.next(p)) {
    // this thread's rows: lane / 4 and lane / 4 + 8
    const int64_t n_rows = int64_t(w.t.n) * p.g;
    const int end = w.t.end;
    const int key0 = w.u0 * kUnit, key1 = min(w.u1 * kUnit, end);
    const int steps = key1 > key0 ? (key1 - key0 + kKeys - 1) / kKeys : 0;
    const int mine = steps > warp ? (steps - warp + kRWarps - 1) / kRWarps : 0;  // steps warp, warp + 4, ...

    // one lane issues the copies of step i: one box per (K or V, column block);
    // a step never crosses a page (pages hold a multiple of 16 slots)
    int page_reg = 0;  // page of step (i & ~31) + lane
    const auto issue = [&](int i) {
      if ((i & 31) == 0 && i + lane < mine)
        page_reg = chunk_page(p.chunk, w.t.b, (key0 + (warp + (i + lane) * kRWarps) * kKeys) >> p.chunk.page_shift);
      const int page = __shfl_sync(0xffffffffu, page_reg, i & 31);
      if (lane == 0) {
        const int s = (it + i) % kStages;
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

    int lim[2];
    uint32_t qf[D / 16][4];
    int low = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t r = int64_t(w.t.tile) * kRowsM + (lane >> 2) + 8 * i;
      lim[i] = -1;
      if (r < n_rows) {
        const int tok = int(r / p.g), h = int(r % p.g);
        lim[i] = row_limit(p, w.t.row0, w.t.n, w.t.past, tok);
        low = min(low, lim[i]);
        const uint16_t* q = static_cast<const uint16_t*>(p.q) + int64_t(w.t.row0 + tok) * p.q_ss +
                            int64_t(w.hkv) * p.q_sh + int64_t(h) * p.q_sq;
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
    low = __reduce_min_sync(0xffffffffu, low);

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    const float cs = p.scale_log2;

    for (int i = 0; i < mine; ++i) {
      const int s = (it + i) % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.full[warp][s], ((it + i) / kStages) & 1, wc))) break;
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
      uint32_t pf[4];
      float f[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float x = -INFINITY;
#pragma unroll
        for (int n = 0; n < kKeys / 8; ++n) x = fmaxf(x, fmaxf(acc[n][2 * r], acc[n][2 * r + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        const float mn = fmaxf(m[r], Fp16Weights<T>::below(x * cs, Fp16Weights<T>::kRows));
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
      pf[0] = pack2<T>(acc[0][0], acc[0][1]);
      pf[1] = pack2<T>(acc[0][2], acc[0][3]);
      pf[2] = pack2<T>(acc[1][0], acc[1][1]);
      pf[3] = pack2<T>(acc[1][2], acc[1][3]);
      if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          o[n][0] *= f[0];
          o[n][1] *= f[0];
          o[n][2] *= f[1];
          o[n][3] *= f[1];
        }
      }
      // Slots at or past the tile's last visible key may hold anything: a weight
      // of zero does not silence a NaN, so their values are cleared.  A value
      // that is not finite at a key that some rows see and others do not is
      // rare (looked for in these steps only) and goes to the rows that see it
      // one by one.
      static_assert(kKeys == 16, "one product's depth of keys");
      uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
      if (k0 + kKeys > end) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int key = k0 + j * 8 + (lane & 3) * 2;
          keep[j] = (key < end ? 0xffffu : 0u) | (key + 1 < end ? 0xffff0000u : 0u);
        }
      }
      const int vkey = (((lane >> 3) & 1) << 3) + (lane & 7), vch = lane >> 4;  // this lane's row and chunk of a load
      const auto load_v = [&](int dp, uint32_t (&b)[4]) {
        const int ch = dp * 2 + vch;
        ldsm4_t(b, vb + uint32_t(ch >> 3) * (kKeys * 128) + sw128_offset(vkey, ch & 7));
        b[0] &= keep[0];
        b[1] &= keep[1];
        b[2] &= keep[0];
        b[3] &= keep[1];
      };
      bool odd = false;
      if (k0 + kKeys - 1 > low) {
#pragma unroll
        for (int dp = 0; dp < D / 16; ++dp) {
          uint32_t b[4];
          load_v(dp, b);
#pragma unroll
          for (int j = 0; j < 4; ++j) odd |= not_finite2<T>(b[j]);
        }
        odd = __any_sync(0xffffffffu, odd);
      }
      if (!odd) {
#pragma unroll
        for (int dp = 0; dp < D / 16; ++dp) {
          uint32_t b[4];
          load_v(dp, b);
          mma16816<T>(o[2 * dp], pf, b[0], b[1]);
          mma16816<T>(o[2 * dp + 1], pf, b[2], b[3]);
        }
      } else {
#pragma unroll 1
        for (int k = 0; k < min(kKeys, end - k0); ++k) {
          const int from = (lane & 28) | ((k & 7) >> 1);
          const float w0 = __shfl_sync(0xffffffffu, k & 8 ? (k & 1 ? acc[1][1] : acc[1][0]) : (k & 1 ? acc[0][1] : acc[0][0]), from);
          const float w1 = __shfl_sync(0xffffffffu, k & 8 ? (k & 1 ? acc[1][3] : acc[1][2]) : (k & 1 ? acc[0][3] : acc[0][2]), from);
          const bool see0 = k0 + k <= lim[0], see1 = k0 + k <= lim[1];
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            uint32_t x;
            asm volatile("ld.shared.b32 %0, [%1];"
                         : "=r"(x)
                         : "r"(vb + uint32_t(n >> 3) * (kKeys * 128) + sw128_offset(k, n & 7) + (lane & 3) * 4)
                         : "memory");
            const float2 v = unpack2<T>(x);
            if (see0) {
              o[n][0] += weighted(w0, v.x);
              o[n][1] += weighted(w0, v.y);
            }
            if (see1) {
              o[n][2] += weighted(w1, v.x);
              o[n][3] += weighted(w1, v.y);
            }
          }
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
      mbar_wait_hw(&sm.full[warp][(it + i) % kStages], ((it + i) / kStages) & 1, wc);
    it += issued;

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
    const int64_t flat = int64_t(w.t.tile) * kRowsM + row;
    const bool valid = flat < n_rows, whole = w.whole();
    const int tok = int(flat / p.g), h = int(flat % p.g);
    if (valid) {
      float top = -INFINITY, sum = 0.f, wt[kRWarps];
#pragma unroll
      for (int i = 0; i < kRWarps; ++i) top = fmaxf(top, sm.m[i][row]);
#pragma unroll
      for (int i = 0; i < kRWarps; ++i) {
        wt[i] = top == -INFINITY ? 0.f : ex2_approx(sm.m[i][row] - top);
        sum += sm.l[i][row] * wt[i];
      }
      const float none = whole && sum == 0.f ? no_weights(row_limit(p, w.t.row0, w.t.n, w.t.past, tok) >= 0) : 0.f;
      const float inv = sum != 0.f ? 1.f / sum : none;
      const int64_t part = int64_t(w.slot()) * kRowsM + row;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const int d = c * 64 + sub * 8;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kRWarps; ++i) {
          const float4* x = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm.kv[i]) + row * D +
                                                            (d ^ ((row & 3) * 8)));
          const float4 a = x[0], b = x[1];
          v[0] = fmaf(a.x, wt[i], v[0]); v[1] = fmaf(a.y, wt[i], v[1]);
          v[2] = fmaf(a.z, wt[i], v[2]); v[3] = fmaf(a.w, wt[i], v[3]);
          v[4] = fmaf(b.x, wt[i], v[4]); v[5] = fmaf(b.y, wt[i], v[5]);
          v[6] = fmaf(b.z, wt[i], v[6]); v[7] = fmaf(b.w, wt[i], v[7]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= inv;
        if (!whole) {
          float4* dst = reinterpret_cast<float4*>(p.part + part * D + d);
          dst[0] = make_float4(v[0], v[1], v[2], v[3]);
          dst[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
          uint16_t* dst = static_cast<uint16_t*>(p.o) + int64_t(w.t.row0 + tok) * p.o_ss + int64_t(w.hkv) * p.o_sh +
                          int64_t(h) * p.o_sq + d;
          *reinterpret_cast<uint4*>(dst) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]),
                                                      pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
        }
      }
      if (sub == 0) {
        if (!whole)
          p.part_ml[part] = make_float2(top, sum);
        else if (p.lse)
          p.lse[int64_t(w.hkv * p.g + h) * p.chunk.T + w.t.row0 + tok] =
              sum != 0.f ? (top + __log2f(sum)) * 0.69314718055994531f : none - INFINITY;
      }
    }
    if (!whole) {
      int owner, pieces;
      const bool joins = piece_arrive(p, w, 1, kRThreads, threadIdx.x == 0, &sm.joins, &owner, &pieces);
      if (joins && valid) join_row<T, D>(p, w.hkv, owner, pieces, kRowsM, row, sub, w.t.row0 + tok, h);
    }
    fence_proxy_async_smem();  // the output rows in the rings were read and written by plain accesses
    __syncthreads();
  }
}

// ---------------------------------------------------------------- many rows
// The forward kernel's pipeline (attn_fwd.cu) over pages, kept full across
// items: a persistent CTA walks its items of the plan, and every warp role walks
// the same pieces at its own pace, so the next piece's Q and K load and its first
// products run while the last one's rows are still written out (one item per CTA,
// as in attn_fwd.cu, spent 19 of 93 us per 41-unit item outside its key loop).
//   warps 0, 3  TMA producers (Q per piece and the K ring; the V ring, of which it
//               also clears what no weight may meet)
//   warp 1      MMA issuer
//   warp 2      walks the plan and hands the pieces to the others through a ring
//               in shared memory
//   warps 4-7 and 8-11: two softmax groups
// A tile's rows are tpt = 128 / g tokens times the g heads of one kv head,
// token-major, so a short chunk fills its rows with heads and every K/V tile
// feeds all heads that share it.
// The work is a line of positions, alternating between the two groups: group i &
// 1 takes position i.  With two row tiles a unit of 128 keys is two positions
// (the tiles); with one row tile a unit is one position, so that the groups work
// on two units of the same rows at a time and merge their outputs at the end of
// the piece (the tensor core would otherwise wait out every softmax: 17 rows over
// 131072 keys 151 us, with this 111).  Issue order: QK(0), QK(1), then PV(i),
// QK(i+2) for each i.
// Measured (one B200): 2 x 4098 rows over 5122 keys, 32/8 heads of 128: 672 us a call
// back to back = 1023 TFLOP/s, 62% of the measured burst peak and 73% of the sustained
// one (the power cap is on); this kernel alone after a pause, between events, 622.
// What bounds it is the one warp that issues the products: 1750 cycles a position, of
// which their issue takes 750 and the waits, commits and the walk the rest, while a
// softmax group waits for its scores 40% of its time.  (So the weights are handed over
// once per position: by halves, the first product beginning under the second half's
// exponentials, 612 us against 593 of the kernel on one box.  A second issuing warp,
// one per group, was slower: 712 there.)  With one row tile the key loop streams K and
// V at 6.3 TB/s, 96% of the measured copy rate.  A row that sees nothing makes the
// tile's `low` -1, so that every unit of the tile waits to be looked over: 8 x 400 rows
// over 4400 keys 224 us, with three such rows a sequence 324.
constexpr int kTThreads = 384;
constexpr int kLaunchRegs = 168;           // 128*88 + 256*208 = 384*168 after setmaxnreg
constexpr int kKStages = 3;
constexpr int kVStages = 2;

constexpr int kRing = 4;

// A wait of a whole warp: the usual case, a phase that is complete or nearly so,
// in a few instructions, the rest in a call, so that the MMA issuer's loop stays
// short (with the wait's own loop in line, five times, 3% longer).
__device__ __noinline__ bool warp_wait_long(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, WaitCtx{abort_flag, status, kTimeoutNs}));
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtx& w) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || warp_wait_long(bar, parity, w.abort_flag, w.status);
}

// What a piece is, as the warp roles read it.
struct Piece {
  int hkv, u0, u1;              // kv head, units [u0, u1); u1 < 0: no piece, the end
  int b, tile, row0, n, past;   // the sequence and the tile's index in it
  int end, nt;                  // keys [0, end) are visible to some row; row tiles (1 or 2)
  int low;                      // keys [0, low] are visible to every row
  int whole;                    // the only piece of its item
  int slot;                     // otherwise: where its partial rows go
  int odd;                      // set on the way: values that are not finite at keys that only some rows see
  int pad[2];
};
constexpr int kOddBits = 256;

template <int D>
struct TilesSmem {
  static constexpr int kTileElems = 128 * D;
  alignas(1024) uint16_t q[2][kTileElems];
  alignas(1024) uint16_t k[kKStages][kTileElems];
  alignas(1024) uint16_t v[kVStages][kTileElems];
  float2 ml[128];  // the second group's maximum and sum, for the merge of one row tile
  Piece ring[kRing];
  // where a piece is odd: bit (u - u0) % kOddBits of unit u (units that far apart share one)
  uint32_t odd_units[kRing][kOddBits / 32];
  uint64_t bar_piece_full[kRing];
  uint64_t bar_piece_empty[kRing];
  uint64_t bar_ml_full;   // the second group's ml and output can be read
  uint64_t bar_ml_empty;  // they have been
  uint64_t bar_q_full;
  uint64_t bar_q_empty;
  uint64_t bar_k_full[kKStages];
  uint64_t bar_k_empty[kKStages];
  uint64_t bar_v_full[kVStages];
  uint64_t bar_v_clean[kVStages];
  uint64_t bar_v_empty[kVStages];
  uint64_t bar_s_full[2];
  uint64_t bar_p_ready[2];
  uint64_t bar_o_final[2];
  uint64_t bar_drain;
  uint32_t tmem_base;
  int abort_flag;
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
__device__ __forceinline__ void issue_pv(uint32_t tO, uint32_t tP, uint64_t vdesc, bool accumulate) {
  constexpr uint32_t idesc = idesc16<T>(128, D, 0, 1);
  constexpr MNMajorSteps<8> st;
  mma_chain_ts_w<8>(tO, tP, 8u, vdesc, st.v, idesc, accumulate ? 1u : 0u);
}

// Weights of a row of 128 columns.  (The polynomial exponentials
// that attn_fwd.cu gives part of the columns cost more issue slots here than the
// special function units had to spare: with 5 of every 16 pairs 634 us, with none
// 612, at 2 x 4098 rows.)
template <class T>
__device__ __forceinline__ void exp_pack(const uint32_t (&sr)[128], float2 cs2, float2 nm2, uint32_t (&pk)[64],
                                         float2 (&ls)[2]) {
#pragma unroll
  for (int c = 0; c < 64; ++c) {
    const float2 x = __ffma2_rn(make_float2(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1])), cs2, nm2);
    const float2 pv = make_float2(ex2_approx(x.x), ex2_approx(x.y));
    ls[c & 1] = __fadd2_rn(ls[c & 1], pv);
    pk[c] = pack2<T>(pv.x, pv.y);
  }
}

// 32 consecutive elements of a row, rounded.
template <class T>
__device__ __forceinline__ void store32(uint16_t* dst, const uint32_t (&v)[32], bool wide) {
  uint32_t pk[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) pk[i] = pack2<T>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
  if (wide) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + 16 * i), "r"(pk[8 * i]),
                   "r"(pk[8 * i + 1]), "r"(pk[8 * i + 2]), "r"(pk[8 * i + 3]), "r"(pk[8 * i + 4]), "r"(pk[8 * i + 5]),
                   "r"(pk[8 * i + 6]), "r"(pk[8 * i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<uint4*>(dst)[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
  }
}

// Row r of a value tile (keys down, 128-byte swizzled): whether it holds an
// element that is not finite; and those set to 0, before the product with it: a
// weight of zero does not silence a NaN.  (The rows that see such a key get it
// back in add_odd.)
template <class T, int D>
__device__ __forceinline__ bool row_odd(const uint16_t* v, int r) {
  constexpr uint32_t e = std::is_same<T, __nv_bfloat16>::value ? 0x7f807f80u : 0x7c007c00u;
  constexpr uint32_t one = std::is_same<T, __nv_bfloat16>::value ? 0x00800080u : 0x04000400u;
  uint32_t top = 0;  // bits 15 and 31: an exponent of all ones carries into them
#pragma unroll
  for (int h = 0; h < D / 64; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // any order of a row's 16-byte chunks will do: this one has no bank conflicts
      const uint4 x = *reinterpret_cast<const uint4*>(v + h * 128 * 64 + r * 64 + ((i + r) & 7) * 8);
      top |= ((x.x & e) + one) | ((x.y & e) + one) | ((x.z & e) + one) | ((x.w & e) + one);
    }
  return (top & 0x80008000u) != 0;
}
// Rows [from, to) of the value tile of unit u looked over by a warp.  (By the V
// producer: in the MMA warp it cost the issue loop 10%.)
template <class T, int D>
__device__ __noinline__ void look_over(uint16_t* v, int from, int to, Piece& w, uint32_t* odd_units, int u) {
  bool odd = false;
  for (int r = from + int(threadIdx.x & 31); r < to; r += 32)
    if (row_odd<T, D>(v, r)) {
      odd = true;
      for (int i = 0; i < D; ++i) {
        uint16_t* x = v + (i / 64) * 128 * 64 + r * 64 + i % 64;
        if (not_finite2<T>(*x)) *x = 0;
      }
    }
  if (odd) {  // (every lane that found one writes the same)
    const int bit = (u - w.u0) % kOddBits;
    volatile uint32_t* units = odd_units + bit / 32;
    *units = *units | 1u << (bit % 32);
    *reinterpret_cast<volatile int*>(&w.odd) = 1;
    fence_proxy_async_smem();
  }
  __syncwarp();
}
// Rows [from, 128) cleared by a warp.
template <int D>
__device__ __noinline__ void clear_tail(uint16_t* v, int from) {
  for (int c = from * 8 + int(threadIdx.x & 31); c < 128 * 8; c += 32)
#pragma unroll
    for (int h = 0; h < D / 64; ++h) *reinterpret_cast<uint4*>(v + h * 128 * 64 + c * 8) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

// Row r of row tile x of a piece, which this thread has written (partial, or to
// o): the values that look_over took out of the piece's units, from the pages
// (an infinity or a NaN stays one whatever its positive weight).  Only the units
// where it found some: with every row going over every key of the piece, one
// infinity in each of 160 chunks of 20 rows over 20000 keys (one row of each sees
// nothing) took 52 ms, and over some 40 times as many keys the other warps' waits
// would have run out; now 0.48, and 0.38 without any.
template <class T, int D>
__device__ __noinline__ void add_odd(const CacheAttn& p, const Piece& w, const uint32_t* odd_units, int x, int r) {
  const int tok = (w.tile * 2 + x) * p.tpt + r / p.g;
  uint16_t* o = static_cast<uint16_t*>(p.o) + int64_t(w.row0 + tok) * p.o_ss + int64_t(w.hkv) * p.o_sh +
                int64_t(r % p.g) * p.o_sq;
  float* part = p.part + (int64_t(w.slot) * kTilesM + x * 128 + r) * D;
  const int from = max(w.low + 1, 0);
  const int to = min(row_limit(p, w.row0, w.n, w.past, tok) + 1, w.u1 * kUnit);
  for (int u = max(w.u0, from / kUnit); u * kUnit < to; ++u) {
    const int bit = (u - w.u0) % kOddBits;
    if (!(odd_units[bit / 32] >> (bit % 32) & 1)) continue;
    for (int k = max(u * kUnit, from); k < min((u + 1) * kUnit, to); ++k) {
      const int page = chunk_page(p.chunk, w.b, k >> p.chunk.page_shift);
      if (page == p.chunk.n_pages) continue;
      const uint4* v = reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(p.v) + int64_t(page) * p.v_sp +
          int64_t(k & ((1 << p.chunk.page_shift) - 1)) * p.v_ss + int64_t(w.hkv) * p.v_sh);
#pragma unroll 1
      for (int i = 0; i < D / 8; ++i) {
        const uint4 e = __ldg(v + i);
        const uint32_t two[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (!not_finite2<T>(two[c])) continue;
          const int at = i * 4 + c;
          float2 f = unpack2<T>(two[c]);
          if (isfinite(f.x)) f.x = 0.f;
          if (isfinite(f.y)) f.y = 0.f;
          if (w.whole) {
            const float2 was = unpack2<T>(reinterpret_cast<uint32_t*>(o)[at]);
            reinterpret_cast<uint32_t*>(o)[at] = pack2<T>(was.x + f.x, was.y + f.y);
          } else {
            part[2 * at] += f.x;
            part[2 * at + 1] += f.y;
          }
        }
      }
    }
  }
}

template <class T, int D>
__global__ void __launch_bounds__(kTThreads, 1)
    attn_cache_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CacheAttn p) {
  extern __shared__ uint8_t smem_raw[];
  TilesSmem<D>& sm =
      *reinterpret_cast<TilesSmem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // (a shuffle, so that the compiler knows the role to be one per warp)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    mbar_init(&sm.bar_q_full, 1);
    mbar_init(&sm.bar_q_empty, 1);
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&sm.bar_k_full[i], 1);
      mbar_init(&sm.bar_k_empty[i], 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&sm.bar_v_full[i], 1);
      mbar_init(&sm.bar_v_clean[i], 1);
      mbar_init(&sm.bar_v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.bar_s_full[i], 1);
      mbar_init(&sm.bar_p_ready[i], 4);  // one arrival per softmax warp
      mbar_init(&sm.bar_o_final[i], 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.bar_piece_full[i], 1);
      mbar_init(&sm.bar_piece_empty[i], 11);  // every warp but the one that writes it
    }
    mbar_init(&sm.bar_ml_full, 4);
    mbar_init(&sm.bar_ml_empty, 4);
    mbar_init(&sm.bar_drain, 1);
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const WaitCtx wc{&sm.abort_flag, p.chunk.status, kTimeoutNs};
  // piece i of this CTA, or false when a wait ran out; at the end u1 < 0
  const auto piece_wait = [&](int i) {
    return __all_sync(0xffffffffu, mbar_wait(&sm.bar_piece_full[i % kRing], (i / kRing) & 1, wc));
  };
  const auto piece_done = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.bar_piece_empty[i % kRing]);
  };

  if (warp < 4) {
    regs_dec<88>();
    if (warp == 0 || warp == 3) {
      // =============================== TMA producers, one of Q and K and one of
      // V: lane l copies box l of a tile, (64-wide column block l % (D/64)) of
      // page l / (D/64)
      const bool is_k = warp == 0;
      const int n_stage = is_k ? kKStages : kVStages;
      uint64_t* full = is_k ? sm.bar_k_full : sm.bar_v_full;
      uint64_t* empty = is_k ? sm.bar_k_empty : sm.bar_v_empty;
      uint16_t* ring = is_k ? sm.k[0] : sm.v[0];
      const CUtensorMap* map = is_k ? &tm_k : &tm_v;
      const int box = min(1 << p.chunk.page_shift, 128), n_box = 128 / box;
      const int col = lane % (D / 64), pg = lane / (D / 64);
      int ku = 0, s = 0, qs = 0;  // units so far, ring slot, pieces whose Q is on its way
      bool ok = true;
      for (int pc = 0; ok; ++pc) {
        ok = piece_wait(pc);
        Piece& w = sm.ring[pc % kRing];
        const int u0 = w.u0, u1 = w.u1, end = w.end, b = w.b, hkv = w.hkv;
        if (!ok || u1 < 0) break;
        if (!is_k && lane < kOddBits / 32) sm.odd_units[pc % kRing][lane] = 0;
        int page = 0;  // of this lane's box in the next unit
        const auto next_page = [&](int u) {
          const int key = u * kUnit + pg * box;
          if (pg < n_box && u < u1 && key < end) page = chunk_page(p.chunk, b, key >> p.chunk.page_shift);
        };
        next_page(u0);
        for (int u = u0; u < u1; ++u) {
          const int key = u * kUnit + pg * box;  // first key of this lane's box
          const bool mine = pg < n_box && key < end;
          const int slot = key & ((1 << p.chunk.page_shift) - 1);
          const uint32_t bytes = uint32_t(min(n_box, (end - u * kUnit + box - 1) / box)) * box * D * 2;
          if (ku >= n_stage && !warp_wait(&empty[s], ((ku / n_stage) - 1) & 1, wc)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
          __syncwarp();
          if (mine)
            tma_load_4d(ring + s * (128 * D) + col * 128 * 64 + pg * box * 64, map, &full[s], col * 64, slot, hkv, page);
          next_page(u + 1);
          if (!is_k && u >= (w.low + 1) / kUnit) {
            // A weight of zero does not silence a NaN.  The values of keys that
            // only some rows see may be anything: those that are not finite are
            // cleared.  So may what lies at or past the tile's last visible key
            // (the rest of the sequence's last page, pages that were not
            // loaded): cleared.  The MMA issuer waits for it (bar_v_clean).
            ok = warp_wait(&full[s], (ku / n_stage) & 1, wc);
            if (!ok) {
              ++ku;
              break;
            }
            uint16_t* v = ring + s * (128 * D);
            if (w.low + 1 < end) look_over<T, D>(v, max(w.low + 1 - u * kUnit, 0), min(end - u * kUnit, 128), w, sm.odd_units[pc % kRing], u);
            if (end - u * kUnit < 128) clear_tail<D>(v, end - u * kUnit);
            if (lane == 0) mbar_arrive(&sm.bar_v_clean[s]);
          }
          ++ku;
          s = s + 1 == n_stage ? 0 : s + 1;
          if (is_k && u == u0) {  // Q, once the last piece's products have read theirs
            if (pc > 0 && !warp_wait(&sm.bar_q_empty, (pc - 1) & 1, wc)) {
              ok = false;
              break;
            }
            if (lane == 0) {
              mbar_arrive_expect_tx(&sm.bar_q_full, uint32_t(p.tpt * p.g) * D * 2 * w.nt);
              for (int i = 0; i < w.nt; ++i)
                for (int c = 0; c < D / 64; ++c)
                  tma_load_4d(&sm.q[i][c * 128 * 64], &tm_q, &sm.bar_q_full, c * 64, 0, hkv,
                              w.row0 + (w.tile * 2 + i) * p.tpt);
            }
            ++qs;
          }
        }
        if (!ok) break;
        piece_done(pc);
      }
      __syncwarp();
      // Drain: the copies this CTA issued must land before its shared memory
      // can be released, whatever the consumers did.
      if (qs > 0) mbar_wait_hw(&sm.bar_q_full, (qs - 1) & 1, wc);
      for (int j = max(ku - n_stage, 0); j < ku; ++j) mbar_wait_hw(&full[j % n_stage], (j / n_stage) & 1, wc);
    } else if (warp == 1) {
      // =============================== MMA issuer: the warp runs converged and
      // one elected lane issues
      constexpr uint32_t kStageStep = (128u * D * 2u) >> 4;
      const uint64_t qd0 = sdesc_sw128(smem_u32(sm.q[0]), 16, 1024);
      const uint64_t kd0 = sdesc_sw128(smem_u32(sm.k[0]), 16, 1024);
      const uint64_t vd0 = sdesc_sw128(smem_u32(sm.v[0]), 16384, 1024);
      // two cursors over the positions: QK's runs two positions ahead of PV's
      int q_pc = 0, q_nt = 0, q_units = 0, q_u = 0, q_x = 0;  // piece, its row tiles and units; unit, row tile
      int ku = 0, ks = 0, vu = 0, vs = 0;
      bool ok = true, q_more = true;
      const auto q_piece = [&]() {
        ok = piece_wait(q_pc);
        const Piece& w = sm.ring[q_pc % kRing];
        q_units = w.u1 - w.u0;
        q_nt = w.nt;
        q_more = ok && w.u1 >= 0;
        q_u = q_x = 0;
      };
      // QK of the cursor's position into group t's scores, and one step on
      const auto qk = [&](int t) {
        if (q_x == 0) {
          ok = warp_wait(&sm.bar_k_full[ks], (ku / kKStages) & 1, wc) &&
               (q_u > 0 || warp_wait(&sm.bar_q_full, q_pc & 1, wc));
          if (!ok) return;
        }
        issue_qk<T, D>(tmem + uint32_t(t * 128), qd0 + uint32_t(q_x) * kStageStep, kd0 + uint32_t(ks) * kStageStep);
        tc_commit_w(&sm.bar_s_full[t]);
        if (++q_x < q_nt) return;
        q_x = 0;
        tc_commit_w(&sm.bar_k_empty[ks]);
        ++ku;
        ks = ks + 1 == kKStages ? 0 : ks + 1;
        if (++q_u < q_units) return;
        tc_commit_w(&sm.bar_q_empty);
        ++q_pc;
        q_piece();
      };
      q_piece();
      if (q_more) qk(0);
      if (ok && q_more) qk(1);
      int pos = 0;
      uint32_t cleans = 0;  // phase of bar_v_clean, a bit for each stage
      for (int pc = 0; ok; ++pc) {
        ok = piece_wait(pc);
        const Piece& w = sm.ring[pc % kRing];
        const int u0 = w.u0, u1 = w.u1, nt = w.nt, unclean = (w.low + 1) / kUnit;
        if (!ok || u1 < 0) break;
        for (int u = u0; ok && u < u1; ++u) {
          for (int x = 0; x < nt; ++x, ++pos) {
            const int t = pos & 1;
            const uint32_t tS = tmem + uint32_t(t * 128), tO = tmem + 256u + uint32_t(t * D);
            const uint32_t ph = (pos >> 1) & 1;
            if (x == 0) {
              ok = warp_wait(&sm.bar_v_full[vs], (vu / kVStages) & 1, wc);
              if (u >= unclean) {  // the V producer looks it over first
                ok = ok && warp_wait(&sm.bar_v_clean[vs], (cleans >> vs) & 1, wc);
                cleans ^= 1u << vs;
              }
              if (!ok) break;
            }
            // the group's first position of the piece overwrites its output
            const bool acc = u - u0 >= (nt == 2 ? 1 : 2);
            ok = warp_wait(&sm.bar_p_ready[t], ph, wc);
            if (!ok) break;
            tc_fence_after();
            issue_pv<T, D>(tO, tS, vd0 + uint32_t(vs) * kStageStep, acc);
            if (u1 - u <= (nt == 2 ? 1 : 2)) tc_commit_w(&sm.bar_o_final[t]);  // the group's last one of the piece
            if (x == nt - 1) {
              tc_commit_w(&sm.bar_v_empty[vs]);
              ++vu;
              vs = vs + 1 == kVStages ? 0 : vs + 1;
            }
            if (q_more) {
              qk(t);
              if (!ok) break;
            }
          }
        }
        piece_done(pc);
      }
      // MMAs already issued must finish before TMEM can be released.
      tc_commit_w(&sm.bar_drain);
      mbar_wait_hw(&sm.bar_drain, 0, wc);
    } else if (warp == 2) {
      // =============================== the plan
      asm volatile("griddepcontrol.wait;" ::: "memory");  // it is written
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
      Walk w;
      bool more = w.begin(p);
      for (int i = 0;; ++i) {
        Piece x{};
        x.u1 = -1;
        if (more) {
          x.hkv = w.hkv;
          x.u0 = w.u0;
          x.u1 = w.u1;
          x.b = w.t.b;
          x.tile = w.t.tile;
          x.row0 = w.t.row0;
          x.n = w.t.n;
          x.past = w.t.past;
          x.end = w.t.end;
          x.nt = w.t.nt;
          x.low = w.t.low;
          x.whole = w.whole();
          x.slot = w.slot();
        }
        if (i >= kRing &&
            !warp_wait(&sm.bar_piece_empty[i % kRing], ((i / kRing) - 1) & 1, wc))
          break;
        if (lane == 0) {
          sm.ring[i % kRing] = x;
          mbar_arrive(&sm.bar_piece_full[i % kRing]);
        }
        __syncwarp();
        if (!more) break;
        more = w.next(p);
      }
    }
  } else {
    regs_inc<208>();
    // =============================== softmax / epilogue; tcgen05.ld/st are
    // warp-collective: every branch around them is warp-uniform
    const int t = warp >= 8 ? 1 : 0, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_off = uint32_t(quarter * 32) << 16;
    const uint32_t tS = tmem + uint32_t(t * 128) + lane_off;
    const uint32_t tO = tmem + 256u + uint32_t(t * D) + lane_off;
    uint32_t pos = 0;   // positions of all pieces so far (both groups)
    uint32_t seen = 0;  // this group's positions so far
    uint32_t outs = 0;  // pieces in which it had one
    uint32_t merges = 0;  // merged pieces
    bool ok = true;
    for (int pc = 0; ok; ++pc) {
      ok = piece_wait(pc);
      const Piece& w = sm.ring[pc % kRing];
      if (!ok || w.u1 < 0) break;
      // which positions of the piece are this group's: with two row tiles tile
      // x of every unit, with one the units x, x + 2, ...
      const int x = int((pos & 1) ^ uint32_t(t));
      int count, key, key_step, low, hi;
      {
        const int nt = w.nt, units = w.u1 - w.u0;
        count = nt == 2 ? units : (units - x + 1) >> 1;
        key = (w.u0 + (nt == 2 ? 0 : x)) * kUnit;  // first key of the group's next position
        key_step = nt == 2 ? kUnit : 2 * kUnit;
        pos += uint32_t(units * nt);
        // rows that are no row of the sequence count as seeing everything and
        // are never stored
        const int tok = (w.tile * 2 + (nt == 2 ? x : 0)) * p.tpt + r / p.g;
        const int lim = r < p.tpt * p.g && tok < w.n ? row_limit(p, w.row0, w.n, w.past, tok) : 0x7fffffff;
        low = min(__reduce_min_sync(0xffffffffu, lim), w.end - 1);  // every row of the warp sees the keys <= low
        hi = min(lim, w.end - 1);
      }
      float m = -INFINITY, l = 0.f;
      const float cs = p.scale_log2;
      for (int j = 0; j < count; ++j, key += key_step) {
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.bar_s_full[t], seen & 1, wc));
        if (!ok) break;
        ++seen;
        tc_fence_after();
        uint32_t sr[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
        tmem_ld_wait_regs(sr);
        if (key + 127 > low) {
          const int last = hi - key;  // key + c is visible iff c <= last
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c > last) sr[c] = __float_as_uint(-INFINITY);
        }
        __syncwarp();
        float mp[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) mp[c] = __uint_as_float(sr[c]);
#pragma unroll
        for (int c = 8; c < 120; c += 16)
#pragma unroll
          for (int k = 0; k < 8; ++k) mp[k] = fmax3(mp[k], __uint_as_float(sr[c + k]), __uint_as_float(sr[c + 8 + k]));
#pragma unroll
        for (int k = 0; k < 8; ++k) mp[k] = fmaxf(mp[k], __uint_as_float(sr[120 + k]));
        const float xmax = Fp16Weights<T>::below(fmaxf(fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])),
                                                       fmaxf(fmaxf(mp[4], mp[5]), fmaxf(mp[6], mp[7]))) * cs,
                                                 Fp16Weights<T>::kTiles);
        // Lazy rescale of O, by selects.  A row that has seen no key yet has m =
        // -inf: its O and l are 0 and any first maximum "grows" it with f = 0.
        float f = 1.f;
        bool rescale = false;
        if (j == 0) {
          m = xmax;
        } else {
          const bool grow = xmax > m + Fp16Weights<T>::kLag;
          rescale = __any_sync(0xffffffffu, grow);
          const float fg = ex2_approx(m - xmax);
          f = grow ? fg : 1.f;
          m = grow ? xmax : m;
        }
        const float sub = m == -INFINITY ? 0.f : m;
        uint32_t pk[64];
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 cs2 = make_float2(cs, cs), nm2 = make_float2(-sub, -sub);
        exp_pack<T>(sr, cs2, nm2, pk, ls);
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
        tmem_st32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.bar_p_ready[t]);
        l = l * f + ((ls[0].x + ls[1].x) + (ls[0].y + ls[1].y));
      }
      if (!ok) break;
      // ---- epilogue
      if (count > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.bar_o_final[t], outs & 1, wc));
        if (!ok) break;
        ++outs;
        tc_fence_after();
      }
      const int nt = w.nt, whole = w.whole;
      const int tile_row = (nt == 2 ? x * 128 : 0) + r;  // row of the item
      const int tok = (w.tile * 2 + (nt == 2 ? x : 0)) * p.tpt + r / p.g, head = r % p.g;
      const bool valid = r < p.tpt * p.g && tok < w.n;
      const int row = w.row0 + tok;
      // With one row tile and more than one unit both groups hold part of the
      // keys of the same rows: the first one reads both outputs (the same TMEM
      // lanes) and adds them, O = f0 O_0 + f1 O_1.
      const bool merge = nt == 1 && w.u1 - w.u0 > 1;
      const float none = no_weights(whole && hi >= 0);
      float f0, f1 = 0.f;
      bool writes = true, some;
      if (!merge) {
        writes = nt == 2 || x == 0;
        some = l != 0.f;
        f0 = some ? 1.f / l : none;
      } else if (t == 1) {
        writes = false;
        sm.ml[r] = make_float2(m, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.bar_ml_full);
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.bar_ml_empty, merges & 1, wc));  // until the output has been read
        if (!ok) break;
        ++merges;
        tc_fence_after();
      } else {
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.bar_ml_full, merges & 1, wc));
        if (!ok) break;
        ++merges;
        tc_fence_after();
        const float2 other = sm.ml[r];
        const float top = fmaxf(m, other.x);
        const float sub = top == -INFINITY ? 0.f : top;
        const float w0 = ex2_approx(m - sub), w1 = ex2_approx(other.x - sub);
        const float sum = l * w0 + other.y * w1;
        some = sum != 0.f;
        f0 = some ? w0 / sum : none;
        f1 = some ? w1 / sum : none;
        m = top;
        l = sum;
      }
      if (writes) {
        uint16_t* dst = static_cast<uint16_t*>(p.o) + int64_t(row) * p.o_ss + int64_t(w.hkv) * p.o_sh +
                        int64_t(head) * p.o_sq;
        float* part = p.part + (int64_t(w.slot) * kTilesM + tile_row) * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32], ow[32];
          tmem_ld32(tO + c * 32, ov);
          if (merge) {
            tmem_ld32(tO + uint32_t(D) + c * 32, ow);
            tmem_ld_wait_regs(ov, ow);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              ov[i] = __float_as_uint(fmaf(__uint_as_float(ov[i]), f0, __uint_as_float(ow[i]) * f1));
          } else {
            tmem_ld_wait_regs(ov);
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * f0);
          }
          if (valid) {
            if (whole) {
              store32<T>(dst + c * 32, ov, p.wide_o);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                reinterpret_cast<uint4*>(part + c * 32)[i] =
                    make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
            }
          }
        }
        tc_fence_before();
        if (merge) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.bar_ml_empty);
        }
        if (valid) {
          if (!whole)
            p.part_ml[int64_t(w.slot) * kTilesM + tile_row] = make_float2(m, l);
          else if (p.lse)
            p.lse[int64_t(w.hkv * p.g + head) * p.chunk.T + row] =
                some ? (m + __log2f(l)) * 0.69314718055994531f : none - INFINITY;
          if (*reinterpret_cast<const volatile int*>(&w.odd)) add_odd<T, D>(p, w, sm.odd_units[pc % kRing], nt == 2 ? x : 0, r);
        }
      }
      piece_done(pc);
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

// The split items of the tiles kernel (4 to 9 us): a block takes 32 rows of the item whose
// first piece is CTA blockIdx.x's last one.  (The rows kernel's last piece does
// this itself: its items have 16 rows, these 256, which one SM alone would take
// 20 to 70 us to add.)
template <class T, int D>
__global__ void __launch_bounds__(256) attn_cache_join_kernel(const __grid_constant__ CacheAttn p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x;
  const int4 j = __ldcg(reinterpret_cast<const int4*>(p.ws.joins + c));
  const int n = __ldcg(&p.ws.joins[c].n), pieces = j.x, hkv = j.y, tile = j.z, row0 = j.w;
  if (pieces <= 1) return;
  const int r = blockIdx.y * 32 + (threadIdx.x >> 3);
  const int tok = (tile * 2 + (r >> 7)) * p.tpt + (r & 127) / p.g;
  if ((r & 127) >= p.tpt * p.g || tok >= n) return;
  join_row<T, D>(p, hkv, c, pieces, kTilesM, r, threadIdx.x & 7, row0 + tok, (r & 127) % p.g);
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
  bool tiles;  // attn_cache_tiles, or attn_cache_rows
  int ctas, max_tiles, rows;
  size_t head, cuts, joins, arrived, first, tile, cum, part, ml, total;  // workspace offsets
};

// The tiles kernel when an average chunk has more than 16 rows per kv head, one
// tile of the rows kernel.  Measured with either kernel, captured calls back to
// back, us, rows / tiles, 32/8 heads of 128 (16/4 of 64), one token each: 1 x 1024
// keys 16.0 / 17.0 (14.6 / 15.7), 32 x 1024 35 / 37 (19 / 22), 128 ragged up to 4096
// 93 / 99 (42 / 51), 256 up to 2048 109 / 137 (51 / 79), 48 up to 32768 165 / 158
// (58 / 86); four tokens (16 rows) at 32 x 1024 38 / 50; six tokens (two row tiles) at
// 48 up to 32768 318 / 176.  (Single tokens over a few long caches of 128-wide heads
// would gain 4% from the tiles kernel, many short ones lose 25%: which it is, only the
// device knows.)  A batch of single tokens and one long chunk goes by its average too,
// and suits neither kernel: 255 tokens and 700 rows over 8192 keys each 1793 / 1808
// (the tokens alone 1304, the rows alone 113), 128 tokens and 380 rows over 1024 keys
// 143 / 137 (96 and 36).  Sequences without new tokens do not count (B <= T).
// False: more tiles than the plan's 32-bit indices.
bool plan_launch(const hia_cache& c, const hia_cache_chunk& k, int64_t T, int g, Launch* out) {
  Launch& L = *out;
  L = Launch{};
  const int n_sm = sm_count();
  const int64_t B = std::max<int64_t>(1, std::min<int64_t>(k.B, T));
  L.tiles = T * g > 16 * B;
  L.rows = L.tiles ? kTilesM : kRowsM;
  L.ctas = std::min(L.tiles ? n_sm : 2 * n_sm, kPlanThreads - 1);
  const int64_t tiles = L.tiles ? T / (2 * (128 / g)) + B : T * g / kRowsM + B;
  if (tiles >= (int64_t(1) << 30)) return false;
  L.max_tiles = int(tiles);
  size_t o = 0;
  const auto take = [&](size_t bytes) {
    const size_t at = o;
    o = a256(o + bytes);
    return at;
  };
  L.head = take(8);
  L.cuts = take(size_t(L.ctas + 1) * sizeof(Cut));
  L.joins = take(size_t(L.ctas) * sizeof(Join));
  L.arrived = take(size_t(L.ctas) * 4);
  L.first = take(size_t(k.B + 1) * 4);
  L.tile = take(size_t(tiles) * sizeof(Tile));
  L.cum = take(size_t(tiles + 1) * 8);
  L.part = take(size_t(2) * L.ctas * L.rows * c.D * 4);
  L.ml = take(size_t(2) * L.ctas * L.rows * 8);
  L.total = o;
  return true;
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

// A launch that may start while the one before it on the stream still runs
// (griddepcontrol.wait in the kernel waits for it).
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

template <class T, int D>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CacheAttn& p,
                   const Launch& L, cudaStream_t st) {
  static_assert(sizeof(TilesSmem<D>) + 1024 <= 232448, "shared memory budget");
  static_assert(2 * (sizeof(RowsSmem<D>) + 1024 + 1024) <= 233472, "two blocks an SM");
  static PerContext<int> ready_tiles, ready_rows;
  const size_t smem = (L.tiles ? sizeof(TilesSmem<D>) : sizeof(RowsSmem<D>)) + 1024;
  cudaError_t e = L.tiles ? smem_optin(ready_tiles, attn_cache_tiles_kernel<T, D>, smem, kLaunchRegs)
                          : smem_optin(ready_rows, attn_cache_rows_kernel<T, D>, smem, 0);
  if (e != cudaSuccess) return e;
  prof_begin(kAttnCachePlan, st);
  attn_cache_plan_kernel<<<1, kPlanThreads, 0, st>>>(p);
  prof_end(kAttnCachePlan, st);
  if (L.tiles) {
    prof_begin(kAttnCacheTiles, st);
    e = launch_after(attn_cache_tiles_kernel<T, D>, dim3(L.ctas), kTThreads, smem, st, tq, tk, tv, p);
    prof_end(kAttnCacheTiles, st);
    if (e != cudaSuccess) return e;
    prof_begin(kAttnCacheJoin, st);
    e = launch_after(attn_cache_join_kernel<T, D>, dim3(L.ctas, kTilesM / 32), 256, 0, st, p);
    prof_end(kAttnCacheJoin, st);
  } else {
    prof_begin(kAttnCacheRows, st);
    e = launch_after(attn_cache_rows_kernel<T, D>, dim3(L.ctas), kRThreads, smem, st, tk, tv, p);
    prof_end(kAttnCacheRows, st);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace
}  // namespace hia

extern "C" size_t hia_attn_cache_workspace_bytes(const hia_cache* c, const hia_cache_chunk* k, int64_t T, int Hq) {
  int rc;
  hia::Launch L;
  if (!hia::attn_args_ok(c, k, T, Hq, &rc) || !hia::plan_launch(*c, *k, T, Hq / c->Hkv, &L)) return 0;
  return L.total;
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
  // (q too: a tensor map's strides are not 0)
  if ((rc = own_rows_check(q, T, c->Hkv, g)) || (rc = own_rows_check(o, T, c->Hkv, g))) return rc;
  if (!aligned_to(bound, 4) || !aligned_to(lse, 4)) return HIA_ERR_UNSUPPORTED;
  Launch L;
  if (!plan_launch(*c, *k, T, g, &L)) return HIA_ERR_UNSUPPORTED;
  if (ws_bytes < L.total || !aligned_to(ws, 256)) return HIA_ERR_INVALID_ARG;
  int* status = device_status_word();
  if (!status) return HIA_ERR_CUDA;
  char* b = static_cast<char*>(ws);
  CacheAttn p{};
  p.chunk = chunk_dev(*c, *k, T, status);
  p.ws = PlanWs{reinterpret_cast<int*>(b + L.head),    reinterpret_cast<Cut*>(b + L.cuts),
                reinterpret_cast<Join*>(b + L.joins),
                reinterpret_cast<int*>(b + L.arrived), reinterpret_cast<int*>(b + L.first),
                reinterpret_cast<Tile*>(b + L.tile),   reinterpret_cast<long long*>(b + L.cum)};
  p.q = q.ptr;
  p.q_ss = q.stride_s;
  p.q_sh = q.stride_hkv;
  p.q_sq = q.stride_hq;
  p.v = c->v;
  p.v_sp = c->stride_page;
  p.v_ss = c->stride_s;
  p.v_sh = c->stride_h;
  p.o = o.ptr;
  p.o_ss = o.stride_s;
  p.o_sh = o.stride_hkv;
  p.o_sq = o.stride_hq;
  p.wide_o = aligned_to(o.ptr, 32) && o.stride_s % 16 == 0 && o.stride_hkv % 16 == 0 && (g == 1 || o.stride_hq % 16 == 0);
  p.lse = lse;
  p.bound = bound;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.Hkv = c->Hkv;
  p.g = g;
  p.tpt = L.tiles ? 128 / g : 0;
  p.ctas = L.ctas;
  p.max_tiles = L.max_tiles;
  p.item_cost = L.tiles ? 2 : 1;
  p.part = reinterpret_cast<float*>(b + L.part);
  p.part_ml = reinterpret_cast<float2*>(b + L.ml);

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
