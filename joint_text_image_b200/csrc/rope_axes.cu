// rope_axes.cu -- rotary positions with several axes, and the append of a
// chunk of new tokens to the paged key/value cache.
//
// Row t has positions pos[t][0 .. n_axes); pair j < D/2 of every head turns by
// a_j = pos[t][axis_j] freq_j (fp32 arithmetic, one rounding):
//   y_j = x_j cos a_j - x_{j+D/2} sin a_j,  y_{j+D/2} = x_{j+D/2} cos a_j + x_j sin a_j,
// the convention of HunyuanImage3Attention.forward (v*cos + rotate_half(v)*sin).
// The gradient is the turn by -a_j.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "cache.cuh"
#include "devctx.h"

namespace hia {
namespace {

// The plan as a kernel argument; frequencies in turns per unit of position.
struct RopeArg {
  double turns[HIA_ROPE_MAX_PAIRS];
  uint8_t axis[HIA_ROPE_MAX_PAIRS];
  int D, n_axes;
};

// 8 consecutive elements of a row half, as fetched and as fp32.
template <class T>
struct Half8 {
  uint4 u;
  __device__ __forceinline__ void load(const T* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = u; }
  __device__ __forceinline__ void get(float (&v)[8]) const;
  __device__ __forceinline__ void set(const float (&v)[8]);
};
template <>
__device__ __forceinline__ void Half8<__nv_bfloat16>::get(float (&v)[8]) const {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void Half8<__nv_bfloat16>::set(const float (&v)[8]) {
  u = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
template <>
__device__ __forceinline__ void Half8<__half>::get(float (&v)[8]) const {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(reinterpret_cast<const __half2*>(&u)[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <>
__device__ __forceinline__ void Half8<__half>::set(const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) reinterpret_cast<__half2*>(&u)[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
}
template <>
struct Half8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// One tensor of the pass: head (k, i), i < g, of row t is read at src + t*ss +
// k*sh + i*sq and written at dst + t*ds + k*dh + i*dq (elements).  Where both
// sides step evenly through all heads they are one group (g = H).
struct RowsPart {
  const void* src;
  void* dst;
  const float* w;  // QK RMSNorm weight (append with a norm)
  int64_t ss, sh, sq, ds, dh, dq;
  int g, per_group, passes;  // heads and passes of a group, passes in all (0: absent)
};

struct RowsArgs {
  RopeArg rope;
  RowsPart part[3];  // q, k and, appending, v
  const int32_t* pos;
  float sign;        // +1 turns forward, -1 back (the gradient)
  float eps;
  int T, turn;
  int passes, groups;  // passes of a row, and warps that share them
  // appending: the destination of k (part 1) and v (part 2) is a slot of a page
  ChunkDev chunk;
  int64_t stride_page, stride_s;
};

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxHeads = 1 << 16;

// A warp owns one row, or a share of its passes.  Lane = hs * CPH + c holds
// elements c*8 .. c*8+7 of both halves of one head (CPH = D / 16 lanes a head,
// 32 / CPH heads a pass), so each load and store of a head is two runs of D
// bytes, partner elements meet in one lane, and the lane's 8 angles stay in
// registers for all heads of the row: computed once per warp, D / 64 pairs a
// lane, and exchanged through shared memory.
// The bytes bound the kernel only if a pass is cheap: pointers advance by
// fixed steps (found by multiplication per head, addresses were two thirds of
// the instructions and the kernel issue-bound), and the row's first pass is
// loaded before anything else is looked up.
// Arithmetic is fp32 (the norm's sum of squares too); the one rounding to 16
// bits is the store's, so a normed row is not rounded between turn and norm.
// Measured (one B200, calls back to back), 32 + 8 heads of 128: 10244 rows (210
// MB) 43.4 us = 4.8 TB/s of the measured 6.5; the gradient of 32400 rows (664 MB)
// 112.7 us = 5.9 TB/s; appending 2 x 4098 rows with turn and norm (201 MB) 51.3
// us = 3.9 TB/s.  What bounds the larger two is the latency of their loads (10 of
// 18 cycles between a warp's instructions), with issue slots 32% used; with the
// norm its arithmetic as well (slots 40%).
// CPH_ = 0: D / 16 at run time (a head dimension other than 64 or 128).
template <class T, int CPH_, bool APPEND, bool NORM>
__global__ void __launch_bounds__(kThreads, NORM ? 7 : 8) rope_axes_kernel(const __grid_constant__ RowsArgs a) {
  __shared__ alignas(16) float cos_s[kWarps][HIA_ROPE_MAX_PAIRS], sin_s[kWarps][HIA_ROPE_MAX_PAIRS];
  __shared__ alignas(16) float w_s[NORM ? 2 : 1][NORM ? 128 : 1];
  constexpr int U = 1;  // passes in flight (2, 3, 4 with 24 or 16 warps an SM: no faster, the append slower)
  const int wib = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cph = CPH_ ? CPH_ : a.rope.D / 16, half = cph * 8, hpi = 32 / cph;
  const int c = lane % cph, hs = lane / cph;
  const bool on = hs < hpi;  // 32 % cph lanes idle
  const unsigned gmask = CPH_ ? ((1u << CPH_) - 1u) << (hs * CPH_) : 0u;
  if (NORM) {
    for (int i = threadIdx.x; i < 4 * half; i += kThreads)
      w_s[i >= 2 * half][i % (2 * half)] = __ldg((i >= 2 * half ? a.part[1].w : a.part[0].w) + i % (2 * half));
    __syncthreads();
  }
  const int64_t item = int64_t(blockIdx.x) * kWarps + wib;
  const int t = int(a.groups == 1 ? item : item / a.groups);
  if (t >= a.T) return;
  int n = a.passes, skip = 0;  // this warp's passes, and those before them
  if (a.groups > 1) {
    const int share = int(item - int64_t(t) * a.groups);
    skip = int(int64_t(n) * share / a.groups);
    n = int(int64_t(n) * (share + 1) / a.groups) - skip;
  }

  // the way through the passes of q, then k, then v
  int p = 0, in = 0, left = 0, g = 0;  // part, this lane's head within the group, passes left of the part, heads of a group
  const T* src = nullptr;
  T* dst = nullptr;
  int64_t s_in = 0, s_out = 0, d_in = 0, d_out = 0;  // steps to the next pass, within a group and to the next group
  const auto enter = [&]() {
    while (skip >= a.part[p].passes) {
      skip -= a.part[p].passes;
      ++p;
    }
    const RowsPart& x = a.part[p];
    const int k = skip / x.per_group, i = (skip - k * x.per_group) * hpi + hs;
    left = x.passes - skip;
    skip = 0;
    g = x.g;
    in = i;
    src = static_cast<const T*>(x.src) + t * x.ss + k * x.sh + i * x.sq + c * 8;
    dst = static_cast<T*>(x.dst) + (APPEND && p > 0 ? int64_t(0) : t * x.ds) + k * x.dh + i * x.dq + c * 8;
    s_in = hpi * x.sq;
    d_in = hpi * x.dq;
    s_out = x.sh - (x.per_group - 1) * s_in;
    d_out = x.dh - (x.per_group - 1) * d_in;
  };
  struct Pass {
    Half8<T> lo, hi;
    T* dst;
    int part;  // -1: no head of this lane
  };
  const auto fetch = [&](Pass& x) {
    if (left == 0) {
      ++p;
      enter();
    }
    x.part = on && in < g ? p : -1;
    x.dst = dst;
    if (x.part >= 0) {
      x.lo.load(src);
      x.hi.load(src + half);
    }
    // the group's last pass is the one that reaches its last head
    const bool wrap = in - hs + hpi >= g;
    in = wrap ? hs : in + hpi;
    src += wrap ? s_out : s_in;
    dst += wrap ? d_out : d_in;
    --left;
  };
  enter();
  Pass x[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < n) fetch(x[u]);

  // appending: the row's sequence (a 32-way search over the row starts) and slot
  int64_t slot = 0;
  int where = 0;  // 0 not in a sequence (or in a skipped one), 1 in one without a page, 2 with one
  if (APPEND) {
    if (t >= __ldg(a.chunk.rows) && t < __ldg(a.chunk.rows + a.chunk.B)) {
      int l = 0, h = a.chunk.B;  // rows[l] <= t < rows[h]
      while (h - l > 1) {
        const int st = (h - l + 31) / 32;
        const int i = l + lane * st;
        const unsigned le = __ballot_sync(0xffffffffu, i < h && __ldg(a.chunk.rows + min(i, h)) <= t);
        // the last probe at or before t (probe 0 is, when rows is ordered)
        const int last = le ? 31 - __clz(le) : 0;
        const int nl = l + last * st;
        h = min(h, nl + st);
        l = nl;
      }
      const Seq s = chunk_seq(a.chunk, l);
      const int i = t - s.row0;
      if (i >= 0 && i < s.n) {
        const int at = s.past + i;
        const int page = chunk_page(a.chunk, l, at >> a.chunk.page_shift);
        where = page < a.chunk.n_pages ? 2 : 1;
        slot = int64_t(page) * a.stride_page + int64_t(at & ((1 << a.chunk.page_shift) - 1)) * a.stride_s;
      }
    }
  }

  float cs[8], sn[8];
  if (!APPEND || a.turn) {
    for (int j = lane; j < half; j += 32) {
      // angle in turns, reduced to [-1/2, 1/2] in fp64; the fp32 rounding of
      // the fraction is put back to first order
      const double y = double(__ldg(a.pos + int64_t(t) * a.rope.n_axes + a.rope.axis[j])) * a.rope.turns[j];
      const double r = y - rint(y);
      const float f = float(r), d = float(r - double(f)) * 6.2831853f;
      float s0, c0;
      sincospif(2.f * f, &s0, &c0);
      cos_s[wib][j] = fmaf(-s0, d, c0);
      sin_s[wib][j] = a.sign * fmaf(c0, d, s0);
    }
    __syncwarp();
    if (on) {
#pragma unroll
      for (int k = 0; k < 8; k += 4) {
        const float4 x4 = *reinterpret_cast<const float4*>(&cos_s[wib][c * 8 + k]);
        const float4 y4 = *reinterpret_cast<const float4*>(&sin_s[wib][c * 8 + k]);
        cs[k] = x4.x; cs[k + 1] = x4.y; cs[k + 2] = x4.z; cs[k + 3] = x4.w;
        sn[k] = y4.x; sn[k + 1] = y4.y; sn[k + 2] = y4.z; sn[k + 3] = y4.w;
      }
    }
  }

  for (int i = 0; i < n; i += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= n) break;
      const int part = x[u].part;
      if (part >= 0 && (!APPEND || where >= (part > 0 ? 2 : 1))) {
        if (!APPEND || (part < 2 && (NORM || a.turn))) {
          float l[8], r[8];
          x[u].lo.get(l);
          x[u].hi.get(r);
          if (!APPEND || a.turn) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float y = fmaf(-r[k], sn[k], l[k] * cs[k]);
              r[k] = fmaf(l[k], sn[k], r[k] * cs[k]);
              l[k] = y;
            }
          }
          if (NORM) {
            // pairs of elements at a time (packed fp32 arithmetic)
            float2 q2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
              const float2 lk = make_float2(l[k], l[k + 1]), rk = make_float2(r[k], r[k + 1]);
              q2 = __ffma2_rn(lk, lk, __ffma2_rn(rk, rk, q2));
            }
            float q = q2.x + q2.y;
#pragma unroll
            for (int o = 1; o < (CPH_ ? CPH_ : 1); o <<= 1) q += __shfl_xor_sync(gmask, q, o);
            const float nr = rsqrtf(q * (1.f / float(2 * half)) + a.eps);
            const float2 n2 = make_float2(nr, nr);
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
              const float2 wl = *reinterpret_cast<const float2*>(w_s[part] + c * 8 + k);
              const float2 wr = *reinterpret_cast<const float2*>(w_s[part] + half + c * 8 + k);
              const float2 lk = __fmul2_rn(wl, __fmul2_rn(make_float2(l[k], l[k + 1]), n2));
              const float2 rk = __fmul2_rn(wr, __fmul2_rn(make_float2(r[k], r[k + 1]), n2));
              l[k] = lk.x;
              l[k + 1] = lk.y;
              r[k] = rk.x;
              r[k + 1] = rk.y;
            }
          }
          x[u].lo.set(l);
          x[u].hi.set(r);
        }
        T* d = x[u].dst;
        if (APPEND && part > 0) d += slot;
        x[u].lo.store(d);
        x[u].hi.store(d + half);
      }
      if (i + U + u < n) fetch(x[u]);
    }
  }
}

__global__ void __launch_bounds__(256) rope_axes_tables_kernel(const __grid_constant__ RopeArg plan,
                                                               int64_t T,
                                                               const int32_t* __restrict__ pos,
                                                               float* __restrict__ cos_out,
                                                               float* __restrict__ sin_out) {
  // turns[] holds radians here: angle and cos/sin in fp64, rounded once, as
  // the 2D tables do.  10244 rows of 128 take 12 us in a graph, of which their
  // bytes (10.6 MB) need 1.6 (once per training step).  What bounds it is the
  // reading of the plan, another entry in every lane, from the kernel's arguments
  // (the pipe that serves divergent constants is 90% busy, the fp64 one 6%).
  const int half = plan.D / 2;
  const int64_t n = T * half;
  for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t t = i / half;
    const int j = int(i - t * half);
    double s, c;
    sincos(double(pos[t * plan.n_axes + plan.axis[j]]) * plan.turns[j], &s, &c);
    const int64_t o = t * plan.D + j;
    cos_out[o] = cos_out[o + half] = float(c);
    sin_out[o] = sin_out[o + half] = float(s);
  }
}

bool plan_ok(const hia_rope_plan* p) {
  if (!p || p->D < 16 || p->D > 256 || p->D % 16 || p->n_axes < 1 || p->n_axes > HIA_ROPE_MAX_AXES) return false;
  for (int j = 0; j < p->D / 2; ++j)
    if (p->axis[j] >= p->n_axes || !std::isfinite(p->freq[j])) return false;
  return true;
}

RopeArg rope_arg(const hia_rope_plan* p, double unit) {
  RopeArg r{};
  r.D = p->D;
  r.n_axes = p->n_axes;
  for (int j = 0; j < p->D / 2; ++j) {
    r.axis[j] = p->axis[j];
    r.turns[j] = p->freq[j] * unit;
  }
  return r;
}

constexpr double kTurnsPerRadian = 0.15915494309189533577;

// The tensors of H heads in groups of g, of which a pass takes hpi.
RowsPart make_part(const hia_tensor& src, const hia_tensor& dst, int H, int g, const float* w, int hpi) {
  RowsPart x{src.ptr,    dst.ptr,         w,  src.stride_s, src.stride_hkv, src.stride_hq, dst.stride_s,
             dst.stride_hkv, dst.stride_hq, g, 0,            0};
  if (g == 1) {
    x.sq = x.sh;
    x.dq = x.dh;
  }
  if (x.sh == g * x.sq && x.dh == g * x.dq) x.g = H;
  x.per_group = (x.g + hpi - 1) / hpi;
  x.passes = H ? H / x.g * x.per_group : 0;
  return x;
}

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

template <class T, bool APPEND, bool NORM>
cudaError_t launch_rows(RowsArgs& a, int D, cudaStream_t st) {
  // Few rows: the passes of a row are shared out over several warps, down to
  // one each, until about 24 warps an SM have work.
  for (const RowsPart& x : a.part) a.passes += x.passes;
  a.groups = int(std::min<int64_t>(a.passes, std::max<int64_t>(1, int64_t(sm_count()) * 24 / a.T)));
  const int64_t grid = (int64_t(a.T) * a.groups + kWarps - 1) / kWarps;  // < 2^31: T < 2^31
  const KernelId id = APPEND ? kCacheAppend : kRopeAxes;
  prof_begin(id, st);
  if (D == 128)
    rope_axes_kernel<T, 8, APPEND, NORM><<<unsigned(grid), kThreads, 0, st>>>(a);
  else if (D == 64)
    rope_axes_kernel<T, 4, APPEND, NORM><<<unsigned(grid), kThreads, 0, st>>>(a);
  else if constexpr (!APPEND)
    rope_axes_kernel<T, 0, APPEND, NORM><<<unsigned(grid), kThreads, 0, st>>>(a);
  prof_end(id, st);
  return cudaGetLastError();
}

int rope_axes(const hia_rope_plan* plan, int64_t T, const int32_t* pos, int dtype, int Hq, int Hkv, const hia_tensor& q,
              const hia_tensor& k, const hia_tensor& qo, const hia_tensor& ko, float sign, void* stream) {
  if (!plan_ok(plan) || T < 0 || Hq <= 0 || Hkv <= 0) return HIA_ERR_INVALID_ARG;
  if (dtype != HIA_BF16 && dtype != HIA_FP16 && dtype != HIA_FP32) return HIA_ERR_UNSUPPORTED;
  if (Hq % Hkv || Hq > kMaxHeads || T >= (int64_t(1) << 31)) return HIA_ERR_UNSUPPORTED;
  if (T == 0) return HIA_OK;
  const int g = Hq / Hkv;
  const size_t size = dtype == HIA_FP32 ? 4 : 2;
  if (!pos || !q.ptr || !qo.ptr || !k.ptr != !ko.ptr) return HIA_ERR_INVALID_ARG;
  int rc;
  if ((rc = rows_check(q, true, g, size)) || (rc = rows_check(qo, true, g, size))) return rc;
  if (k.ptr && ((rc = rows_check(k, false, 1, size)) || (rc = rows_check(ko, false, 1, size)))) return rc;
  if ((rc = own_rows_check(qo, T, Hkv, g)) || (k.ptr && (rc = own_rows_check(ko, T, Hkv, 1)))) return rc;
  RowsArgs a{};
  a.rope = rope_arg(plan, kTurnsPerRadian);
  const int hpi = 32 / (plan->D / 16);
  a.part[0] = make_part(q, qo, Hq, g, nullptr, hpi);
  a.part[1] = make_part(k, ko, k.ptr ? Hkv : 0, 1, nullptr, hpi);
  a.pos = pos;
  a.sign = sign;
  a.T = int(T);
  a.turn = 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == HIA_BF16   ? launch_rows<__nv_bfloat16, false, false>(a, plan->D, st)
                        : dtype == HIA_FP16 ? launch_rows<__half, false, false>(a, plan->D, st)
                                            : launch_rows<float, false, false>(a, plan->D, st);
  return e == cudaSuccess ? HIA_OK : HIA_ERR_CUDA;
}

}  // namespace

int rows_check(const hia_tensor& t, bool q_heads, int g, size_t size) {
  if (t.stride_s < 0 || t.stride_hkv < 0 || t.stride_hq < 0) return HIA_ERR_INVALID_ARG;
  const int64_t per16 = int64_t(16 / size);
  if (!aligned_to(t.ptr, 16) || t.stride_s % per16 || t.stride_hkv % per16) return HIA_ERR_UNSUPPORTED;
  if (q_heads && g > 1 && t.stride_hq % per16) return HIA_ERR_UNSUPPORTED;
  return HIA_OK;
}

int own_rows_check(const hia_tensor& t, int64_t T, int Hkv, int g) {
  const bool shared = (T > 1 && t.stride_s == 0) || (Hkv > 1 && t.stride_hkv == 0) || (g > 1 && t.stride_hq == 0);
  return shared ? HIA_ERR_UNSUPPORTED : HIA_OK;
}

int cache_check(const hia_cache* c, const hia_cache_chunk* k, int64_t T, int Hq) {
  if (!c || !k || T < 0 || Hq <= 0 || c->Hkv <= 0 || c->n_pages < 0 || k->B < 0 || k->max_pages < 0)
    return HIA_ERR_INVALID_ARG;
  if (c->dtype != HIA_BF16 && c->dtype != HIA_FP16) return HIA_ERR_UNSUPPORTED;
  if ((c->D != 64 && c->D != 128) || Hq % c->Hkv || Hq > kMaxHeads || T >= (1 << 30)) return HIA_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return HIA_ERR_UNSUPPORTED;
  if (int64_t(k->max_pages) * c->page_size >= (1 << 30)) return HIA_ERR_UNSUPPORTED;
  if (c->stride_page < 0 || c->stride_s < 0 || c->stride_h < 0 || k->page_stride < 0) return HIA_ERR_INVALID_ARG;
  if (T == 0 || k->B == 0) return HIA_OK;
  if (!c->k || !c->v || !k->rows || !k->past || !k->pages || c->n_pages == 0) return HIA_ERR_INVALID_ARG;
  if (c->stride_s == 0 || (c->Hkv > 1 && c->stride_h == 0) || (c->n_pages > 1 && c->stride_page == 0))
    return HIA_ERR_UNSUPPORTED;  // slots that share memory
  if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16) || c->stride_page % 8 || c->stride_s % 8 || c->stride_h % 8)
    return HIA_ERR_UNSUPPORTED;
  if (!aligned_to(k->rows, 4) || !aligned_to(k->past, 4) || !aligned_to(k->pages, 4)) return HIA_ERR_UNSUPPORTED;
  return HIA_OK;
}

ChunkDev chunk_dev(const hia_cache& c, const hia_cache_chunk& k, int64_t T, int* status) {
  int shift = 4;
  while ((1 << shift) < c.page_size) ++shift;
  return ChunkDev{k.rows, k.past, k.pages, k.page_stride, k.B, int(T), k.max_pages, c.n_pages, shift, status};
}

}  // namespace hia

extern "C" int hia_rope_plan_init(hia_rope_plan* p, int D, int n_axes, const int32_t* sections, double base,
                                  int per_axis) {
  if (!p || D < 16 || D > 256 || D % 16 || n_axes < 1 || n_axes > HIA_ROPE_MAX_AXES) return HIA_ERR_INVALID_ARG;
  if (!std::isfinite(base) || !(base > 0.0) || (per_axis && !sections)) return HIA_ERR_INVALID_ARG;
  if (sections) {
    int64_t sum = 0;
    for (int i = 0; i < n_axes; ++i) {
      if (sections[i] < 0) return HIA_ERR_INVALID_ARG;
      sum += sections[i];
    }
    if (sum != D / 2) return HIA_ERR_INVALID_ARG;
  }
  hia_rope_plan r{};
  r.D = D;
  r.n_axes = n_axes;
  for (int j = 0, ax = 0, first = 0; j < D / 2; ++j) {
    if (sections)
      while (j - first >= sections[ax]) first += sections[ax++];
    r.axis[j] = uint8_t(sections ? ax : j % n_axes);
    r.freq[j] = per_axis ? std::pow(base, -double(j - first) / sections[ax]) : std::pow(base, -2.0 * j / D);
  }
  for (int j = 0; j < D / 2; ++j)
    if (!std::isfinite(r.freq[j])) return HIA_ERR_INVALID_ARG;
  *p = r;
  return HIA_OK;
}

extern "C" int hia_rope_axes_tables(const hia_rope_plan* plan, int64_t T, const int32_t* pos, float* c, float* s,
                                    void* stream) {
  using namespace hia;
  if (!plan_ok(plan) || T < 0) return HIA_ERR_INVALID_ARG;
  if (T >= (int64_t(1) << 31)) return HIA_ERR_UNSUPPORTED;
  if (T == 0) return HIA_OK;
  if (!pos || !c || !s) return HIA_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t blocks = (T * (plan->D / 2) + 255) / 256;
  prof_begin(kRopeAxesTables, st);
  rope_axes_tables_kernel<<<int(std::min<int64_t>(blocks, sm_count() * 16)), 256, 0, st>>>(rope_arg(plan, 1.0),
                                                                                          T, pos, c, s);
  prof_end(kRopeAxesTables, st);
  return cudaGetLastError() == cudaSuccess ? HIA_OK : HIA_ERR_CUDA;
}

extern "C" int hia_rope_axes_fwd(const hia_rope_plan* plan, int64_t T, const int32_t* pos, int dtype, int Hq, int Hkv,
                                 hia_tensor q, hia_tensor k, hia_tensor q_out, hia_tensor k_out, void* stream) {
  return hia::rope_axes(plan, T, pos, dtype, Hq, Hkv, q, k, q_out, k_out, 1.f, stream);
}

extern "C" int hia_rope_axes_bwd(const hia_rope_plan* plan, int64_t T, const int32_t* pos, int dtype, int Hq, int Hkv,
                                 hia_tensor dq_out, hia_tensor dk_out, hia_tensor dq, hia_tensor dk, void* stream) {
  return hia::rope_axes(plan, T, pos, dtype, Hq, Hkv, dq_out, dk_out, dq, dk, -1.f, stream);
}

extern "C" int hia_cache_append(const hia_cache* cache, const hia_cache_chunk* chunk, int64_t T, int Hq,
                                const hia_rope_plan* plan, const int32_t* pos, const hia_qk_norm* norm, hia_tensor q,
                                hia_tensor k, hia_tensor v, hia_tensor q_out, void* stream) {
  using namespace hia;
  int rc = cache_check(cache, chunk, T, Hq);
  if (rc) return rc;
  const int Hkv = cache->Hkv, g = Hq / Hkv, D = cache->D;
  if (plan && (!plan_ok(plan) || plan->D != D)) return HIA_ERR_INVALID_ARG;
  if (norm) {
    if (!norm->wq || !norm->wk || !std::isfinite(norm->eps) || norm->eps < 0.f) return HIA_ERR_INVALID_ARG;
    if (!aligned_to(norm->wq, 16) || !aligned_to(norm->wk, 16)) return HIA_ERR_UNSUPPORTED;
  }
  if (T == 0 || chunk->B == 0) return HIA_OK;
  if (!k.ptr || !v.ptr || !q.ptr != !q_out.ptr || (plan && !pos)) return HIA_ERR_INVALID_ARG;
  if ((rc = rows_check(k, false, 1, 2)) || (rc = rows_check(v, false, 1, 2))) return rc;
  if (q.ptr && ((rc = rows_check(q, true, g, 2)) || (rc = rows_check(q_out, true, g, 2)) ||
                (rc = own_rows_check(q_out, T, Hkv, g))))
    return rc;
  int* status = device_status_word();
  if (!status) return HIA_ERR_CUDA;
  RowsArgs a{};
  if (plan) a.rope = rope_arg(plan, kTurnsPerRadian);
  a.turn = plan != nullptr;
  a.rope.D = D;
  const hia_tensor kd{cache->k, 0, 0, cache->stride_h, 0}, vd{cache->v, 0, 0, cache->stride_h, 0};
  const int hpi = 32 / (D / 16);
  a.part[0] = make_part(q, q_out, q.ptr ? Hq : 0, g, norm ? norm->wq : nullptr, hpi);
  a.part[1] = make_part(k, kd, Hkv, 1, norm ? norm->wk : nullptr, hpi);
  a.part[2] = make_part(v, vd, Hkv, 1, nullptr, hpi);
  a.pos = pos;
  a.sign = 1.f;
  a.eps = norm ? norm->eps : 0.f;
  a.T = int(T);
  a.chunk = chunk_dev(*cache, *chunk, T, status);
  a.stride_page = cache->stride_page;
  a.stride_s = cache->stride_s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache->dtype == HIA_BF16)
    e = norm ? launch_rows<__nv_bfloat16, true, true>(a, D, st) : launch_rows<__nv_bfloat16, true, false>(a, D, st);
  else
    e = norm ? launch_rows<__half, true, true>(a, D, st) : launch_rows<__half, true, false>(a, D, st);
  return e == cudaSuccess ? HIA_OK : HIA_ERR_CUDA;
}
