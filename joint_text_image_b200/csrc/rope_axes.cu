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

// 8 consecutive elements of a row half, as loaded and as fp32 pairs.
template <class T>
struct Half8 {
  uint4 u;
  __device__ void load(const T* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = u; }
  __device__ void get(float2 (&v)[4]) const;
  __device__ void set(const float2 (&v)[4]);
};
template <>
__device__ __forceinline__ void Half8<__nv_bfloat16>::get(float2 (&v)[4]) const {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(&u)[i]);
}
template <>
__device__ __forceinline__ void Half8<__nv_bfloat16>::set(const float2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) reinterpret_cast<__nv_bfloat162*>(&u)[i] = __floats2bfloat162_rn(v[i].x, v[i].y);
}
template <>
__device__ __forceinline__ void Half8<__half>::get(float2 (&v)[4]) const {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __half22float2(reinterpret_cast<const __half2*>(&u)[i]);
}
template <>
__device__ __forceinline__ void Half8<__half>::set(const float2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) reinterpret_cast<__half2*>(&u)[i] = __floats2half2_rn(v[i].x, v[i].y);
}
template <>
struct Half8<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ void get(float2 (&v)[4]) const {
    v[0] = make_float2(a.x, a.y);
    v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y);
    v[3] = make_float2(b.z, b.w);
  }
  __device__ void set(const float2 (&v)[4]) {
    a = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    b = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  }
};

// One tensor of the pass: head h of row t is read at src + t*ss + (h/g)*sh +
// (h%g)*sq and written at dst + t*ds + (h/g)*dh + (h%g)*dq (elements).
struct RowsPart {
  const void* src;
  void* dst;
  const float* w;  // QK RMSNorm weight (append with a norm)
  int64_t ss, sh, sq, ds, dh, dq;
  int H, g;
  uint32_t inv_g;  // ceil(2^32 / g): h / g = h * inv_g >> 32 for h < 2^16 (0: g = 1)
};

struct RowsArgs {
  RopeArg rope;
  RowsPart part[3];  // q, k and, appending, v; H = 0: absent
  const int32_t* pos;
  float sign;        // +1 turns forward, -1 back (the gradient)
  float eps;
  int T, heads, turn;
  int rows, groups;  // rows of a block, and blocks that share a row's heads
  // appending: the destination of k (part 1) and v (part 2) is a slot of a page
  ChunkDev chunk;
  int64_t stride_page, stride_s, stride_h;
};

constexpr int kThreads = 128;
constexpr int kMaxRows = 2;  // rows of a block
constexpr int kMaxHeads = 1 << 16;

// A block owns `rows` rows (2; 1 where rows are few) and a group of their
// heads.  A head is CPH = D / 16 lanes: lane c holds elements c*8 .. c*8+7 of
// both halves, so each load and store of a head is two runs of D bytes and
// partner elements meet in one lane.  The block's (row, head) pairs go round
// its 128 / CPH lane groups, U at a time in flight; the first U are on their
// way while the angles are computed, once per row, and exchanged through
// shared memory (two rows and short blocks: 10244 rows of 40 heads in 2.2 waves
// of longer blocks left a third of the SMs idle at the end).
// CPH_ = 0: D / 16 at run time (a head dimension other than 64 or 128).
template <class T, int CPH_, bool APPEND, bool NORM>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 6 : 8) rope_axes_kernel(const __grid_constant__ RowsArgs a) {
  __shared__ float2 angle_s[kMaxRows][HIA_ROPE_MAX_PAIRS];  // (cos, sin) of pair j
  __shared__ float w_s[NORM ? 2 : 1][NORM ? 128 : 1];
  __shared__ int64_t slot_s[kMaxRows];  // appending: element offset of the row's slot
  __shared__ int where_s[kMaxRows];     // appending: 0 not in a sequence, 1 in one without a page, 2 with one
  constexpr int U = sizeof(T) == 4 ? 2 : 3;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cph = CPH_ ? CPH_ : a.rope.D / 16, half = cph * 8, n_lg = kThreads / cph;
  const int c = tid % cph, lg = tid / cph;
  const unsigned gmask = CPH_ ? ((1u << CPH_) - 1u) << (lane & ~(CPH_ - 1)) : 0u;
  const int per = (a.heads + a.groups - 1) / a.groups;  // heads of a group
  const int t0 = int(blockIdx.x / a.groups) * a.rows, h0 = int(blockIdx.x % a.groups) * per;
  const int n_h = min(per, a.heads - h0), n_t = min(a.rows, a.T - t0);
  const int n = n_h * n_t;  // (row, head) pairs
  if (n <= 0) return;

  struct Place {
    int row, part, h, kv, in;
  };
  const auto place = [&](int i) {
    Place p;
    p.row = i >= n_h ? 1 : 0;
    p.h = h0 + i - p.row * n_h;
    p.part = 0;
    if (p.h >= a.part[0].H) {
      p.h -= a.part[0].H;
      p.part = 1;
      if (APPEND && p.h >= a.part[1].H) {
        p.h -= a.part[1].H;
        p.part = 2;
      }
    }
    const RowsPart& x = a.part[p.part];
    p.kv = x.inv_g ? int(__umulhi(uint32_t(p.h), x.inv_g)) : p.h;
    p.in = p.h - p.kv * x.g;
    return p;
  };
  Half8<T> lo[U], hi[U];
  const auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * n_lg;
      if (i < n && lg < n_lg) {
        const Place p = place(i);
        const RowsPart& x = a.part[p.part];
        const T* src = static_cast<const T*>(x.src) + (t0 + p.row) * x.ss + p.kv * x.sh + p.in * x.sq + c * 8;
        lo[u].load(src);
        hi[u].load(src + half);
      }
    }
  };
  fetch(lg);

  if (!APPEND || a.turn) {
    for (int i = tid; i < n_t * half; i += kThreads) {
      const int row = i >= half ? 1 : 0, j = i - row * half;
      // angle in turns, reduced to [-1/2, 1/2] in fp64; the fp32 rounding of
      // the fraction is put back to first order
      const double x = double(__ldg(a.pos + int64_t(t0 + row) * a.rope.n_axes + a.rope.axis[j])) * a.rope.turns[j];
      const double r = x - rint(x);
      const float f = float(r), d = float(r - double(f)) * 6.2831853f;
      float s0, c0;
      sincospif(2.f * f, &s0, &c0);
      angle_s[row][j] = make_float2(fmaf(-s0, d, c0), a.sign * fmaf(c0, d, s0));
    }
  }
  if (NORM)
    for (int i = tid; i < 4 * half; i += kThreads)
      w_s[i >= 2 * half][i % (2 * half)] = __ldg((i >= 2 * half ? a.part[1].w : a.part[0].w) + i % (2 * half));
  // appending: each row's sequence (a 32-way search over the row starts) and slot
  if (APPEND && warp < n_t) {
    const int t = t0 + warp;
    int where = 0;
    int64_t slot = 0;
    if (t >= __ldg(a.chunk.rows) && t < __ldg(a.chunk.rows + a.chunk.B)) {
      int l = 0, h = a.chunk.B;  // rows[l] <= t < rows[h]
      while (h - l > 1) {
        const int step = (h - l + 31) / 32;
        const int i = l + lane * step;
        const unsigned le = __ballot_sync(0xffffffffu, i < h && __ldg(a.chunk.rows + min(i, h)) <= t);
        // the last probe at or before t (probe 0 is, when rows is ordered)
        const int last = le ? 31 - __clz(le) : 0;
        const int nl = l + last * step;
        h = min(h, nl + step);
        l = nl;
      }
      const Seq s = chunk_seq(a.chunk, l);
      const int i = t - s.row0;
      if (i >= 0 && i < s.n) {  // not in a skipped sequence
        const int at = s.past + i;
        const int page = chunk_page(a.chunk, l, at >> a.chunk.page_shift);
        where = page < a.chunk.n_pages ? 2 : 1;
        slot = int64_t(page) * a.stride_page + int64_t(at & ((1 << a.chunk.page_shift) - 1)) * a.stride_s;
      }
    }
    if (lane == 0) {
      where_s[warp] = where;
      slot_s[warp] = slot;
    }
  }
  __syncthreads();

  for (int i0 = lg; i0 - lg < n; i0 += U * n_lg) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * n_lg;
      if (i >= n || lg >= n_lg) break;
      const Place p = place(i);
      const RowsPart& x = a.part[p.part];
      if (!APPEND || p.part < 2) {
        float2 l[4], r[4];
        lo[u].get(l);
        hi[u].get(r);
        if (!APPEND || a.turn) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(&angle_s[p.row][c * 8 + 2 * k]);
            const float2 cs = make_float2(v.x, v.z), sn = make_float2(v.y, v.w), ns = make_float2(-v.y, -v.w);
            const float2 y = __ffma2_rn(r[k], ns, __fmul2_rn(l[k], cs));
            r[k] = __ffma2_rn(l[k], sn, __fmul2_rn(r[k], cs));
            l[k] = y;
          }
        }
        if (NORM) {
          float2 q2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int k = 0; k < 4; ++k) q2 = __ffma2_rn(l[k], l[k], __ffma2_rn(r[k], r[k], q2));
          float q = q2.x + q2.y;
#pragma unroll
          for (int o = 1; o < (CPH_ ? CPH_ : 1); o <<= 1) q += __shfl_xor_sync(gmask, q, o);
          const float nr = rsqrtf(q / float(2 * half) + a.eps);
          const float2 n2 = make_float2(nr, nr);
          const float2* wl = reinterpret_cast<const float2*>(w_s[p.part] + c * 8);
          const float2* wr = reinterpret_cast<const float2*>(w_s[p.part] + half + c * 8);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            l[k] = __fmul2_rn(wl[k], __fmul2_rn(l[k], n2));
            r[k] = __fmul2_rn(wr[k], __fmul2_rn(r[k], n2));
          }
        }
        lo[u].set(l);
        hi[u].set(r);
      }
      T* dst = static_cast<T*>(x.dst) + c * 8;
      if (APPEND && where_s[p.row] < (p.part > 0 ? 2 : 1)) continue;
      if (APPEND && p.part > 0)
        dst += slot_s[p.row] + p.h * a.stride_h;
      else
        dst += (t0 + p.row) * x.ds + p.kv * x.dh + p.in * x.dq;
      lo[u].store(dst);
      hi[u].store(dst + half);
    }
    fetch(i0 + U * n_lg);
  }
}

__global__ void __launch_bounds__(256) rope_axes_tables_kernel(const __grid_constant__ RopeArg plan,
                                                               int64_t T,
                                                               const int32_t* __restrict__ pos,
                                                               float* __restrict__ cos_out,
                                                               float* __restrict__ sin_out) {
  // turns[] holds radians here: angle and cos/sin in fp64, rounded once, as
  // the 2D tables do
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

RowsPart make_part(const hia_tensor& src, const hia_tensor& dst, int H, int g, const float* w) {
  return RowsPart{src.ptr, dst.ptr, w, src.stride_s, src.stride_hkv, src.stride_hq, dst.stride_s, dst.stride_hkv,
                  dst.stride_hq, H, g, g > 1 ? uint32_t(((uint64_t(1) << 32) + g - 1) / g) : 0u};
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
  // Few rows: one a block, and its heads shared out over blocks, down to one
  // head per lane group, until about 8 blocks an SM have work.
  const int64_t slots = int64_t(sm_count()) * 8;
  const int n_lg = kThreads / (D / 16);
  a.rows = a.T >= 2 * slots ? kMaxRows : 1;
  a.groups = a.T >= slots ? 1 : int(std::min<int64_t>((a.heads + n_lg - 1) / n_lg, std::max<int64_t>(1, slots / a.T)));
  const int64_t grid = (int64_t(a.T) + a.rows - 1) / a.rows * a.groups;  // < 2^31: few rows where groups > 1
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
  RowsArgs a{};
  a.rope = rope_arg(plan, kTurnsPerRadian);
  a.part[0] = make_part(q, qo, Hq, g, nullptr);
  a.part[1] = make_part(k, ko, k.ptr ? Hkv : 0, 1, nullptr);
  a.pos = pos;
  a.sign = sign;
  a.T = int(T);
  a.heads = Hq + a.part[1].H;
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
  if (q.ptr && ((rc = rows_check(q, true, g, 2)) || (rc = rows_check(q_out, true, g, 2)))) return rc;
  int* status = device_status_word();
  if (!status) return HIA_ERR_CUDA;
  RowsArgs a{};
  if (plan) a.rope = rope_arg(plan, kTurnsPerRadian);
  a.turn = plan != nullptr;
  a.rope.D = D;
  hia_tensor kd{cache->k, 0, 0, 0, 0}, vd{cache->v, 0, 0, 0, 0};
  a.part[0] = make_part(q, q_out, q.ptr ? Hq : 0, g, norm ? norm->wq : nullptr);
  a.part[1] = make_part(k, kd, Hkv, 1, norm ? norm->wk : nullptr);
  a.part[2] = make_part(v, vd, Hkv, 1, nullptr);
  a.pos = pos;
  a.sign = 1.f;
  a.eps = norm ? norm->eps : 0.f;
  a.T = int(T);
  a.heads = a.part[0].H + 2 * Hkv;
  a.chunk = chunk_dev(*cache, *chunk, T, status);
  a.stride_page = cache->stride_page;
  a.stride_s = cache->stride_s;
  a.stride_h = cache->stride_h;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache->dtype == HIA_BF16)
    e = norm ? launch_rows<__nv_bfloat16, true, true>(a, D, st) : launch_rows<__nv_bfloat16, true, false>(a, D, st);
  else
    e = norm ? launch_rows<__half, true, true>(a, D, st) : launch_rows<__half, true, false>(a, D, st);
  return e == cudaSuccess ? HIA_OK : HIA_ERR_CUDA;
}
