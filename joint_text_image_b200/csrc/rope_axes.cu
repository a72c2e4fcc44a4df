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

// 8 consecutive elements of a row half, as loaded (raw) and as fp32.
template <class T>
struct Half8;
template <>
struct Half8<__nv_bfloat16> {
  uint4 u;
  __device__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
  __device__ void get(float (&v)[8]) const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(h[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  __device__ void set(const float (&v)[8]) {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  }
};
template <>
struct Half8<__half> {
  uint4 u;
  __device__ void load(const __half* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ void store(__half* p) const { *reinterpret_cast<uint4*>(p) = u; }
  __device__ void get(float (&v)[8]) const {
    const __half2* h = reinterpret_cast<const __half2*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(h[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  __device__ void set(const float (&v)[8]) {
    __half2* h = reinterpret_cast<__half2*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
  }
};
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
  __device__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ void set(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
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
};

struct RowsArgs {
  RopeArg rope;
  RowsPart part[3];  // q, k and, appending, v; H = 0: absent
  const int32_t* pos;
  float sign;        // +1 turns forward, -1 back (the gradient)
  float eps;
  int T, heads, groups, turn;
  // appending: the destination of k (part 1) and v (part 2) is a slot of a page
  ChunkDev chunk;
  int64_t stride_page, stride_s, stride_h;
};

constexpr int kWarps = 8;

// A warp owns one row and a group of its heads.  Lane = hs * CPH + c holds
// elements c*8 .. c*8+7 of both halves of one head (CPH = D / 16 lanes a head,
// 32 / CPH heads a pass), so each load and store of a head is two runs of D
// bytes and its partner elements meet in one lane.  The angles of the row are
// computed once per warp, D / 64 pairs a lane, and exchanged through shared
// memory; the first heads are already on their way meanwhile.
// CPH_ = 0: D / 16 at run time (a head dimension other than 64 or 128).
template <class T, int CPH_, bool APPEND, bool NORM>
__global__ void __launch_bounds__(kWarps * 32) rope_axes_kernel(const __grid_constant__ RowsArgs a) {
  __shared__ float2 angle_s[kWarps][HIA_ROPE_MAX_PAIRS];
  constexpr int U = sizeof(T) == 4 ? 2 : 4;  // heads in flight per lane
  const int wib = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int D = CPH_ ? CPH_ * 16 : a.rope.D, cph = CPH_ ? CPH_ : D / 16, hpi = 32 / cph;
  const int c = lane % cph, hs = lane / cph;
  const bool on = hs < hpi;  // 32 % cph lanes idle
  const unsigned gmask = CPH_ ? ((CPH_ == 32 ? 0u : (1u << CPH_)) - 1u) << (hs * CPH_) : 0u;
  const int64_t items = int64_t(a.T) * a.groups;
  const int per = (a.heads + a.groups - 1) / a.groups;  // heads of a group
  for (int64_t it = int64_t(blockIdx.x) * kWarps + wib; it < items; it += int64_t(gridDim.x) * kWarps) {
    const int t = int(it / a.groups), grp = int(it % a.groups);
    const int h0 = grp * per, h1 = min(h0 + per, a.heads);

    // appending: the row's sequence (a 32-way search over the row starts) and slot
    int64_t slot_off = 0;
    bool in_page = false;
    if (APPEND) {
      int lo = 0, hi = a.chunk.B;  // rows[lo] <= t < rows[hi] if t is in a sequence
      if (t < __ldg(a.chunk.rows) || t >= __ldg(a.chunk.rows + a.chunk.B)) continue;
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + lane * step;
        const unsigned le = __ballot_sync(0xffffffffu, i < hi && __ldg(a.chunk.rows + min(i, hi)) <= t);
        // the last probe at or before t (probe 0 is, when rows is ordered)
        const int last = le ? 31 - __clz(le) : 0;
        const int nlo = lo + last * step;
        hi = min(hi, nlo + step);
        lo = nlo;
      }
      const Seq s = chunk_seq(a.chunk, lo);
      const int i = t - s.row0;
      if (i < 0 || i >= s.n) continue;  // skipped sequence
      const int at = s.past + i;
      const int page = chunk_page(a.chunk, lo, at >> a.chunk.page_shift);
      in_page = page < a.chunk.n_pages;
      slot_off = int64_t(page) * a.stride_page + int64_t(at & ((1 << a.chunk.page_shift) - 1)) * a.stride_s;
    }

    const auto part_of = [&](int& h) {  // h becomes the head within its part
      if (h < a.part[0].H) return 0;
      h -= a.part[0].H;
      if (!APPEND || h < a.part[1].H) return 1;
      h -= a.part[1].H;
      return 2;
    };
    Half8<T> lo8[U], hi8[U];
    const auto fetch = [&](int hb) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        int h = hb + u * hpi;
        if (on && h < h1) {
          const int p = part_of(h);
          const RowsPart& x = a.part[p];
          const T* src = static_cast<const T*>(x.src) + int64_t(t) * x.ss + int64_t(h / x.g) * x.sh +
                         int64_t(h % x.g) * x.sq;
          lo8[u].load(src + c * 8);
          hi8[u].load(src + D / 2 + c * 8);
        }
      }
    };
    fetch(h0 + hs);

    float cs[8], sn[8];
    if (a.turn) {
      __syncwarp();
      for (int j = lane; j < D / 2; j += 32) {
        // angle in turns, reduced to [-1/2, 1/2] in fp64; the fp32 rounding of
        // the fraction is put back to first order
        const double x = double(__ldg(a.pos + int64_t(t) * a.rope.n_axes + a.rope.axis[j])) * a.rope.turns[j];
        const double r = x - rint(x);
        const float f = float(r), d = float(r - double(f)) * 6.2831853f;
        float s0, c0;
        sincospif(2.f * f, &s0, &c0);
        angle_s[wib][j] = make_float2(fmaf(-s0, d, c0), a.sign * fmaf(c0, d, s0));
      }
      __syncwarp();
      if (on) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 v = angle_s[wib][c * 8 + k];
          cs[k] = v.x;
          sn[k] = v.y;
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        cs[k] = 1.f;
        sn[k] = 0.f;
      }
    }

    for (int hb = h0 + hs; hb - hs < h1; hb += U * hpi) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        int h = hb + u * hpi;
        if (!on || h >= h1) break;
        const int p = part_of(h);
        const RowsPart& x = a.part[p];
        if (!APPEND || p < 2) {
          float l[8], r[8], yl[8], yr[8];
          lo8[u].get(l);
          hi8[u].get(r);
          if (!APPEND || a.turn) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              yl[k] = fmaf(l[k], cs[k], -r[k] * sn[k]);
              yr[k] = fmaf(r[k], cs[k], l[k] * sn[k]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              yl[k] = l[k];
              yr[k] = r[k];
            }
          }
          if (NORM) {
            float ss = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) ss = fmaf(yl[k], yl[k], fmaf(yr[k], yr[k], ss));
#pragma unroll
            for (int o = 1; o < (CPH_ ? CPH_ : 1); o <<= 1) ss += __shfl_xor_sync(gmask, ss, o);
            const float rr = rsqrtf(ss / float(D) + a.eps);
            const float4* w = reinterpret_cast<const float4*>(x.w + c * 8);
            const float4* w2 = reinterpret_cast<const float4*>(x.w + D / 2 + c * 8);
            const float4 w0 = __ldg(w), w1 = __ldg(w + 1), v0 = __ldg(w2), v1 = __ldg(w2 + 1);
            const float wl[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
            const float wr[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              yl[k] = wl[k] * (yl[k] * rr);
              yr[k] = wr[k] * (yr[k] * rr);
            }
          }
          lo8[u].set(yl);
          hi8[u].set(yr);
        }
        T* dst = static_cast<T*>(x.dst);
        if (APPEND && p > 0) {
          if (!in_page) continue;
          dst += slot_off + int64_t(h) * a.stride_h;
        } else {
          dst += int64_t(t) * x.ds + int64_t(h / x.g) * x.dh + int64_t(h % x.g) * x.dq;
        }
        lo8[u].store(dst + c * 8);
        hi8[u].store(dst + D / 2 + c * 8);
      }
      fetch(hb + U * hpi);
    }
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

RowsPart rows_part(const hia_tensor& src, const hia_tensor& dst, int H, int g, const float* w) {
  return RowsPart{src.ptr, dst.ptr, w, src.stride_s, src.stride_hkv, src.stride_hq, dst.stride_s, dst.stride_hkv,
                  dst.stride_hq, H, g};
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
void launch_rows(RowsArgs& a, int D, cudaStream_t st) {
  // Few rows: the heads of a row are shared out over several warps, until
  // about 16 warps an SM have work.
  const int n_sm = sm_count();
  const int hpi = std::max(1, 32 / (D / 16));
  const int most = (a.heads + hpi - 1) / hpi;
  a.groups = int(std::min<int64_t>(most, std::max<int64_t>(1, int64_t(n_sm) * 16 / std::max(a.T, 1))));
  const int64_t blocks = (int64_t(a.T) * a.groups + kWarps - 1) / kWarps;
  const int grid = int(std::min<int64_t>(blocks, int64_t(n_sm) * 32));
  const KernelId id = APPEND ? kCacheAppend : kRopeAxes;
  prof_begin(id, st);
  if (D == 128)
    rope_axes_kernel<T, 8, APPEND, NORM><<<grid, kWarps * 32, 0, st>>>(a);
  else if (D == 64)
    rope_axes_kernel<T, 4, APPEND, NORM><<<grid, kWarps * 32, 0, st>>>(a);
  else if constexpr (!APPEND)
    rope_axes_kernel<T, 0, APPEND, NORM><<<grid, kWarps * 32, 0, st>>>(a);
  prof_end(id, st);
}

int rope_axes(const hia_rope_plan* plan, int64_t T, const int32_t* pos, int dtype, int Hq, int Hkv, const hia_tensor& q,
              const hia_tensor& k, const hia_tensor& qo, const hia_tensor& ko, float sign, void* stream) {
  if (!plan_ok(plan) || T < 0 || Hq <= 0 || Hkv <= 0) return HIA_ERR_INVALID_ARG;
  if (dtype != HIA_BF16 && dtype != HIA_FP16 && dtype != HIA_FP32) return HIA_ERR_UNSUPPORTED;
  if (Hq % Hkv || T >= (int64_t(1) << 31)) return HIA_ERR_UNSUPPORTED;
  if (T == 0) return HIA_OK;
  const int g = Hq / Hkv;
  const size_t size = dtype == HIA_FP32 ? 4 : 2;
  if (!pos || !q.ptr || !qo.ptr || !k.ptr != !ko.ptr) return HIA_ERR_INVALID_ARG;
  int rc;
  if ((rc = rows_check(q, true, g, size)) || (rc = rows_check(qo, true, g, size))) return rc;
  if (k.ptr && ((rc = rows_check(k, false, 1, size)) || (rc = rows_check(ko, false, 1, size)))) return rc;
  RowsArgs a{};
  a.rope = rope_arg(plan, kTurnsPerRadian);
  a.part[0] = rows_part(q, qo, Hq, g, nullptr);
  a.part[1] = rows_part(k, ko, k.ptr ? Hkv : 0, 1, nullptr);
  a.pos = pos;
  a.sign = sign;
  a.T = int(T);
  a.heads = Hq + a.part[1].H;
  a.turn = 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == HIA_BF16)
    launch_rows<__nv_bfloat16, false, false>(a, plan->D, st);
  else if (dtype == HIA_FP16)
    launch_rows<__half, false, false>(a, plan->D, st);
  else
    launch_rows<float, false, false>(a, plan->D, st);
  return cudaGetLastError() == cudaSuccess ? HIA_OK : HIA_ERR_CUDA;
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
  if ((c->D != 64 && c->D != 128) || Hq % c->Hkv || T >= (1 << 30)) return HIA_ERR_UNSUPPORTED;
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
  a.part[0] = rows_part(q, q_out, q.ptr ? Hq : 0, g, norm ? norm->wq : nullptr);
  a.part[1] = rows_part(k, kd, Hkv, 1, norm ? norm->wk : nullptr);
  a.part[2] = rows_part(v, vd, Hkv, 1, nullptr);
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
  if (cache->dtype == HIA_BF16) {
    if (norm) launch_rows<__nv_bfloat16, true, true>(a, D, st);
    else launch_rows<__nv_bfloat16, true, false>(a, D, st);
  } else {
    if (norm) launch_rows<__half, true, true>(a, D, st);
    else launch_rows<__half, true, false>(a, D, st);
  }
  return cudaGetLastError() == cudaSuccess ? HIA_OK : HIA_ERR_CUDA;
}
