// Norm of every query and key head and its rotation to its row's position, in one pass
// (hymba_qk_norm_rope):
//   y = x / sqrt(mean(x^2) + eps) * w;   pair (a, b) -> m (a cos - b sin, a sin + b cos)
#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace hymba {

namespace {

constexpr int kHeadWarps = 8;
constexpr int kAhead = 4;
constexpr int kMaxPairs = 128;  // head_dim <= 256
constexpr double kTwoPi = 6.283185307179586476925286766559;

struct HeadsParams {
  hymba_qk_norm_rope_args a;
  int lanes;       // lanes per head: a power of two, 8 elements each
  int parts;       // units per row: the heads of a row are split over this many warps
  int chunk;       // loads (of 32 / lanes heads) a warp keeps in flight, at most kAhead
  long long units; // batch * n_rows * parts
  double turns[kMaxPairs];  // f_i / (2 pi): turns per position
};

// Four elements of a head: 8 bytes of bf16, 16 of fp32.
template <typename T>
struct Vec4;
template <>
struct Vec4<__nv_bfloat16> {
  using R = uint2;
  static __device__ __forceinline__ void get(const R &r, float *x) {
    x[0] = bf16_lo(r.x), x[1] = bf16_hi(r.x), x[2] = bf16_lo(r.y), x[3] = bf16_hi(r.y);
  }
  static __device__ __forceinline__ R put(const float *x) {
    return make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  }
};
template <>
struct Vec4<float> {
  using R = float4;
  static __device__ __forceinline__ void get(const R &r, float *x) { x[0] = r.x, x[1] = r.y, x[2] = r.z, x[3] = r.w; }
  static __device__ __forceinline__ R put(const float *x) { return make_float4(x[0], x[1], x[2], x[3]); }
};

// Which eight elements of a head a lane holds, and where an element's pair is.
enum Partner {
  kNone,    // no rotation: elements 8 l ..
  kPairs,   // pairs (2i, 2i+1): elements 8 l .., four pairs
  kHalves,  // halves of the whole head: elements 4 l .. and d/2 + 4 l .., four pairs
  kShared   // halves of a part of the head: elements 8 l .., the pairs through shared memory
};

// A warp takes one unit: a row of a sequence and a share of its heads.  Its lanes first
// compute the row's angles, one pair each (fp64 turns p * f / 2 pi, of which only the
// fraction goes to the fp32 sincospi), and keep the factors of their own pairs in registers
// for all heads of the unit.  32 / lanes heads are in flight per load, kAhead loads ahead of
// the arithmetic.
//
// Bound by instructions more than by HBM: per element a share of the conversions, of the
// norm's sum over the head's lanes and of the rotation.  With a head's halves in lanes of
// their own the rotation took eight shuffles per eight elements (109 us at 8 x 4224 rows of
// 30 heads); a lane that holds both elements of its pairs needs none.
template <typename T, int PARTNER>
__global__ void __launch_bounds__(32 * kHeadWarps)
    qk_norm_rope_kernel(const __grid_constant__ HeadsParams p) {
  pdl_wait();
  pdl_trigger();
  using V = Vec4<T>;
  __shared__ float2 s_trig[PARTNER == kNone ? 1 : kHeadWarps * kMaxPairs];
  __shared__ float s_stage[PARTNER == kShared ? kHeadWarps * 256 : 1];
  const hymba_qk_norm_rope_args &a = p.a;
  const int warp = warp_id(), lane = lane_id();
  const long long unit = (long long)blockIdx.x * kHeadWarps + warp;
  if (unit >= p.units) return;
  const int part = int(unit % p.parts);
  const long long row_id = unit / p.parts;
  const int r = int(row_id % a.n_rows);
  const long long b = row_id / a.n_rows;
  const int lanes = p.lanes, li = lane & (lanes - 1), slot = lane / lanes, per = 32 / lanes;
  const int d = a.head_dim, rot = a.rope.dim, half = rot >> 1;
  const bool live = 8 * li < d;
  // the lane's elements: four from e0, four from e1
  const int e0 = PARTNER == kHalves ? 4 * li : 8 * li, e1 = PARTNER == kHalves ? half + 4 * li : e0 + 4;

  // kPairs, kHalves: cos and sin of the lane's four pairs; kShared: of its eight elements'
  constexpr int NF = PARTNER == kNone ? 1 : PARTNER == kShared ? 8 : 4;
  float cs[NF], sn[NF];
  if constexpr (PARTNER != kNone) {
    const double pos = double(a.pos0 + (a.positions ? a.positions[row_id] : (long long)r));
    float2 *trig = s_trig + warp * kMaxPairs;
    for (int i = lane; i < half; i += 32) {
      double t = pos * p.turns[i];
      t -= rint(t);
      float s, c;
      sincospif(float(2.0 * t), &s, &c);
      trig[i] = make_float2(c * a.rope.attn_factor, s * a.rope.attn_factor);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const int i = PARTNER == kPairs ? 4 * li + j : PARTNER == kHalves ? e0 + j : e0 + j < half ? e0 + j : e0 + j - half;
      const float2 t = i < half ? trig[i] : make_float2(1.f, 0.f);  // behind the rotated part
      cs[j] = t.x;
      sn[j] = PARTNER == kShared && e0 + j < half ? -t.y : t.y;
    }
  }

  const int nq = a.q.n_heads, heads = nq + a.k.n_heads;
  const int groups = (heads + per - 1) / per;
  const float inv_d = 1.0f / float(d);
  const T *qi = reinterpret_cast<const T *>(a.q.in) + b * a.q.in_batch + r * a.q.in_row;
  const T *ki = reinterpret_cast<const T *>(a.k.in) + b * a.k.in_batch + r * a.k.in_row;
  T *qo = reinterpret_cast<T *>(a.q.out) + b * a.q.out_batch + r * a.q.out_row;
  T *ko = reinterpret_cast<T *>(a.k.out) + b * a.k.out_batch + r * a.k.out_row;
  for (int g0 = part * p.chunk; g0 < groups; g0 += p.parts * p.chunk) {
    typename V::R ra[kAhead], rb[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int hh = (g0 + u) * per + slot;
      ra[u] = rb[u] = typename V::R{};
      if (live && u < p.chunk && hh < heads) {
        const T *src = hh < nq ? qi + hh * a.q.in_head : ki + (hh - nq) * a.k.in_head;
        ra[u] = *reinterpret_cast<const typename V::R *>(src + e0);
        rb[u] = *reinterpret_cast<const typename V::R *>(src + e1);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (u >= p.chunk || g0 + u >= groups) break;  // the same for the whole warp
      const int hh = (g0 + u) * per + slot;
      float x[8];
      V::get(ra[u], x);
      V::get(rb[u], x + 4);
      if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
        for (int m = lanes >> 1; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float inv = rsqrtf(fmaf(ss, inv_d, a.eps));
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= inv;
        const float *weight = hh < nq ? a.q.weight : a.k.weight;
        if (weight && live) {
          const float4 w0 = __ldg(reinterpret_cast<const float4 *>(weight + e0));
          const float4 w1 = __ldg(reinterpret_cast<const float4 *>(weight + e1));
          const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] *= w[j];
        }
      }
      float y[8];
      if constexpr (PARTNER == kNone) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[j];
      } else if constexpr (PARTNER == kPairs || PARTNER == kHalves) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int f = PARTNER == kPairs ? 2 * j : j, s = PARTNER == kPairs ? 2 * j + 1 : j + 4;
          y[f] = fmaf(x[f], cs[j], -x[s] * sn[j]);
          y[s] = fmaf(x[s], cs[j], x[f] * sn[j]);
          if (PARTNER == kPairs && e0 + 2 * j >= rot) {  // not rotated: as it is, whatever its pair holds
            y[f] = x[f];
            y[s] = x[s];
          }
        }
      } else {
        // each lane's eight elements at 8 lane: the warp's heads side by side
        float *st = s_stage + warp * 256;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) st[8 * lane + j] = x[j];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = e0 + j;
          const int other = e < half ? e + half : e - half;
          y[j] = e < rot ? fmaf(x[j], cs[j], st[8 * (lane - li) + other] * sn[j]) : x[j];
        }
      }
      if (live && hh < heads) {
        T *dst = hh < nq ? qo + hh * a.q.out_head : ko + (hh - nq) * a.k.out_head;
        *reinterpret_cast<typename V::R *>(dst + e0) = V::put(y);
        *reinterpret_cast<typename V::R *>(dst + e1) = V::put(y + 4);
      }
    }
  }
}

template <typename T>
void heads_launch(const HeadsParams &p, int partner, unsigned grid, cudaStream_t s) {
  const dim3 g(grid), blk(32 * kHeadWarps);
  if (partner == kNone) launch_kernel(qk_norm_rope_kernel<T, kNone>, g, blk, 0, s, p);
  else if (partner == kPairs) launch_kernel(qk_norm_rope_kernel<T, kPairs>, g, blk, 0, s, p);
  else if (partner == kHalves) launch_kernel(qk_norm_rope_kernel<T, kHalves>, g, blk, 0, s, p);
  else launch_kernel(qk_norm_rope_kernel<T, kShared>, g, blk, 0, s, p);
}

}  // namespace

hymba_status qk_norm_rope(const hymba_qk_norm_rope_args &a, cudaStream_t s) {
  HeadsParams p;
  p.a = a;
  p.lanes = 1;
  while (p.lanes * 8 < a.head_dim) p.lanes *= 2;
  const int half = a.rope.dim / 2;
  for (int i = 0; i < half; ++i) {
    const double f = pow(a.rope.base, -2.0 * i / a.rope.dim);
    double t = f / kTwoPi;
    if (a.rope.scaling == HYMBA_ROPE_SCALE_LINEAR) {
      t /= a.rope.factor;
    } else if (a.rope.scaling == HYMBA_ROPE_SCALE_WAVELENGTH) {
      double keep = (a.rope.orig_len * t - a.rope.low_turns) / (a.rope.high_turns - a.rope.low_turns);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      t = keep * t + (1.0 - keep) * t / a.rope.factor;
    }
    p.turns[i] = t;
  }
  for (int i = half; i < kMaxPairs; ++i) p.turns[i] = 0.0;
  const int partner = half == 0 ? kNone
                      : a.rope.layout == HYMBA_ROPE_PAIRS ? kPairs
                      : a.rope.dim == a.head_dim ? kHalves : kShared;
  // One warp per row amortises the row's angles over all of its heads; with too few rows to
  // give every SM 16 warps, a row's heads are split over several warps, down to one load of
  // 32 / lanes heads each.
  const int heads = a.q.n_heads + a.k.n_heads, per = 32 / p.lanes;
  const long long rows = (long long)a.batch * a.n_rows;
  const int loads = (heads + per - 1) / per;
  const long long want = (148 * 16 + rows - 1) / rows;
  p.parts = int(want < loads ? want : loads);
  p.chunk = (loads + p.parts - 1) / p.parts;
  if (p.chunk > kAhead) p.chunk = kAhead;
  p.units = rows * p.parts;
  const long long grid = (p.units + kHeadWarps - 1) / kHeadWarps;
  if (grid > 0x7fffffffLL) {
    set_error("too many rows");
    return HYMBA_ERR_UNSUPPORTED;
  }
  if (a.dtype == HYMBA_BF16) heads_launch<__nv_bfloat16>(p, partner, (unsigned)grid, s);
  else heads_launch<float>(p, partner, (unsigned)grid, s);
  note_launch(1);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("head norm/rotation launch failed: %s", cudaGetErrorString(e));
    return HYMBA_ERR_CUDA;
  }
  return HYMBA_OK;
}

}  // namespace hymba
