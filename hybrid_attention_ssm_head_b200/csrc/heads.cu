// Norm of every query and key head and its rotation to its row's position, in one pass
// (hymba_qk_norm_rope):
//   y = x / sqrt(mean(x^2) + eps) * w;   pair (a, b) -> m (a cos - b sin, a sin + b cos)
#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace hymba {

namespace {

constexpr int kHeadWarps = 4;
constexpr int kAhead = 4;
constexpr int kMaxPairs = 128;  // head_dim <= 256
constexpr double kTwoPi = 6.283185307179586476925286766559;

struct HeadsParams {
  hymba_qk_norm_rope_args a;
  int lanes;       // lanes per head: a power of two, 8 elements each
  int parts;       // units per row: the heads of a row are split over this many warps
  int chunk;       // loads (of 32 / lanes heads) a warp keeps in flight, at most kAhead
  unsigned units;  // batch * n_rows * parts
  double turns[kMaxPairs];  // f_i / (2 pi): turns per position
};

// Four elements of a head: 8 bytes of bf16, 16 of fp32.
template <typename T>
struct Vec4;
template <>
struct Vec4<__nv_bfloat16> {
  using R = uint2;
  static __device__ __forceinline__ void get(const R &r, float2 *x) {
    x[0] = make_float2(bf16_lo(r.x), bf16_hi(r.x));
    x[1] = make_float2(bf16_lo(r.y), bf16_hi(r.y));
  }
  static __device__ __forceinline__ R put(const float2 *x) {
    return make_uint2(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y));
  }
};
template <>
struct Vec4<float> {
  using R = float4;
  static __device__ __forceinline__ void get(const R &r, float2 *x) {
    x[0] = make_float2(r.x, r.y);
    x[1] = make_float2(r.z, r.w);
  }
  static __device__ __forceinline__ R put(const float2 *x) { return make_float4(x[0].x, x[0].y, x[1].x, x[1].y); }
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
// 30 heads of 64); a lane that holds both elements of its pairs needs none: 62 us, 4.2 TB/s.
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
  const unsigned unit = blockIdx.x * kHeadWarps + warp;
  if (unit >= p.units) return;
  const unsigned row_id = p.parts == 1 ? unit : unit / (unsigned)p.parts;
  const int part = int(unit - row_id * p.parts);
  const int b = int(row_id / (unsigned)a.n_rows), r = int(row_id - b * (unsigned)a.n_rows);
  const int lanes = p.lanes, li = lane & (lanes - 1), slot = lane / lanes, per = 32 / lanes;
  const int d = a.head_dim, rot = a.rope.dim, half = rot >> 1;
  const bool live = 8 * li < d;
  // the lane's elements: four from e0, four from e1
  const int e0 = PARTNER == kHalves ? 4 * li : 8 * li, e1 = PARTNER == kHalves ? half + 4 * li : e0 + 4;

  const int nq = a.q.n_heads, heads = nq + a.k.n_heads;
  const int groups = (heads + per - 1) / per;
  const float inv_d = 1.0f / float(d);
  const T *qi = reinterpret_cast<const T *>(a.q.in) + b * a.q.in_batch + r * a.q.in_row;
  const T *ki = reinterpret_cast<const T *>(a.k.in) + b * a.k.in_batch + r * a.k.in_row;
  T *qo = reinterpret_cast<T *>(a.q.out) + b * a.q.out_batch + r * a.q.out_row;
  T *ko = reinterpret_cast<T *>(a.k.out) + b * a.k.out_batch + r * a.k.out_row;

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
      // elements two by two: e0, e0 + 1 | .. | e1 + 2, e1 + 3
      float2 x[4];
      V::get(ra[u], x);
      V::get(rb[u], x + 2);
      if (a.norm) {
        const float2 s2 = ffma2(x[3], x[3], ffma2(x[2], x[2], ffma2(x[1], x[1], fmul2(x[0], x[0]))));
        float ss = s2.x + s2.y;
        for (int m = lanes >> 1; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float inv = rsqrtf(fmaf(ss, inv_d, a.eps));
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = fmul2(x[j], make_float2(inv, inv));
        const float *weight = hh < nq ? a.q.weight : a.k.weight;
        if (weight && live) {
          const float4 w0 = __ldg(reinterpret_cast<const float4 *>(weight + e0));
          const float4 w1 = __ldg(reinterpret_cast<const float4 *>(weight + e1));
          x[0] = fmul2(x[0], make_float2(w0.x, w0.y));
          x[1] = fmul2(x[1], make_float2(w0.z, w0.w));
          x[2] = fmul2(x[2], make_float2(w1.x, w1.y));
          x[3] = fmul2(x[3], make_float2(w1.z, w1.w));
        }
      }
      float2 y[4];
      if constexpr (PARTNER == kNone) {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = x[j];
      } else if constexpr (PARTNER == kPairs) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[j] = make_float2(fmaf(x[j].x, cs[j], -x[j].y * sn[j]), fmaf(x[j].y, cs[j], x[j].x * sn[j]));
          if (e0 + 2 * j >= rot) y[j] = x[j];  // not rotated: as it is, whatever its pair holds
        }
      } else if constexpr (PARTNER == kHalves) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 c2 = make_float2(cs[2 * j], cs[2 * j + 1]), s2 = make_float2(sn[2 * j], sn[2 * j + 1]);
          const float2 n2 = make_float2(-s2.x, -s2.y);
          y[j] = ffma2(x[j], c2, fmul2(x[j + 2], n2));
          y[j + 2] = ffma2(x[j + 2], c2, fmul2(x[j], s2));
        }
      } else {
        // each lane's eight elements at 8 lane: the warp's heads side by side
        float *st = s_stage + warp * 256;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<float2 *>(&st[8 * lane + 2 * j]) = x[j];
        __syncwarp();
        auto turn = [&](float v, int j) {
          const int e = e0 + j, other = e < half ? e + half : e - half;
          return e < rot ? fmaf(v, cs[j], st[8 * (lane - li) + other] * sn[j]) : v;
        };
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = make_float2(turn(x[j].x, 2 * j), turn(x[j].y, 2 * j + 1));
      }
      if (live && hh < heads) {
        T *dst = hh < nq ? qo + hh * a.q.out_head : ko + (hh - nq) * a.k.out_head;
        *reinterpret_cast<typename V::R *>(dst + e0) = V::put(y);
        *reinterpret_cast<typename V::R *>(dst + e1) = V::put(y + 2);
      }
    }
  }
}

template <typename T>
void heads_launch(const HeadsParams &p, int partner, dim3 g, cudaStream_t s) {
  const dim3 blk(32 * kHeadWarps);
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
  // 32 / lanes heads each.  (A warp over the same row of several sequences, which could share
  // the angles, was slower: 73 against 64 us at 8 x 4224 rows of 30 heads.)
  const int heads = a.q.n_heads + a.k.n_heads, per = 32 / p.lanes;
  const long long rows = (long long)a.batch * a.n_rows;
  const int loads = (heads + per - 1) / per;
  const long long want = (148 * 16 + rows - 1) / rows;
  p.parts = int(want < loads ? want : loads);
  p.chunk = (loads + p.parts - 1) / p.parts;
  if (p.chunk > kAhead) p.chunk = kAhead;
  const long long units = rows * p.parts;
  if (units > 0x7fffffffLL) {
    set_error("too many rows");
    return HYMBA_ERR_UNSUPPORTED;
  }
  p.units = (unsigned)units;
  const dim3 grid((unsigned)((units + kHeadWarps - 1) / kHeadWarps));
  if (a.dtype == HYMBA_BF16) heads_launch<__nv_bfloat16>(p, partner, grid, s);
  else heads_launch<float>(p, partner, grid, s);
  note_launch(1);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("head norm/rotation launch failed: %s", cudaGetErrorString(e));
    return HYMBA_ERR_CUDA;
  }
  return HYMBA_OK;
}

}  // namespace hymba
