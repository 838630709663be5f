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

// Eight elements of a head as one (bf16) or two (fp32) 16-byte vectors.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const void *p) { r = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void zero() { r = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
    }
  }
  static __device__ __forceinline__ void store(void *p, const float (&x)[8]) {
    st_global_v4(p, pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                 pack_bf16x2(x[6], x[7]));
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  static __device__ __forceinline__ void store(void *p, const float (&x)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// How an element finds its pair's other element.
enum Partner {
  kNone,      // no rotation
  kInLane,    // pairs (2i, 2i+1): in the same lane
  kByShuffle, // halves dim/2 = 8 n apart: the same element of the lane n away
  kByShared   // other halves: through shared memory
};

// A warp takes one unit: a row of a sequence and a share of its heads.  Its lanes first
// compute the row's angles, one pair each (fp64 turns p * f / 2 pi, of which only the
// fraction goes to the fp32 sincospi), and keep the factors of their own eight elements in
// registers for all heads of the unit.  32 / lanes heads are in flight per load, four loads
// ahead of the arithmetic.
template <typename T, int PARTNER>
__global__ void __launch_bounds__(32 * kHeadWarps)
    qk_norm_rope_kernel(const __grid_constant__ HeadsParams p) {
  pdl_wait();
  pdl_trigger();
  __shared__ float2 s_trig[PARTNER == kNone ? 1 : kHeadWarps * kMaxPairs];
  __shared__ float s_stage[PARTNER == kByShared ? kHeadWarps * 256 : 1];
  const hymba_qk_norm_rope_args &a = p.a;
  const int warp = warp_id(), lane = lane_id();
  const long long unit = (long long)blockIdx.x * kHeadWarps + warp;
  if (unit >= p.units) return;
  const int part = int(unit % p.parts);
  const long long row_id = unit / p.parts;
  const int r = int(row_id % a.n_rows);
  const long long b = row_id / a.n_rows;
  const int lanes = p.lanes, li = lane & (lanes - 1), slot = lane / lanes, per = 32 / lanes;
  const int d = a.head_dim, e0 = 8 * li;
  const bool live = e0 < d;
  const int rot = a.rope.dim, half = rot >> 1;

  float cs[PARTNER == kNone ? 1 : 8], sn[PARTNER == kNone ? 1 : 8];
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
    // y_e = x_e c_e + x_partner s_e, with c = 1, s = 0 behind the rotated part
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = e0 + j;
      cs[j] = 1.f;
      sn[j] = 0.f;
      if (e < rot) {
        const bool second = PARTNER == kInLane ? (e & 1) : e >= half;
        const float2 t = trig[PARTNER == kInLane ? e >> 1 : second ? e - half : e];
        cs[j] = t.x;
        sn[j] = second ? t.y : -t.y;
      }
    }
  }

  const int heads = a.q.n_heads + a.k.n_heads;
  const int groups = (heads + per - 1) / per;
  const float inv_d = 1.0f / float(d);
  for (int g0 = part * p.chunk; g0 < groups; g0 += p.parts * p.chunk) {
    Vec8<T> raw[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int hh = (g0 + u) * per + slot;
      raw[u].zero();
      if (live && u < p.chunk && hh < heads) {
        const bool is_q = hh < a.q.n_heads;
        const long long at = b * (is_q ? a.q.in_batch : a.k.in_batch) + r * (is_q ? a.q.in_row : a.k.in_row) +
                             (is_q ? hh * a.q.in_head : (hh - a.q.n_heads) * a.k.in_head) + e0;
        raw[u].load(reinterpret_cast<const T *>(is_q ? a.q.in : a.k.in) + at);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (u >= p.chunk || g0 + u >= groups) break;  // the same for the whole warp
      const int hh = (g0 + u) * per + slot;
      const bool is_q = hh < a.q.n_heads;
      float x[8];
      raw[u].get(x);
      if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
        for (int m = lanes >> 1; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float inv = 1.0f / sqrtf(fmaf(ss, inv_d, a.eps));
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= inv;
        const float *weight = is_q ? a.q.weight : a.k.weight;
        if (weight && live && hh < heads) {
          const float4 w0 = __ldg(reinterpret_cast<const float4 *>(weight + e0));
          const float4 w1 = __ldg(reinterpret_cast<const float4 *>(weight + e0) + 1);
          const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] *= w[j];
        }
      }
      float y[8];
      if constexpr (PARTNER == kNone) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[j];
      } else if constexpr (PARTNER == kInLane) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = e0 + j < rot ? fmaf(x[j], cs[j], x[j ^ 1] * sn[j]) : x[j];
      } else if constexpr (PARTNER == kByShuffle) {
        const int away = half >> 3;
        const int from = e0 < half ? lane + away : e0 < rot ? lane - away : lane;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float o = __shfl_sync(0xffffffffu, x[j], from);
          y[j] = e0 + j < rot ? fmaf(x[j], cs[j], o * sn[j]) : x[j];
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
        const long long at = b * (is_q ? a.q.out_batch : a.k.out_batch) + r * (is_q ? a.q.out_row : a.k.out_row) +
                             (is_q ? hh * a.q.out_head : (hh - a.q.n_heads) * a.k.out_head) + e0;
        Vec8<T>::store(reinterpret_cast<T *>(is_q ? a.q.out : a.k.out) + at, y);
      }
    }
  }
}

template <typename T>
void heads_launch(const HeadsParams &p, int partner, unsigned grid, cudaStream_t s) {
  const dim3 g(grid), blk(32 * kHeadWarps);
  if (partner == kNone) launch_kernel(qk_norm_rope_kernel<T, kNone>, g, blk, 0, s, p);
  else if (partner == kInLane) launch_kernel(qk_norm_rope_kernel<T, kInLane>, g, blk, 0, s, p);
  else if (partner == kByShuffle) launch_kernel(qk_norm_rope_kernel<T, kByShuffle>, g, blk, 0, s, p);
  else launch_kernel(qk_norm_rope_kernel<T, kByShared>, g, blk, 0, s, p);
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
                      : a.rope.layout == HYMBA_ROPE_PAIRS ? kInLane
                      : half % 8 == 0 ? kByShuffle : kByShared;
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
