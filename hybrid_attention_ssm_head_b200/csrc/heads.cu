// Norm of every query and key head and its rotation to its row's position, in one pass
// (hymba_qk_norm_rope):
//   y = x / sqrt(mean(x^2) + eps) * w;   pair (a, b) -> m (a cos - b sin, a sin + b cos)
#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace hymba {

namespace {

constexpr int kHeadWarps = 4;
constexpr int kAhead = 4;       // loads in flight of a warp that takes several
constexpr int kMaxPairs = 128;  // head_dim <= 256
constexpr double kTwoPi = 6.283185307179586476925286766559;

struct HeadsParams {
  hymba_qk_norm_rope_args a;
  int lanes;       // lanes per head: a power of two, 2 N elements each
  int parts;       // units per row: the heads of a row are split over this many warps
  int chunk;       // loads (of 32 / lanes heads) a warp keeps in flight, at most kAhead
  unsigned units;  // batch * n_rows * parts
  double turns[kMaxPairs];  // f_i / (2 pi): turns per position
};

// N elements of a head: 8 or 16 bytes of bf16, 16 of fp32.
template <typename T, int N>
struct Vec;
template <>
struct Vec<__nv_bfloat16, 4> {
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
struct Vec<__nv_bfloat16, 8> {
  using R = uint4;
  static __device__ __forceinline__ void get(const R &r, float2 *x) {
    x[0] = make_float2(bf16_lo(r.x), bf16_hi(r.x));
    x[1] = make_float2(bf16_lo(r.y), bf16_hi(r.y));
    x[2] = make_float2(bf16_lo(r.z), bf16_hi(r.z));
    x[3] = make_float2(bf16_lo(r.w), bf16_hi(r.w));
  }
  static __device__ __forceinline__ R put(const float2 *x) {
    return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y), pack_bf16x2(x[2].x, x[2].y),
                      pack_bf16x2(x[3].x, x[3].y));
  }
};
template <>
struct Vec<float, 4> {
  using R = float4;
  static __device__ __forceinline__ void get(const R &r, float2 *x) {
    x[0] = make_float2(r.x, r.y);
    x[1] = make_float2(r.z, r.w);
  }
  static __device__ __forceinline__ R put(const float2 *x) { return make_float4(x[0].x, x[0].y, x[1].x, x[1].y); }
};

// Which 2 N elements of a head a lane holds, and where an element's pair is.
enum Partner {
  kNone,    // no rotation: elements 2 N l ..
  kPairs,   // pairs (2i, 2i+1): elements 2 N l .., N pairs
  kHalves,  // halves of the whole head: elements N l .. and d/2 + N l .., N pairs
  kShared   // halves of a part of the head: elements 2 N l .., the pairs through shared memory
};

// A warp takes one unit: a row of a sequence and a share of its heads.  Its lanes first
// compute the row's angles, one pair each (fp64 turns p * f / 2 pi, of which only the
// fraction goes to the fp32 sincospi), and keep the factors of their own pairs in registers
// for all heads of the unit.  32 / lanes heads are in flight per load, kAhead loads ahead of
// the arithmetic.
//
// Bound by the latency inside a warp: it lives for one row, and angles, loads, sums and turns follow
// one another.  8 x 4224 rows of 30 heads of 64, halves, under ncu: 18 warps an SM (96 registers a
// thread) with an instruction every 8.1 cycles each, of which 2.0 are fixed waits between dependent
// instructions, 1.6 loads, 1.5 shuffles and shared memory; instructions issue in 56 % of the cycles,
// DRAM moves 3.6 TB/s.  What helped was fewer of them in a row: with a head's halves in lanes
// of their own the rotation took eight shuffles per eight elements (109 us); a lane that holds
// both elements of its pairs needs none (62 us), and with sixteen elements a lane the sums' shuffles
// are a third (56 us, 4.6 TB/s).  Not kept: loads two or three ahead (59, 64 us), the first loads
// ahead of the angles (66 us with eight elements), registers cut for more warps (61 us).
template <typename T, int PARTNER, int N, int AHEAD>
__global__ void __launch_bounds__(32 * kHeadWarps)
    qk_norm_rope_kernel(const __grid_constant__ HeadsParams p) {
  pdl_wait();
  pdl_trigger();
  using V = Vec<T, N>;
  __shared__ float2 s_trig[PARTNER == kNone ? 1 : kHeadWarps * kMaxPairs];
  __shared__ float s_stage[PARTNER == kShared ? kHeadWarps * 64 * N : 1];
  const hymba_qk_norm_rope_args &a = p.a;
  const int warp = warp_id(), lane = lane_id();
  const unsigned unit = blockIdx.x * kHeadWarps + warp;
  if (unit >= p.units) return;
  const unsigned row_id = p.parts == 1 ? unit : unit / (unsigned)p.parts;
  const int part = int(unit - row_id * p.parts);
  const int b = int(row_id / (unsigned)a.n_rows), r = int(row_id - b * (unsigned)a.n_rows);
  const int lanes = p.lanes, li = lane & (lanes - 1), slot = lane / lanes, per = 32 / lanes;
  const int d = a.head_dim, rot = a.rope.dim, half = rot >> 1;
  const bool live = 2 * N * li < d;
  // the lane's elements: N from e0, N from e1
  const int e0 = PARTNER == kHalves ? N * li : 2 * N * li, e1 = PARTNER == kHalves ? half + N * li : e0 + N;

  const int nq = a.q.n_heads, heads = nq + a.k.n_heads;
  const int groups = (heads + per - 1) / per;
  const float inv_d = 1.0f / float(d);
  const T *qi = reinterpret_cast<const T *>(a.q.in) + b * a.q.in_batch + r * a.q.in_row;
  const T *ki = reinterpret_cast<const T *>(a.k.in) + b * a.k.in_batch + r * a.k.in_row;
  T *qo = reinterpret_cast<T *>(a.q.out) + b * a.q.out_batch + r * a.q.out_row;
  T *ko = reinterpret_cast<T *>(a.k.out) + b * a.k.out_batch + r * a.k.out_row;

  typename V::R ra[AHEAD], rb[AHEAD];
  auto request = [&](int g0) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int hh = (g0 + u) * per + slot;
      ra[u] = rb[u] = typename V::R{};
      if (live && u < p.chunk && hh < heads) {
        const T *src = hh < nq ? qi + hh * a.q.in_head : ki + (hh - nq) * a.k.in_head;
        ra[u] = *reinterpret_cast<const typename V::R *>(src + e0);
        rb[u] = *reinterpret_cast<const typename V::R *>(src + e1);
      }
    }
  };
  if constexpr (AHEAD == 1) request(part);

  // kPairs, kHalves: cos and sin of the lane's N pairs; kShared: of its elements'
  constexpr int NF = PARTNER == kNone ? 1 : PARTNER == kShared ? 2 * N : N;
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
      const int i = PARTNER == kPairs ? N * li + j : PARTNER == kHalves ? e0 + j : e0 + j < half ? e0 + j : e0 + j - half;
      const float2 t = i < half ? trig[i] : make_float2(1.f, 0.f);  // behind the rotated part
      cs[j] = t.x;
      sn[j] = PARTNER == kShared && e0 + j < half ? -t.y : t.y;
    }
  }

  for (int g0 = part * p.chunk; g0 < groups; g0 += p.parts * p.chunk) {
    if constexpr (AHEAD > 1) request(g0);
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (u >= p.chunk || g0 + u >= groups) break;  // the same for the whole warp
      const int hh = (g0 + u) * per + slot;
      // elements two by two: e0, e0 + 1 | .. | e1 + 2, e1 + 3
      float2 x[N];
      V::get(ra[u], x);
      V::get(rb[u], x + N / 2);
      if (a.norm) {
        float2 s2 = fmul2(x[0], x[0]);
#pragma unroll
        for (int j = 1; j < N; ++j) s2 = ffma2(x[j], x[j], s2);
        float ss = s2.x + s2.y;
        for (int m = lanes >> 1; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float inv = rsqrtf(fmaf(ss, inv_d, a.eps));
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = fmul2(x[j], make_float2(inv, inv));
        const float *weight = hh < nq ? a.q.weight : a.k.weight;
        if (weight && live) {
#pragma unroll
          for (int j = 0; j < N; j += 2) {
            const float4 w = __ldg(reinterpret_cast<const float4 *>(weight + (2 * j < N ? e0 + 2 * j : e1 + 2 * j - N)));
            x[j] = fmul2(x[j], make_float2(w.x, w.y));
            x[j + 1] = fmul2(x[j + 1], make_float2(w.z, w.w));
          }
        }
      }
      float2 y[N];
      if constexpr (PARTNER == kNone) {
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = x[j];
      } else if constexpr (PARTNER == kPairs) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          y[j] = make_float2(fmaf(x[j].x, cs[j], -x[j].y * sn[j]), fmaf(x[j].y, cs[j], x[j].x * sn[j]));
          if (e0 + 2 * j >= rot) y[j] = x[j];  // not rotated: as it is, whatever its pair holds
        }
      } else if constexpr (PARTNER == kHalves) {
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          const float2 c2 = make_float2(cs[2 * j], cs[2 * j + 1]), s2 = make_float2(sn[2 * j], sn[2 * j + 1]);
          const float2 n2 = make_float2(-s2.x, -s2.y);
          y[j] = ffma2(x[j], c2, fmul2(x[j + N / 2], n2));
          y[j + N / 2] = ffma2(x[j + N / 2], c2, fmul2(x[j], s2));
        }
      } else {
        // each lane's elements at 2 N lane: the warp's heads side by side
        float *st = s_stage + warp * 64 * N;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < N; ++j) *reinterpret_cast<float2 *>(&st[2 * N * lane + 2 * j]) = x[j];
        __syncwarp();
        auto turn = [&](float v, int j) {
          const int e = e0 + j, other = e < half ? e + half : e - half;
          return e < rot ? fmaf(v, cs[j], st[2 * N * (lane - li) + other] * sn[j]) : v;
        };
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = make_float2(turn(x[j].x, 2 * j), turn(x[j].y, 2 * j + 1));
      }
      if (live && hh < heads) {
        T *dst = hh < nq ? qo + hh * a.q.out_head : ko + (hh - nq) * a.k.out_head;
        *reinterpret_cast<typename V::R *>(dst + e0) = V::put(y);
        *reinterpret_cast<typename V::R *>(dst + e1) = V::put(y + N / 2);
      }
    }
  }
}

template <typename T, int N, int AHEAD>
void heads_launch_ahead(const HeadsParams &p, int partner, dim3 g, cudaStream_t s) {
  const dim3 blk(32 * kHeadWarps);
  if (partner == kNone) launch_kernel(qk_norm_rope_kernel<T, kNone, N, AHEAD>, g, blk, 0, s, p);
  else if (partner == kPairs) launch_kernel(qk_norm_rope_kernel<T, kPairs, N, AHEAD>, g, blk, 0, s, p);
  else if (partner == kHalves) launch_kernel(qk_norm_rope_kernel<T, kHalves, N, AHEAD>, g, blk, 0, s, p);
  else launch_kernel(qk_norm_rope_kernel<T, kShared, 4, AHEAD>, g, blk, 0, s, p);
}
// A warp whose share of a row is one load requests it ahead of the angles and holds no more:
// 40 x 2976 rows of 6 heads of 48 71 us, as with several loads 114 us; 3 tokens of 30 heads 2.6 and
// 2.9 us.  With two loads a warp the registers for both cost more (57 to 66 us at 30 heads).
template <typename T, int N>
void heads_launch(const HeadsParams &p, int partner, dim3 g, cudaStream_t s) {
  if (p.chunk == 1) heads_launch_ahead<T, N, 1>(p, partner, g, s);
  else heads_launch_ahead<T, N, kAhead>(p, partner, g, s);
}

}  // namespace

hymba_status qk_norm_rope(const hymba_qk_norm_rope_args &a, cudaStream_t s) {
  HeadsParams p;
  p.a = a;
  // A side without heads holds nothing that may be read: the slots of a row's last load behind its
  // last head pick the keys' weight.
  if (a.q.n_heads == 0) p.a.q = hymba_head_rows{};
  if (a.k.n_heads == 0) p.a.k = hymba_head_rows{};
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
  // Sixteen elements a lane where the type and the head's size allow 16-byte loads: fewer lanes
  // share a sum and fewer loads go out (8 x 4224 rows of 30 heads 57 us, with eight 62 us).  A
  // part's halves go through shared memory, eight elements a lane.
  const int n = a.dtype == HYMBA_BF16 && partner != kShared && a.head_dim % 16 == 0 ? 8 : 4;
  p.lanes = 1;
  while (p.lanes * 2 * n < a.head_dim) p.lanes *= 2;
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
  if (n == 8) heads_launch<__nv_bfloat16, 8>(p, partner, grid, s);
  else if (a.dtype == HYMBA_BF16) heads_launch<__nv_bfloat16, 4>(p, partner, grid, s);
  else heads_launch<float, 4>(p, partner, grid, s);
  note_launch(1);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("head norm/rotation launch failed: %s", cudaGetErrorString(e));
    return HYMBA_ERR_CUDA;
  }
  return HYMBA_OK;
}

}  // namespace hymba
