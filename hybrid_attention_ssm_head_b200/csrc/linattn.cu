// Linear attention with a decay for each head, on the CUDA cores (hymba_linear_attention_*):
//   S_t = exp(g_t) S_{t-1} + s_t v_t k_t^T,   o_t = (scale S_t q_t + skip v_t) gate_t
// The state S [dv, dk] is fp32 throughout.
#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "linattn.cuh"

namespace hymba {

namespace {

// ---------------------------------------------------------------------------
// one token per sequence
// ---------------------------------------------------------------------------
constexpr int kStepWarps = 4;
constexpr int kStepAhead = 4;  // 16-byte state loads in flight per lane

template <typename T>
__device__ __forceinline__ float4 load4(const T *p) {
  if constexpr (sizeof(T) == 2) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
  } else {
    return *reinterpret_cast<const float4 *>(p);
  }
}

// Bound by the state's bytes, read and written once.  A CTA takes `rows` of the dv state
// rows of one (sequence, head); LANES lanes hold one row, four columns each, so a warp's loads
// and stores are whole contiguous rows.  A lane's rows are requested together.  Their dot
// products with q are summed over the lanes by halves: each exchange hands half of the rows'
// sums to the other half of the lanes, so four sums over LANES >= 4 lanes take 3 +
// log2(LANES / 4) shuffles and each lands in a lane of its own, which finishes that row.
// Many small CTAs cover each other's ends: with 8 warps and 8 rows a lane, 4 CTAs to an SM,
// 128 x 25 heads of 128 x 64 states took 50 us, with 4 warps and 4 rows, 12 to an SM, 41 us, and
// with the state marked as read and written once (it is back only when every other layer's
// has passed through the cache) 39 us, 5.4 TB/s.  Twelve CTAs leave 40 registers a thread, for which
// 52 to 84 bytes are spilled.
template <typename T, int LANES>
__global__ void __launch_bounds__(32 * kStepWarps, 12)
    linear_step_kernel(const __grid_constant__ hymba_linear_attention a, int rows) {
  pdl_wait();
  pdl_trigger();
  constexpr int PER = 32 / LANES;           // state rows per warp and load
  constexpr int STRIDE = kStepWarps * PER;  // rows of the CTA per load
  constexpr int KEPT = LANES >= kStepAhead ? 1 : kStepAhead / LANES;  // rows' sums a lane ends up with
  const int h = blockIdx.y, b = blockIdx.z;
  const int hk = h / (a.n_heads / a.n_qk_heads);
  const int lane = lane_id(), li = lane % LANES, c0 = 4 * li;
  const bool live = c0 < a.dk;
  const int p_end = min(a.dv, (int)(blockIdx.x + 1) * rows);
  const long long dense = (long long)a.dv * a.dk;
  const float *sin = a.state_in ? a.state_in + b * a.state_in_batch + h * dense : nullptr;
  float *sout = a.state_out + ((long long)b * a.n_heads + h) * dense;
  const bool idle = a.lengths && a.lengths[b] <= 0;
  if (idle && sin == sout) return;
  const float decay = a.log_decay ? linear_decay(a.log_decay[b * a.decay_batch + h * a.decay_head]) : 1.f;
  const float s = a.in_scale ? a.in_scale[b * a.scale_batch + h * a.scale_head] : 1.f;
  const T *vp = reinterpret_cast<const T *>(a.v) + b * a.v_batch + h * a.v_head;
  T *op = reinterpret_cast<T *>(a.o) + b * a.o_batch + h * a.o_head;
  const T *zp = reinterpret_cast<const T *>(a.gate) + (a.gate ? b * a.gate_batch + h * a.gate_head : 0);
  float4 k = make_float4(0.f, 0.f, 0.f, 0.f), q = k;
  if (live) {
    k = load4(reinterpret_cast<const T *>(a.k) + b * a.k_batch + hk * a.k_head + c0);
    q = load4(reinterpret_cast<const T *>(a.q) + b * a.q_batch + hk * a.q_head + c0);
  }
  // which of its rows' sums a lane ends up with, from its number's high bits down; of
  // the lanes that share one the first finishes it
  int u0 = 0;
#pragma unroll
  for (int m = LANES / 2, n = kStepAhead / 2; m > 0 && n > 0; m >>= 1, n >>= 1)
    if (li & m) u0 += n;
  const bool finishes = LANES <= kStepAhead || li % (LANES > kStepAhead ? LANES / kStepAhead : 1) == 0;
  for (int base = blockIdx.x * rows; base < p_end; base += kStepAhead * STRIDE) {
    const int p0 = base + warp_id() * PER + lane / LANES;
    float4 st[kStepAhead];
    float v[kStepAhead], dot[kStepAhead], skip[KEPT], gate[KEPT], vr[KEPT];
#pragma unroll
    for (int u = 0; u < kStepAhead; ++u) {
      const int p = p0 + u * STRIDE;
      st[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      v[u] = 0.f;
      if (p < p_end) {
        if (live && sin) st[u] = __ldcs(reinterpret_cast<const float4 *>(sin + (long long)p * a.dk + c0));
        v[u] = Store<T>::to_f(vp[p]);
      }
    }
#pragma unroll
    for (int i = 0; i < KEPT; ++i) {
      const int p = p0 + (u0 + i) * STRIDE;
      const bool in = finishes && p < p_end;
      vr[i] = in ? Store<T>::to_f(vp[p]) : 0.f;
      skip[i] = in && a.skip ? a.skip[(long long)h * a.dv + p] : 0.f;
      gate[i] = in && a.gate ? Store<T>::to_f(zp[p]) : 1.f;
    }
#pragma unroll
    for (int u = 0; u < kStepAhead; ++u) {
      const int p = p0 + u * STRIDE;
      const float x = s * v[u];
      if (!idle) {
        st[u].x = fmaf(decay, st[u].x, x * k.x);
        st[u].y = fmaf(decay, st[u].y, x * k.y);
        st[u].z = fmaf(decay, st[u].z, x * k.z);
        st[u].w = fmaf(decay, st[u].w, x * k.w);
      }
      dot[u] = fmaf(st[u].x, q.x, st[u].y * q.y) + fmaf(st[u].z, q.z, st[u].w * q.w);
      if (live && p < p_end) __stcs(reinterpret_cast<float4 *>(sout + (long long)p * a.dk + c0), st[u]);
    }
    int n = kStepAhead / 2;
#pragma unroll
    for (int m = LANES / 2; m > 0; m >>= 1) {
      if (n > 0) {
        const bool upper = li & m;
#pragma unroll
        for (int i = 0; i < kStepAhead / 2; ++i)
          if (i < n) {
            const float give = upper ? dot[i] : dot[i + n];
            dot[i] = (upper ? dot[i + n] : dot[i]) + __shfl_xor_sync(0xffffffffu, give, m);
          }
        n >>= 1;
      } else {
        dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], m);
      }
    }
#pragma unroll
    for (int i = 0; i < KEPT; ++i) {
      const int p = p0 + (u0 + i) * STRIDE;
      if (finishes && p < p_end && !idle)
        op[p] = Store<T>::from_f(fmaf(skip[i], vr[i], a.scale * dot[i]) * gate[i]);
    }
  }
}

// ---------------------------------------------------------------------------
// row by row
// ---------------------------------------------------------------------------
constexpr int kScanRows = 16;   // rows staged at a time
constexpr int kFix = 8;         // rows between corrections of the decays
constexpr int kScanState = 64;  // state rows per CTA (two per thread group)

// NC columns of two adjacent state rows per thread, CL threads per row pair: the state stays
// in registers as fp32 pairs.  q, k, v, the gate and the decays of kScanRows rows are staged
// in shared memory as fp32, the next rows' waiting in registers meanwhile.
//
// Bound by the latency of one row after another.  Neighbouring threads take neighbouring pieces
// of four columns, so that a warp's reads of k and q meet no bank twice.  5 heads of 4000 fp32
// rows with dk 128 / 8 heads of 1031 with dk 64 / 800 heads of 15 bf16 rows with dk 128:
//   NC columns of a thread side by side                        398 / 58 / 130 us
//   pieces in turn                                             148 / 55 / 44 us
//   next rows' loads and decays ahead; 16 columns for dk <= 64   137 / 46 / 50 us
// (16 columns for dk 128 as well: 165 us before the last step.)  24 columns up to dk 96: 32 heads
// of 7006 rows with dk 80 1077 us, with 32 columns 1323 us.
//
// Decays near one: a fp32 decay is off by up to 2^-25, the same way at every row of a head
// with one fixed decay, so their product drifts from exp(sum g) by 2^-25 times the rows.
// The staged decays are therefore corrected every kFix rows: exp(sum g) over the product used
// so far is carried in fp64, and the next group's first decay takes it up.  Only decays in fp32's
// normal range take part: the ratio of a smaller one is up to 1.4 or 0.5, and would scale the rows
// added since.  Behind such a decay nothing of the state before it is left that a ratio could
// put right, so the ratio carried so far ends there too.
template <typename T, int NC, int CL>
__global__ void __launch_bounds__(kScanState / 2 * CL)
    linear_scan_kernel(const __grid_constant__ hymba_linear_attention a, const __grid_constant__ LinearSegments g) {
  pdl_wait();
  pdl_trigger();
  constexpr int THR = kScanState / 2 * CL, DK = NC * CL;
  static_assert(THR >= 32, "one warp stages the decays");
  __shared__ __align__(16) float s_q[kScanRows][DK], s_k[kScanRows][DK];
  __shared__ __align__(16) float s_v[kScanRows][kScanState], s_z[kScanRows][kScanState];
  __shared__ float2 s_dx[kScanRows];  // (decay, input scale)
  const int blocks = (a.dv + kScanState - 1) / kScanState;
  const int tid = threadIdx.x, h = blockIdx.y, b = blockIdx.z, seg = blockIdx.x / blocks;
  const int hk = h / (a.n_heads / a.n_qk_heads);
  const int pb = (blockIdx.x % blocks) * kScanState;   // the CTA's first state row
  const int pn = min(kScanState, a.dv - pb);           // and how many (even)
  const int pr = 2 * (tid / CL), c0 = 4 * (tid % CL);  // this thread's row pair and columns c0 + CL c ..
  const bool rows_live = pr < pn;
  const bool outputs = g.pass == 1;                    // else the segment's state alone
  const int L = min(linear_length(a, b), (seg + 1) * g.rows);
  const long long dense = (long long)a.dv * a.dk, heads = (long long)a.batch * a.n_heads, bh = (long long)b * a.n_heads + h;
  const T *qp = reinterpret_cast<const T *>(a.q) + b * a.q_batch + hk * a.q_head;
  const T *kp = reinterpret_cast<const T *>(a.k) + b * a.k_batch + hk * a.k_head;
  const T *vp = reinterpret_cast<const T *>(a.v) + b * a.v_batch + h * a.v_head + pb;
  const T *zp = reinterpret_cast<const T *>(a.gate) + (a.gate ? b * a.gate_batch + h * a.gate_head + pb : 0);
  T *op = reinterpret_cast<T *>(a.o) + b * a.o_batch + h * a.o_head + pb;
  const float *gp = a.log_decay ? a.log_decay + b * a.decay_batch + h * a.decay_head : nullptr;
  const float *sp = a.in_scale ? a.in_scale + b * a.scale_batch + h * a.scale_head : nullptr;

  float2 S[2][NC / 2];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int c = 0; c < NC / 2; ++c) S[r][c] = make_float2(0.f, 0.f);
  // The state the segment starts from: the call's, or (outputs) the one after the segments
  // before it; a segment's own state starts from zero, the first one's from the call's.
  const float *from = a.state_in ? a.state_in + b * a.state_in_batch + h * dense : nullptr;
  if (outputs && g.n > 1) from = a.state_in ? g.state + ((g.n - 1) * heads + bh) * dense : nullptr;
  if (seg > 0) from = outputs ? g.state + ((seg - 1) * heads + bh) * dense : nullptr;
  if (from && rows_live)
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int c = 0; c < NC; c += 4)
        if (c0 + CL * c < a.dk) {
          const float4 x = *reinterpret_cast<const float4 *>(from + (long long)(pb + pr + r) * a.dk + c0 + CL * c);
          S[r][c / 2] = make_float2(x.x, x.y);
          S[r][c / 2 + 1] = make_float2(x.z, x.w);
        }
  auto store_state = [&](float *dst) {
    if (!rows_live) return;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int c = 0; c < NC; c += 4)
        if (c0 + CL * c < a.dk)
          *reinterpret_cast<float4 *>(dst + (long long)(pb + pr + r) * a.dk + c0 + CL * c) =
              make_float4(S[r][c / 2].x, S[r][c / 2].y, S[r][c / 2 + 1].x, S[r][c / 2 + 1].y);
  };
  if (!outputs && seg == 0 && a.state_in)  // a copy for the outputs' pass, which may write in place
    store_state(g.state + ((g.n - 1) * heads + bh) * dense);
  float2 skip = make_float2(0.f, 0.f);
  if (a.skip && rows_live) skip = *reinterpret_cast<const float2 *>(a.skip + (long long)h * a.dv + pb + pr);

  double carry = 1.0;  // exp(sum g) over the product of the decays used so far
  double total = 0.0;  // log2 of this lane's rows' decays
  // The next rows wait in registers while these are computed.
  constexpr int QN = kScanRows * (DK / 4) / THR, VN = kScanRows * (kScanState / 4) / THR;
  float4 rq[QN], rk[QN], rv[VN], rz[VN];
  float2 dx_next = make_float2(0.f, 0.f);
  auto fetch = [&](int t0) {
    const int nt = min(kScanRows, L - t0), t = tid;  // the first warp: one row's decay a lane
    float gt = 0.f, st = 1.f;
    if (t < nt) {
      if (gp) gt = gp[(t0 + t) * a.decay_row];
      if (sp) st = sp[(t0 + t) * a.scale_row];
    }
#pragma unroll
    for (int u = 0; u < QN; ++u) {
      const int i = tid + u * THR, r = i / (DK / 4), c = 4 * (i % (DK / 4));
      rq[u] = rk[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nt && c < a.dk) {
        if (outputs) rq[u] = load4(qp + (t0 + r) * a.q_row + c);
        rk[u] = load4(kp + (t0 + r) * a.k_row + c);
      }
    }
#pragma unroll
    for (int u = 0; u < VN; ++u) {
      const int i = tid + u * THR, r = i / (kScanState / 4), c = 4 * (i % (kScanState / 4));
      rv[u] = rz[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < nt && c < pn) {
        rv[u] = load4(vp + (t0 + r) * a.v_row + c);
        if (outputs && a.gate) rz[u] = load4(zp + (t0 + r) * a.gate_row + c);
      }
    }
    if (tid < 32) {
      double want = 1.0;
      if (t < nt && gp) {
        gt = linear_log_decay(gt);
        want = exp((double)gt);
        total += (double)gt * 1.4426950408889634074;
      }
      float used = (float)want;
      // what the rounding of the other rows of this group of kFix leaves over; then each
      // group's first decay in turn takes up what was left over before it
      double left = t % kFix && used >= FLT_MIN ? want / (double)used : 1.0;
#pragma unroll
      for (int m = kFix >> 1; m > 0; m >>= 1) left *= __shfl_xor_sync(0xffffffffu, left, m);
#pragma unroll
      for (int f = 0; f < kScanRows; f += kFix) {
        double next = carry;
        if (t == f) {
          const double exact = want * carry;
          used = (float)exact;
          next = (used >= FLT_MIN ? exact / (double)used : 1.0) * left;
        }
        carry = __shfl_sync(0xffffffffu, next, f);
      }
      dx_next = make_float2(used, st);
    }
  };
  if (seg * g.rows < L) fetch(seg * g.rows);
  for (int t0 = seg * g.rows; t0 < L; t0 += kScanRows) {
    const int nt = min(kScanRows, L - t0);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < QN; ++u) {
      const int i = tid + u * THR, r = i / (DK / 4), c = 4 * (i % (DK / 4));
      *reinterpret_cast<float4 *>(&s_q[r][c]) = rq[u];
      *reinterpret_cast<float4 *>(&s_k[r][c]) = rk[u];
    }
#pragma unroll
    for (int u = 0; u < VN; ++u) {
      const int i = tid + u * THR, r = i / (kScanState / 4), c = 4 * (i % (kScanState / 4));
      *reinterpret_cast<float4 *>(&s_v[r][c]) = rv[u];
      *reinterpret_cast<float4 *>(&s_z[r][c]) = rz[u];
    }
    if (tid < kScanRows) s_dx[tid] = dx_next;
    __syncthreads();
    if (t0 + kScanRows < L) fetch(t0 + kScanRows);
    for (int t = 0; t < nt; ++t) {
      const float2 dx = s_dx[t];
      const float2 v = *reinterpret_cast<const float2 *>(&s_v[t][pr]);
      const float2 d2 = make_float2(dx.x, dx.x);
      const float2 x0 = make_float2(dx.y * v.x, dx.y * v.x), x1 = make_float2(dx.y * v.y, dx.y * v.y);
      float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
#pragma unroll
      for (int c = 0; c < NC; c += 4) {
        const float4 k = *reinterpret_cast<const float4 *>(&s_k[t][c0 + CL * c]);
        const float4 q = *reinterpret_cast<const float4 *>(&s_q[t][c0 + CL * c]);
        const float2 ka = make_float2(k.x, k.y), kb = make_float2(k.z, k.w);
        const float2 qa = make_float2(q.x, q.y), qb = make_float2(q.z, q.w);
        S[0][c / 2] = ffma2(d2, S[0][c / 2], fmul2(x0, ka));
        S[0][c / 2 + 1] = ffma2(d2, S[0][c / 2 + 1], fmul2(x0, kb));
        S[1][c / 2] = ffma2(d2, S[1][c / 2], fmul2(x1, ka));
        S[1][c / 2 + 1] = ffma2(d2, S[1][c / 2 + 1], fmul2(x1, kb));
        if (outputs) {
          acc0 = ffma2(S[0][c / 2], qa, acc0);
          acc1 = ffma2(S[1][c / 2], qa, acc1);
          acc0 = ffma2(S[0][c / 2 + 1], qb, acc0);
          acc1 = ffma2(S[1][c / 2 + 1], qb, acc1);
        }
      }
      if (!outputs) continue;
      float y0 = acc0.x + acc0.y, y1 = acc1.x + acc1.y;
#pragma unroll
      for (int m = CL >> 1; m > 0; m >>= 1) {
        y0 += __shfl_xor_sync(0xffffffffu, y0, m);
        y1 += __shfl_xor_sync(0xffffffffu, y1, m);
      }
      if (tid % CL == 0 && rows_live) {
        y0 = fmaf(skip.x, v.x, a.scale * y0);
        y1 = fmaf(skip.y, v.y, a.scale * y1);
        if (a.gate) {
          const float2 z = *reinterpret_cast<const float2 *>(&s_z[t][pr]);
          y0 *= z.x;
          y1 *= z.y;
        }
        T *o = op + (t0 + t) * a.o_row + pr;
        if constexpr (sizeof(T) == 2) *reinterpret_cast<uint32_t *>(o) = pack_bf16x2(y0, y1);
        else *reinterpret_cast<float2 *>(o) = make_float2(y0, y1);
      }
    }
  }
  if (!outputs) {
    if (tid < 32) {
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) total += __shfl_xor_sync(0xffffffffu, total, m);
      if (tid == 0 && pb == 0) g.decay[seg * heads + bh] = total;
    }
    store_state(g.state + (seg * heads + bh) * dense);
  } else if (a.state_out && seg == g.n - 1) {
    store_state(a.state_out + bh * dense);
  }
}

// The segments' own states to the states after them, in place: P_j = decay_j P_{j-1} + own_j.
// One thread takes four elements through all segments, eight of them requested at a time.
// Read and written once: with the sum taken where it is used, each segment over those before
// it, 5 heads of 4000 fp32 rows of 128 x 128 states in 84 segments took 716 us, so 398 us (124 us with the later steps).
__global__ void __launch_bounds__(256) linear_prefix_kernel(const __grid_constant__ LinearSegments g, long long size, long long heads) {
  pdl_wait();
  pdl_trigger();
  const long long bh = blockIdx.y + (long long)blockIdx.z * gridDim.y;
  const long long e = 4 * (blockIdx.x * 256ll + threadIdx.x);
  if (e >= size || bh >= heads) return;
  const long long step = heads * size;
  float *p = g.state + bh * size + e;
  const double *d = g.decay + bh;
  float4 S = *reinterpret_cast<const float4 *>(p);
  for (int j = 1; j < g.n - 1; j += 8) {
    float4 x[8];
    float w[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (j + u < g.n - 1) {
        x[u] = *reinterpret_cast<const float4 *>(p + (j + u) * step);
        w[u] = exp2f((float)d[(j + u) * heads]);
      }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (j + u < g.n - 1) {
        S = make_float4(fmaf(w[u], S.x, x[u].x), fmaf(w[u], S.y, x[u].y), fmaf(w[u], S.z, x[u].z), fmaf(w[u], S.w, x[u].w));
        *reinterpret_cast<float4 *>(p + (j + u) * step) = S;
      }
  }
}

hymba_status launched(const char *what) {
  note_launch(1);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("%s launch failed: %s", what, cudaGetErrorString(e));
    return HYMBA_ERR_CUDA;
  }
  return HYMBA_OK;
}

template <typename T>
void scan_launch(const hymba_linear_attention &a, LinearSegments g, cudaStream_t s) {
  constexpr int one = kScanState / 2;
  for (g.pass = g.n > 1 ? 0 : 1; g.pass < 2; ++g.pass) {
    if (g.pass == 1) linear_prefix(a, g, s);
    const dim3 grid((a.dv + kScanState - 1) / kScanState * (g.pass ? g.n : g.n - 1), a.n_heads, a.batch);
    if (a.dk <= 16) launch_kernel(linear_scan_kernel<T, 16, 1>, grid, dim3(one), 0, s, a, g);
    else if (a.dk <= 32) launch_kernel(linear_scan_kernel<T, 16, 2>, grid, dim3(2 * one), 0, s, a, g);
    else if (a.dk <= 64) launch_kernel(linear_scan_kernel<T, 16, 4>, grid, dim3(4 * one), 0, s, a, g);
    else if (a.dk <= 96) launch_kernel(linear_scan_kernel<T, 24, 4>, grid, dim3(4 * one), 0, s, a, g);
    else launch_kernel(linear_scan_kernel<T, 32, 4>, grid, dim3(4 * one), 0, s, a, g);
    note_launch(1);
  }
}

// Few heads of many rows: segments of at least 32 rows, about three CTAs for each SM, as many as
// run beside each other.  Whole / so / with eight for each SM: 2 x 4 heads of 1031 fp32 rows 282 /
// 46 / 46 us, 50 heads of 2000 rows with dk 64 588 / 361 / 398 us, 200 heads 826 / 826 / 1122 us.
LinearSegments scan_segments(const hymba_linear_attention &a) {
  LinearSegments g{};
  const long long ctas = (long long)a.batch * a.n_heads * ((a.dv + kScanState - 1) / kScanState);
  const long long want = std::max<long long>(1, std::min<long long>(3 * 148 / std::max<long long>(1, ctas), a.n_rows / 32));
  g.rows = (int)(((a.n_rows + want - 1) / want + kScanRows - 1) / kScanRows * kScanRows);
  g.n = (a.n_rows + g.rows - 1) / g.rows;
  return g;
}

// Below this many rows a bf16 sequence is taken row by row: a chunk costs its 128 rows however
// many count.  Row by row and in a chunk, dk 64: 25 heads 9.8 and 12.1 us at 24 rows, 12.0 and
// 12.2 at 32, 16.9 and 12.1 at 48; 200 heads 17.5 and 23.9 us at 32, 24.2 and 23.8 at 48; dk 128:
// 25 heads 16.5 and 18.3 us at 32, 800 heads 90 and 104 us at 32, 128 and 105 at 48; dk 16, 16
// heads: 7.5 and 7.7 us at 16, 10.7 and 7.7 at 24.
int few_rows(const hymba_linear_attention &a) { return a.dk > 32 ? 32 : 16; }
bool on_tensor_cores(const hymba_linear_attention &a) { return a.dtype == HYMBA_BF16 && a.n_rows >= few_rows(a); }
LinearSegments segments_of(const hymba_linear_attention &a) {
  return on_tensor_cores(a) ? linear_attention_tc_segments(a) : scan_segments(a);
}
// The workspace of a split: states, then the segments' decays or the chain's tickets.
size_t segment_state_bytes(const hymba_linear_attention &a, const LinearSegments &g) {
  return (size_t)(g.chain ? 1 : g.n) * a.batch * a.n_heads * a.dv * a.dk * 4;
}
size_t segment_rest_bytes(const hymba_linear_attention &a, const LinearSegments &g) {
  return g.chain ? linear_attention_tc_tickets(a) * 4 : (size_t)g.n * a.batch * a.n_heads * 8;
}

}  // namespace

void linear_prefix(const hymba_linear_attention &a, const LinearSegments &g, cudaStream_t s) {
  if (g.n < 3 || g.chain) return;
  const long long size = (long long)a.dv * a.dk;
  launch_kernel(linear_prefix_kernel, dim3((unsigned)((size / 4 + 255) / 256), a.n_heads, a.batch), dim3(256), 0, s, g, size,
                (long long)a.batch * a.n_heads);
  note_launch(1);
}

hymba_status linear_attention_step(const hymba_linear_attention &a, cudaStream_t s) {
  int lanes = 2;
  while (lanes * 4 < a.dk) lanes *= 2;
  // One CTA for all state rows of a (sequence, head) keeps four loads in flight per lane; with
  // fewer (sequence, head) pairs than two CTAs for each SM the rows are split, down to one
  // load per lane.
  const int once = kStepWarps * (32 / lanes);
  const int most = (a.dv + once - 1) / once;
  const long long pairs = (long long)a.batch * a.n_heads;
  const long long want = (2 * 148 + pairs - 1) / pairs;
  const int parts = int(want < most ? want : most);
  const int rows = (most + parts - 1) / parts * once;
  const dim3 grid((a.dv + rows - 1) / rows, a.n_heads, a.batch), block(32 * kStepWarps);
  auto launch = [&](auto *bf16, auto *f32) {
    if (a.dtype == HYMBA_BF16) launch_kernel(bf16, grid, block, 0, s, a, rows);
    else launch_kernel(f32, grid, block, 0, s, a, rows);
  };
  if (lanes == 2) launch(linear_step_kernel<__nv_bfloat16, 2>, linear_step_kernel<float, 2>);
  else if (lanes == 4) launch(linear_step_kernel<__nv_bfloat16, 4>, linear_step_kernel<float, 4>);
  else if (lanes == 8) launch(linear_step_kernel<__nv_bfloat16, 8>, linear_step_kernel<float, 8>);
  else if (lanes == 16) launch(linear_step_kernel<__nv_bfloat16, 16>, linear_step_kernel<float, 16>);
  else launch(linear_step_kernel<__nv_bfloat16, 32>, linear_step_kernel<float, 32>);
  return launched("linear attention step");
}

size_t linear_attention_workspace_bytes(const hymba_linear_attention &a) {
  const LinearSegments g = segments_of(a);
  return g.n > 1 ? (segment_state_bytes(a, g) + segment_rest_bytes(a, g) + 7) / 8 * 8 : 0;
}

hymba_status linear_attention(const hymba_linear_attention &a, void *workspace, cudaStream_t s, int whole_batch) {
  hymba_linear_attention whole = a;
  if (whole_batch > 0) whole.batch = whole_batch;
  LinearSegments g = segments_of(whole);
  if (g.n > 1) {
    g.state = reinterpret_cast<float *>(workspace);
    char *rest = reinterpret_cast<char *>(workspace) + segment_state_bytes(whole, g);
    g.decay = reinterpret_cast<double *>(rest);
    g.ticket = reinterpret_cast<unsigned *>(rest);
    if (g.chain && cudaMemsetAsync(rest, 0, segment_rest_bytes(a, g), s) != cudaSuccess) {
      set_error("cudaMemsetAsync(segment tickets): %s", cudaGetErrorString(cudaGetLastError()));
      return HYMBA_ERR_CUDA;
    }
  }
  if (on_tensor_cores(a)) return linear_attention_tc(a, g, s);
  if (a.dtype == HYMBA_BF16) scan_launch<__nv_bfloat16>(a, g, s);
  else scan_launch<float>(a, g, s);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("linear attention launch failed: %s", cudaGetErrorString(e));
    return HYMBA_ERR_CUDA;
  }
  return HYMBA_OK;
}

}  // namespace hymba
