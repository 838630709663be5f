// Linear attention with a decay for each head over whole sequences, bf16 storage, on the
// tensor cores (tcgen05 + TMA): the recurrence of linattn.cu in chunks of 128 rows.  With
// G_i the sum of the log decays of a chunk's rows 0..i, and S the state before the chunk,
//   o_i  = scale (sum_{j <= i} P_ij v_j + exp(G_i) S q_i)    P_ij = exp(G_i - G_j) s_j (q_i . k_j)
//   S'   = exp(G_end) S + sum_j exp(G_end - G_j) s_j v_j k_j^T
// so a chunk is four products: Q K^T, P V, Q S^T and V^T K' (K' = K with weighted rows).
//
// Precision.  q, k, v enter the products as they are stored.  P is rounded once to bf16, as
// the probabilities of the softmax attention are: with the output's own rounding that is the
// accuracy of bf16 storage.  The state is kept in fp32 registers.  As the operand of Q S^T it
// is split in two bf16 parts (16 bits), more than the bf16 output holds; the weighted keys,
// whose errors would stay in the state, in three (24 bits, all of an fp32 product): with two
// parts the state of 8320 rows was 2.5e-6 off in the 2-norm.  A chunk's contribution is
// summed in tensor memory from zero and added to the state in fp32 by the CUDA cores.
#include "linattn.cuh"
#include "tmap.h"

namespace hymba {

HYMBA_DEVICE_ERROR_WORD(g_err_lin);

namespace {

constexpr int C = 128;         // rows per chunk
constexpr int kThreads = 512;  // TMA, MMA and decay warps (+ one idle), scores, state, output
constexpr int kRegCtrl = 56, kRegScores = 144, kRegState = 184, kRegOut = 128;
static_assert(kRegCtrl + kRegScores + kRegState + kRegOut == 4 * 128, "the warpgroups share 512 x 128 registers");
constexpr int kAtom = C * 128;  // bytes of 128 rows x 64 bf16 columns, 128-byte swizzle

struct Decays {  // of one chunk's rows, log2 units
  float hi[C], lo[C];  // G = hi + lo, hi a multiple of 1/8: differences of hi are exact
  float s[C];          // input scale
  float c[C];          // s exp(G_end of the row's block of 32 - G)
  float w[C];          // s exp(G_end of the chunk - G)
  float e[C];          // exp(G)
};

// NK, NV: 64-column atoms of dk and of the CTA's dv block.  For dk <= 64 two stages of
// (Q, K, V) tiles fit shared memory, and a tile that the gate is loaded into and the output
// is stored from.  Wider keys take one stage, stage the output over V and read the gate from
// global memory.
template <int NK, int NV>
struct Layout {
  static constexpr int STAGES = NK == 1 ? 2 : 1;
  static constexpr bool TILE = NK == 1;
  static constexpr int Q = 0, K = NK * kAtom, V = 2 * NK * kAtom, STAGE = (2 * NK + NV) * kAtom;
  static constexpr int MID = STAGES * STAGE;            // middle parts of the weighted keys
  static constexpr int SB = MID + NK * kAtom;           // state operand: hi, then lo
  static constexpr int SB_PART = NK * NV * (kAtom / 2); // 64 NV rows of 128 bytes per dk atom
  static constexpr int Z = SB + 2 * SB_PART;            // gate and output tile
  // the state product reads 128 state rows whatever dv is: for NV = 1 up to one atom behind V
  static constexpr int DEC = Z + (TILE ? NV * kAtom : 0);
  static constexpr int SKIP = DEC + 2 * (int)sizeof(Decays);
  static constexpr int BAR = SKIP + NV * 64 * 4;
  static constexpr int TOTAL = BAR + 32 * 8 + 1024;  // + alignment of the base
};

// Two fp32 values cut to their high 16 bits, as a bf16 pair: what is cut off is exact in fp32,
// so three such parts hold all 24 bits of a value.
__device__ __forceinline__ uint32_t high_pair(float2 x) {
  return __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
}

// A bounded wait as in common.cuh, in few instructions: the roles' loops have to stay in the
// instruction cache together (see the kernel).  A CTA that starts after another has given up
// does nothing.
__device__ __forceinline__ bool one_wait(uint64_t *bar, uint32_t parity, unsigned limit) {
  const unsigned t0 = (unsigned)clock();
  while (!mbar_try_wait(bar, parity))
    if ((unsigned)clock() - t0 > limit) {
      atomicOr(&g_err_lin, kErrTimeout);
      return false;
    }
  return true;
}
// ... by a whole warp: all of its lanes go on, or none.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, unsigned limit) {
  return __all_sync(0xffffffffu, one_wait(bar, parity, limit));
}

struct Params {
  hymba_linear_attention a;
  int blocks;      // dv blocks of 64 * NV columns
  unsigned wlim;   // bounded waits: SM clock cycles
};

template <int NK, int NV>
__global__ void __launch_bounds__(kThreads, 1)
    linear_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmZ,
                        const __grid_constant__ CUtensorMap tmO,
                        const __grid_constant__ Params prm) {
  pdl_wait();
  pdl_trigger();
  using Lay = Layout<NK, NV>;
  constexpr int ST = Lay::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::BAR);
  uint64_t *full = bars + 0, *empty = bars + 2;            // [ST] Q, K, V stages
  uint64_t *dec_full = bars + 4, *dec_empty = bars + 6;    // [2] decays
  uint64_t *z_full = bars + 8, *z_empty = bars + 9;        // gate tile
  uint64_t *s_full = bars + 10, *p_full = bars + 11;       // scores ready / P written over them
  uint64_t *o_full = bars + 12, *o_empty = bars + 13;      // outputs ready / read
  uint64_t *k_full = bars + 14, *c_full = bars + 15;       // weighted keys / chunk's state ready
  uint64_t *sb_full = bars + 16, *qs_done = bars + 17;     // state operand ready / read
  uint64_t *o_staged = bars + 18;                          // output rows staged
  uint64_t *drain = bars + 19;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 20);
  Decays *dec = reinterpret_cast<Decays *>(smem + Lay::DEC);
  float *s_skip = reinterpret_cast<float *>(smem + Lay::SKIP);

  const hymba_linear_attention &a = prm.a;
  const int warp = warp_id(), lane = lane_id();
  const unsigned wlim = prm.wlim;
  const int blk = blockIdx.x % prm.blocks;
  const int bh = blockIdx.x / prm.blocks;
  const int h = bh % a.n_heads, b = bh / a.n_heads;
  const int hk = h / (a.n_heads / a.n_qk_heads);
  const int p0 = blk * 64 * NV;                    // first state row (column of v and o)
  const int pn = min(64 * NV, a.dv - p0);          // and how many
  const int len = linear_length(a, b);
  const int ksteps = (a.dk + 15) / 16;

  if (warp == 0 && lane == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&full[x], 1);
      mbar_init(&empty[x], 1 + 1);  // products retired, V read or the output staged over it stored
      mbar_init(&dec_full[x], 1);
      mbar_init(&dec_empty[x], 12);
    }
    mbar_init(z_full, 1);
    mbar_init(z_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(p_full, 4);
    mbar_init(o_full, 1);
    mbar_init(o_empty, 4);
    mbar_init(k_full, 128);
    mbar_init(c_full, 1);
    mbar_init(sb_full, 128);
    mbar_init(qs_done, 1);
    mbar_init(o_staged, 4);
    mbar_init(drain, 1);
    fence_barrier_init();
    tmem_slot[1] = *reinterpret_cast<volatile unsigned *>(&g_err_lin);
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  for (int i = threadIdx.x; i < 64 * NV; i += kThreads)
    s_skip[i] = a.skip && i < pn ? a.skip[(long long)h * a.dv + p0 + i] : 0.f;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot[0];
  const bool failed = tmem_slot[1] != 0u;
  const int chunks = failed ? 0 : (len + C - 1) / C;
  const uint32_t tS = tmem, tO = tmem + 128, tX = tmem + 256, tC = tmem + 384;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegCtrl));
    if (warp == 0) {
      if (lane == 0) {
        // ---------------- TMA producer ----------------
        bool ok = true;
        int c = 0, nz = 0;
        for (; c < chunks; ++c) {
          const int st = c % ST;
          const uint32_t ph = uint32_t(c / ST) & 1u;
          if (!one_wait(&empty[st], ph ^ 1u, wlim)) { ok = false; break; }
          uint8_t *dst = smem + st * Lay::STAGE;
          mbar_arrive_expect_tx(&full[st], Lay::STAGE);
          for (int x = 0; x < NK; ++x) {
            tma_load_4d(dst + Lay::K + x * kAtom, &tmK, &full[st], 64 * x, hk, c * C, b);
            tma_load_4d(dst + Lay::Q + x * kAtom, &tmQ, &full[st], 64 * x, hk, c * C, b);
          }
          for (int x = 0; x < NV; ++x)
            tma_load_4d(dst + Lay::V + x * kAtom, &tmV, &full[st], p0 + 64 * x, h, c * C, b);
          if (Lay::TILE && a.gate) {
            if (!one_wait(z_empty, (uint32_t(c) & 1u) ^ 1u, wlim)) { ok = false; ++c; break; }
            mbar_arrive_expect_tx(z_full, NV * kAtom);
            for (int x = 0; x < NV; ++x)
              tma_load_4d(smem + Lay::Z + x * kAtom, &tmZ, z_full, p0 + 64 * x, h, c * C, b);
            ++nz;
          }
        }
        if (!ok) {
          // the copies in flight land before the CTA ends
          for (int q = c > ST ? c - ST : 0; q < c; ++q)
            mbar_wait_drain(&full[q % ST], uint32_t(q / ST) & 1u, &g_err_lin, wlim);
          if (nz) mbar_wait_drain(z_full, uint32_t(nz - 1) & 1u, &g_err_lin, wlim);
        }
      }
    } else if (warp == 1) {
      if (lane == 0) {
        // ---------------- MMA issuer ----------------
        constexpr uint32_t idS = make_idesc(C, 1, 0, 0);
        constexpr uint32_t idPV = make_idesc(64 * NV, 1, 0, 1);
        constexpr uint32_t idQS = make_idesc(64 * NV, 1, 0, 0);
        const uint32_t idC = make_idesc(NK == 1 ? 128 : 16 * ksteps, 1, 1, 1);
        constexpr uint32_t idCl = make_idesc(64, 1, 1, 1);
        const uint32_t mid = smem_u32(smem + Lay::MID), sb = smem_u32(smem + Lay::SB);
        for (int c = 0; c < chunks; ++c) {
          const int st = c % ST;
          const uint32_t ph = uint32_t(c) & 1u;
          const uint32_t q = smem_u32(smem + st * Lay::STAGE + Lay::Q);
          const uint32_t k = smem_u32(smem + st * Lay::STAGE + Lay::K);
          const uint32_t v = smem_u32(smem + st * Lay::STAGE + Lay::V);
          const int jsteps = (min(C, len - c * C) + 15) / 16;  // 16-row steps that hold rows
          // scores (their columns were last read by the previous chunk's P V, in order)
          if (!one_wait(&full[st], uint32_t(c / ST) & 1u, wlim)) break;
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < ksteps; ++x) {
            const uint32_t off = (x >> 2) * kAtom + (x & 3) * 32;
            mma_bf16_ss(tS, make_sdesc(q + off, 16, 1024), make_sdesc(k + off, 16, 1024), idS, x > 0);
          }
          mma_commit(s_full);
          // Q S^T: high part, then low part
          if (!one_wait(sb_full, ph, wlim) || !one_wait(o_empty, ph ^ 1u, wlim)) break;
          tc_fence_after();
#pragma unroll 1
          for (int part = 0; part < 2; ++part)
#pragma unroll 1
            for (int x = 0; x < ksteps; ++x) {
              const uint32_t soff = part * Lay::SB_PART + (x >> 2) * (NV * kAtom / 2) + (x & 3) * 32;
              mma_bf16_ss(tX, make_sdesc(q + (x >> 2) * kAtom + (x & 3) * 32, 16, 1024),
                          make_sdesc(sb + soff, 16, 1024), idQS, part > 0 || x > 0);
            }
          mma_commit(qs_done);
          // P V; in a chunk that ends early only once the rows behind the sequence are zero
          if (a.lengths && len - c * C < C && !one_wait(k_full, ph, wlim)) break;
          if (!one_wait(p_full, ph, wlim)) break;
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < jsteps; ++x)
            mma_bf16_ts(tO, tS + 8 * x, make_sdesc(v + x * 2048, kAtom, 1024), idPV, x > 0);
          mma_commit(o_full);
          // V^T K': high parts (over the keys), middle parts, low parts (over the queries); with
          // dk <= 64 the first two at once, as 64 columns each of one operand, and the low parts
          // added to the middle ones
          if (!one_wait(k_full, ph, wlim)) break;
          tc_fence_after();
          if constexpr (NK == 1) {
#pragma unroll 1
            for (int x = 0; x < jsteps; ++x)
              mma_bf16_ss(tC, make_sdesc(v + x * 2048, kAtom, 1024), make_sdesc(k + x * 2048, mid - k, 1024), idC, x > 0);
#pragma unroll 1
            for (int x = 0; x < jsteps; ++x)
              mma_bf16_ss(tC + 64, make_sdesc(v + x * 2048, kAtom, 1024), make_sdesc(q + x * 2048, kAtom, 1024), idCl, 1);
          } else {
#pragma unroll 1
            for (int part = 0; part < 3; ++part) {
              const uint32_t kp = part == 0 ? k : part == 1 ? mid : q;
#pragma unroll 1
              for (int x = 0; x < jsteps; ++x)
                mma_bf16_ss(tC, make_sdesc(v + x * 2048, kAtom, 1024), make_sdesc(kp + x * 2048, kAtom, 1024), idC,
                            part > 0 || x > 0);
            }
          }
          mma_commit(c_full);
          mma_commit(&empty[st]);
        }
        // the products in flight end before tensor memory is released
        mma_commit(drain);
        mbar_wait_drain(drain, 0, &g_err_lin, wlim);
      }
    } else if (warp == 2) {
      // ---------------- decays: lane l takes rows 4 l .. 4 l + 3 of a chunk ----------------
      const float *gp = a.log_decay ? a.log_decay + b * a.decay_batch + h * a.decay_head : nullptr;
      const float *sp = a.in_scale ? a.in_scale + b * a.scale_batch + h * a.scale_head : nullptr;
      float g[4], s[4];
      auto fetch = [&](int c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const long long t = (long long)c * C + 4 * lane + i;
          const bool in = t < len;
          g[i] = in && gp ? gp[t * a.decay_row] : 0.f;
          s[i] = in ? (sp ? sp[t * a.scale_row] : 1.f) : 0.f;
        }
      };
      if (chunks > 0) fetch(0);
      for (int c = 0; c < chunks; ++c) {
        double G[4];
        float si[4];
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum += (double)linear_log_decay(g[i]) * 1.4426950408889634074;
          G[i] = sum;
          si[i] = s[i];
        }
        if (c + 1 < chunks) fetch(c + 1);
        double before = sum;  // inclusive scan of the lanes' sums, then exclusive
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const double o = __shfl_up_sync(0xffffffffu, before, m);
          if (lane >= m) before += o;
        }
        before -= sum;
#pragma unroll
        for (int i = 0; i < 4; ++i) G[i] += before;
        const double end = __shfl_sync(0xffffffffu, G[3], 31);
        const double blk_end = __shfl_sync(0xffffffffu, G[3], lane | 7);
        if (!warp_wait(&dec_empty[c & 1], (uint32_t(c >> 1) & 1u) ^ 1u, wlim)) break;
        Decays &d = dec[c & 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 4 * lane + i;
          const float hi = (float)rint(G[i] * 8.0) * 0.125f;
          d.hi[r] = hi;
          d.lo[r] = (float)(G[i] - (double)hi);
          d.s[r] = si[i];
          d.c[r] = si[i] * exp2f((float)(blk_end - G[i]));
          d.w[r] = si[i] * exp2f((float)(end - G[i]));
          d.e[r] = exp2f((float)G[i]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&dec_full[c & 1]);
      }
    }
  } else if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegScores));
    // ---------------- scores: one row of the chunk per thread ----------------
    const int w = warp - 4, r = 32 * w + lane;
    const uint32_t lanes = uint32_t(32 * w) << 16;
    for (int c = 0; c < chunks; ++c) {
      const uint32_t ph = uint32_t(c) & 1u;
      const Decays &d = dec[c & 1];
      if (!warp_wait(&dec_full[c & 1], uint32_t(c >> 1) & 1u, wlim)) break;
      const float hi = d.hi[r], lo = d.lo[r];
      if (!warp_wait(s_full, ph, wlim)) break;
      tc_fence_after();
      // Row r of warp w sees the whole blocks of 32 columns before block w, the part of its
      // own block up to its diagonal, and nothing behind.  A whole block's factors split at
      // the block's end, exp(G_r - G_end) and s_j exp(G_end - G_j), neither above one, so
      // only the diagonal block takes an exponential per element.
#pragma unroll 1
      for (int J = 0; J < 4; ++J) {
        uint32_t pk[16];
        if (J > w) {
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = 0u;
        } else {
          uint32_t sc[32];
          tmem_ld32(tS + lanes + 32 * J, sc);
          tmem_wait_ld();
          if (J < w) {
          const float f = ex2_ftz((hi - d.hi[32 * J + 31]) + (lo - d.lo[32 * J + 31]));
          const float2 f2 = make_float2(f, f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 cj = *reinterpret_cast<const float4 *>(&d.c[32 * J + 4 * i]);
            const float2 x = fmul2(fmul2(make_float2(__uint_as_float(sc[4 * i]), __uint_as_float(sc[4 * i + 1])), f2),
                                   make_float2(cj.x, cj.y));
            const float2 y = fmul2(fmul2(make_float2(__uint_as_float(sc[4 * i + 2]), __uint_as_float(sc[4 * i + 3])), f2),
                                   make_float2(cj.z, cj.w));
            pk[2 * i] = pack_bf16x2(x.x, x.y);
            pk[2 * i + 1] = pack_bf16x2(y.x, y.y);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 h4 = *reinterpret_cast<const float4 *>(&d.hi[32 * J + 4 * i]);
            const float4 l4 = *reinterpret_cast<const float4 *>(&d.lo[32 * J + 4 * i]);
            const float4 s4 = *reinterpret_cast<const float4 *>(&d.s[32 * J + 4 * i]);
            const float hj[4] = {h4.x, h4.y, h4.z, h4.w}, lj[4] = {l4.x, l4.y, l4.z, l4.w};
            const float sj[4] = {s4.x, s4.y, s4.z, s4.w};
            float x[4];
#pragma unroll
            for (int m = 0; m < 4; ++m)
              x[m] = 4 * i + m <= lane
                         ? __uint_as_float(sc[4 * i + m]) * (sj[m] * ex2_ftz((hi - hj[m]) + (lo - lj[m])))
                         : 0.f;
            pk[2 * i] = pack_bf16x2(x[0], x[1]);
            pk[2 * i + 1] = pack_bf16x2(x[2], x[3]);
          }
        }
        }
        // P over score columns that this row has read already
        tmem_st16(tS + lanes + 16 * J, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(p_full);
        mbar_arrive(&dec_empty[c & 1]);
      }
    }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegOut));
    // ---------------- output: one row of the chunk per thread ----------------
    const int w = warp - 12, r = 32 * w + lane;
    const uint32_t lanes = uint32_t(32 * w) << 16;
    __nv_bfloat16 *op = reinterpret_cast<__nv_bfloat16 *>(a.o) + b * a.o_batch + h * a.o_head + p0;
    const __nv_bfloat16 *zp =
        reinterpret_cast<const __nv_bfloat16 *>(a.gate) + (a.gate ? b * a.gate_batch + h * a.gate_head + p0 : 0);
    for (int c = 0; c < chunks; ++c) {
      const uint32_t ph = uint32_t(c) & 1u;
      const int st = c % ST;
      const long long t = (long long)c * C + r;
      const bool live = t < len;
      // rows behind a sequence's end inside the tensor must stay as they were, which a tile
      // store would not leave them: such a chunk's rows are stored one by one
      const bool by_row = a.lengths && len - c * C < C;
      if (!warp_wait(&dec_full[c & 1], uint32_t(c >> 1) & 1u, wlim)) break;
      const float e = dec[c & 1].e[r];
      __syncwarp();
      if (lane == 0) mbar_arrive(&dec_empty[c & 1]);
      const uint8_t *vs = smem + st * Lay::STAGE + Lay::V;
      uint8_t *os = Lay::TILE ? smem + Lay::Z : smem + st * Lay::STAGE + Lay::V;
      // the tile: this chunk's gate, or free of the last chunk's output
      if (Lay::TILE && !warp_wait(a.gate ? z_full : z_empty, a.gate ? ph : ph ^ 1u, wlim)) break;
      if (!warp_wait(o_full, ph, wlim)) break;
      if (!Lay::TILE && !warp_wait(c_full, ph, wlim)) break;  // V has been read
      tc_fence_after();
      const float2 e2 = make_float2(e, e), sc2 = make_float2(a.scale, a.scale);
#pragma unroll 1
      for (int x = 0; x < 2 * NV; ++x) {
        uint32_t o1[32], o2[32];
        tmem_ld32(tO + lanes + 32 * x, o1);
        tmem_ld32(tX + lanes + 32 * x, o2);
        tmem_wait_ld();
        if (x == 2 * NV - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_empty);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {  // 8 columns: one 16-byte piece of v, the gate and o
          const int piece = 4 * (x & 1) + m, col = 32 * x + 8 * m;
          const uint32_t off = (x >> 1) * kAtom + r * 128 + ((piece ^ (r & 7)) << 4);
          float2 y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int q = 8 * m + 2 * i;
            y[i] = fmul2(sc2, ffma2(e2, make_float2(__uint_as_float(o2[q]), __uint_as_float(o2[q + 1])),
                                    make_float2(__uint_as_float(o1[q]), __uint_as_float(o1[q + 1]))));
          }
          if (a.skip) {
            const uint4 vv = *reinterpret_cast<const uint4 *>(vs + off);
            const float4 k0 = *reinterpret_cast<const float4 *>(&s_skip[col]);
            const float4 k1 = *reinterpret_cast<const float4 *>(&s_skip[col + 4]);
            y[0] = ffma2(make_float2(k0.x, k0.y), make_float2(bf16_lo(vv.x), bf16_hi(vv.x)), y[0]);
            y[1] = ffma2(make_float2(k0.z, k0.w), make_float2(bf16_lo(vv.y), bf16_hi(vv.y)), y[1]);
            y[2] = ffma2(make_float2(k1.x, k1.y), make_float2(bf16_lo(vv.z), bf16_hi(vv.z)), y[2]);
            y[3] = ffma2(make_float2(k1.z, k1.w), make_float2(bf16_lo(vv.w), bf16_hi(vv.w)), y[3]);
          }
          if (a.gate) {
            uint4 zz = make_uint4(0u, 0u, 0u, 0u);
            if constexpr (Lay::TILE) zz = *reinterpret_cast<const uint4 *>(os + off);
            else if (live && col < pn) zz = __ldg(reinterpret_cast<const uint4 *>(zp + t * a.gate_row + col));
            y[0] = fmul2(y[0], make_float2(bf16_lo(zz.x), bf16_hi(zz.x)));
            y[1] = fmul2(y[1], make_float2(bf16_lo(zz.y), bf16_hi(zz.y)));
            y[2] = fmul2(y[2], make_float2(bf16_lo(zz.z), bf16_hi(zz.z)));
            y[3] = fmul2(y[3], make_float2(bf16_lo(zz.w), bf16_hi(zz.w)));
          }
          const uint4 out = make_uint4(pack_bf16x2(y[0].x, y[0].y), pack_bf16x2(y[1].x, y[1].y),
                                       pack_bf16x2(y[2].x, y[2].y), pack_bf16x2(y[3].x, y[3].y));
          if (!by_row) *reinterpret_cast<uint4 *>(os + off) = out;
          else if (live && col < pn) st_global_v4(op + t * a.o_row + col, out.x, out.y, out.z, out.w);
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_staged);
      if (w == 0 && lane == 0 && one_wait(o_staged, ph, wlim)) {  // every row staged, V read
        if (Lay::TILE) mbar_arrive(&empty[st]);
        if (!by_row) {
          for (int x = 0; x < NV; ++x)
            if (64 * x < pn) tma_store_4d(&tmO, os + x * kAtom, p0 + 64 * x, h, c * C, b);
          bulk_commit();
          bulk_wait_read();
        }
        mbar_arrive(Lay::TILE ? z_empty : &empty[st]);
      }
    }
    if (w == 0 && lane == 0) bulk_wait_all();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegState));
    // ---------------- state: row r of the chunk's keys, row r of the state block ----------------
    const int w = warp - 8, r = 32 * w + lane;
    const uint32_t lanes = uint32_t(32 * w) << 16;
    const long long dense = (long long)a.dv * a.dk;
    const bool mine = r < pn;
    float S[64 * NK];
    {
      const float *src = a.state_in + (a.state_in ? b * a.state_in_batch + h * dense + (long long)(p0 + r) * a.dk : 0);
#pragma unroll
      for (int n = 0; n < 64 * NK; n += 4) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.state_in && mine && n < a.dk) x = *reinterpret_cast<const float4 *>(src + n);
        S[n] = x.x, S[n + 1] = x.y, S[n + 2] = x.z, S[n + 3] = x.w;
      }
    }
    // the state as the operand of Q S^T: high and low bf16 parts
    auto write_state = [&] {
      if (r < 64 * NV) {
        uint8_t *sb = smem + Lay::SB + r * 128;
#pragma unroll
        for (int n = 0; n < 64 * NK; n += 8) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 x = make_float2(S[n + 2 * i], S[n + 2 * i + 1]);
            hi[i] = high_pair(x);
            const float2 y = fsub2(x, make_float2(bf16_lo(hi[i]), bf16_hi(hi[i])));
            lo[i] = pack_bf16x2(y.x, y.y);
          }
          const uint32_t off = (n >> 6) * (NV * kAtom / 2) + ((((n & 63) >> 3) ^ (r & 7)) << 4);
          *reinterpret_cast<uint4 *>(sb + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4 *>(sb + Lay::SB_PART + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_proxy_async();
      mbar_arrive(sb_full);
    };
    bool ok = !failed;
    if (chunks > 0) write_state();
    for (int c = 0; c < chunks; ++c) {
      const int st = c % ST;
      const uint32_t ph = uint32_t(c) & 1u;
      const int rem = len - c * C;
      const Decays &d = dec[c & 1];
      // weighted keys, split over three buffers whose operands have been read: the high parts
      // over the keys, the middle parts beside them, the low parts over the queries (the
      // scores and Q S^T are behind)
      if (!warp_wait(&dec_full[c & 1], uint32_t(c >> 1) & 1u, wlim) ||
          !warp_wait(&full[st], uint32_t(c / ST) & 1u, wlim) || !warp_wait(qs_done, ph, wlim)) {
        ok = false;
        break;
      }
      const float wj = d.w[r], decay = d.e[C - 1];
      uint8_t *krow = smem + st * Lay::STAGE + Lay::K + r * 128, *mrow = smem + Lay::MID + r * 128;
      uint8_t *qrow = smem + st * Lay::STAGE + Lay::Q + r * 128;
#pragma unroll 2
      for (int x = 0; x < 8 * NK; ++x) {
        const uint32_t off = (x >> 3) * kAtom + (((x & 7) ^ (r & 7)) << 4);
        uint4 kk = *reinterpret_cast<const uint4 *>(krow + off);
        if (r >= rem) kk = make_uint4(0u, 0u, 0u, 0u);  // rows behind the sequence, whatever they hold
        const uint32_t in[4] = {kk.x, kk.y, kk.z, kk.w};
        uint32_t hi[4], mid[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 y = fmul2(make_float2(wj, wj), make_float2(bf16_lo(in[i]), bf16_hi(in[i])));
          hi[i] = high_pair(y);
          y = fsub2(y, make_float2(bf16_lo(hi[i]), bf16_hi(hi[i])));
          mid[i] = high_pair(y);
          y = fsub2(y, make_float2(bf16_lo(mid[i]), bf16_hi(mid[i])));
          lo[i] = high_pair(y);
        }
        *reinterpret_cast<uint4 *>(krow + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(mrow + off) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
        *reinterpret_cast<uint4 *>(qrow + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      if (r >= rem) {  // 0 * v must be 0 in the products
        uint8_t *vrow = smem + st * Lay::STAGE + Lay::V + r * 128;
#pragma unroll 1
        for (int x = 0; x < 8 * NV; ++x)
          *reinterpret_cast<uint4 *>(vrow + (x >> 3) * kAtom + ((x & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async();
      mbar_arrive(k_full);
      __syncwarp();
      if (lane == 0) mbar_arrive(&dec_empty[c & 1]);
      // the chunk's contribution
      if (!warp_wait(c_full, ph, wlim)) { ok = false; break; }
      tc_fence_after();
#pragma unroll
      for (int n = 0; n < 64 * NK; n += 32) {
        if (n < 16 * ksteps) {
          uint32_t x[32], y[32];
          tmem_ld32(tC + lanes + n, x);
          if constexpr (NK == 1) tmem_ld32(tC + lanes + 64 + n, y);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (n + i < 16 * ksteps) {
              const float add = NK == 1 ? __uint_as_float(x[i]) + __uint_as_float(y[i]) : __uint_as_float(x[i]);
              S[n + i] = fmaf(decay, S[n + i], add);
            }
        }
      }
      tc_fence_before();
      if (c + 1 < chunks) write_state();  // Q S^T of this chunk is behind (k_full)
    }
    if (ok && a.state_out && mine) {
      float *dst = a.state_out + ((long long)b * a.n_heads + h) * dense + (long long)(p0 + r) * a.dk;
#pragma unroll
      for (int n = 0; n < 64 * NK; n += 4)
        if (n < a.dk) *reinterpret_cast<float4 *>(dst + n) = make_float4(S[n], S[n + 1], S[n + 2], S[n + 3]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// [batch, rows, heads, dim] bf16 as a 4-D map, boxes of 128 rows of 64 columns of one head.
bool head_map(CUtensorMap *map, const void *p, long long batch, long long rows, long long heads, int dim,
              long long sb, long long sr, long long sh) {
  // a stride over an extent of one is never used, but has to be a legal one
  const long long any = (dim + 7) / 8 * 8;
  const uint64_t dims[4] = {(uint64_t)dim, (uint64_t)heads, (uint64_t)rows, (uint64_t)batch};
  const uint64_t strides[3] = {(uint64_t)(heads > 1 ? sh : any) * 2, (uint64_t)(rows > 1 ? sr : any) * 2,
                               (uint64_t)(batch > 1 ? sb : any) * 2};
  const uint32_t box[4] = {64, 1, C, 1};
  return make_tmap(map, p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, dims, strides, box);
}

template <int NK, int NV>
hymba_status chunk_launch(const hymba_linear_attention &a, cudaStream_t s) {
  using Lay = Layout<NK, NV>;
  static_assert(Lay::TOTAL <= 232448, "shared memory of one CTA");
  static DeviceOnce attr_set;
  int dev = 0;
  cudaGetDevice(&dev);
  if (!attr_set.done(dev)) {
    if (cudaFuncSetAttribute(linear_chunk_kernel<NK, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::TOTAL) !=
        cudaSuccess) {
      set_error("linear attention: %s", cudaGetErrorString(cudaGetLastError()));
      return HYMBA_ERR_CUDA;
    }
    attr_set.mark(dev);
  }
  CUtensorMap tq, tk, tv, tz, to;
  if (!head_map(&tq, a.q, a.batch, a.n_rows, a.n_qk_heads, a.dk, a.q_batch, a.q_row, a.q_head) ||
      !head_map(&tk, a.k, a.batch, a.n_rows, a.n_qk_heads, a.dk, a.k_batch, a.k_row, a.k_head) ||
      !head_map(&tv, a.v, a.batch, a.n_rows, a.n_heads, a.dv, a.v_batch, a.v_row, a.v_head) ||
      !head_map(&to, a.o, a.batch, a.n_rows, a.n_heads, a.dv, a.o_batch, a.o_row, a.o_head))
    return HYMBA_ERR_CUDA;
  tz = tv;
  if (a.gate && !head_map(&tz, a.gate, a.batch, a.n_rows, a.n_heads, a.dv, a.gate_batch, a.gate_row, a.gate_head))
    return HYMBA_ERR_CUDA;
  Params p{};
  p.a = a;
  p.blocks = (a.dv + 64 * NV - 1) / (64 * NV);
  const long long cycles = wait_limit_cycles();
  p.wlim = cycles > 0x7fffffffLL ? 0x7fffffffu : (unsigned)cycles;
  const long long grid = (long long)a.batch * a.n_heads * p.blocks;
  if (grid > 0x7fffffffLL) {
    set_error("too many sequences and heads");
    return HYMBA_ERR_UNSUPPORTED;
  }
  launch_kernel(linear_chunk_kernel<NK, NV>, dim3((unsigned)grid), dim3(kThreads), (size_t)Lay::TOTAL, s, tq, tk, tv, tz, to,
                p);
  note_launch(1);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("linear attention launch failed: %s", cudaGetErrorString(e));
    return HYMBA_ERR_CUDA;
  }
  return HYMBA_OK;
}

}  // namespace

hymba_status linear_attention_tc(const hymba_linear_attention &a, cudaStream_t s) {
  const bool wide_k = a.dk > 64, wide_v = a.dv > 64;
  if (wide_k) return wide_v ? chunk_launch<2, 2>(a, s) : chunk_launch<2, 1>(a, s);
  return wide_v ? chunk_launch<1, 2>(a, s) : chunk_launch<1, 1>(a, s);
}

unsigned take_error_linear() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_lin, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_err_lin, &zero, sizeof(zero));
  return v;
}

}  // namespace hymba
