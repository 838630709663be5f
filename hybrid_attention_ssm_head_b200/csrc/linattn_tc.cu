// Linear attention with a decay for each head over whole sequences, bf16 storage, on the
// tensor cores (tcgen05 + TMA): the recurrence of linattn.cu in chunks of 128 rows.  With
// G_i the sum of the log decays of a chunk's rows 0..i, and S the state before the chunk,
//   o_i  = scale (sum_{j <= i} P_ij v_j + exp(G_i) S q_i)    P_ij = exp(G_i - G_j) s_j (q_i . k_j)
//   S'   = exp(G_end) S + sum_j exp(G_end - G_j) s_j v_j k_j^T
// so a chunk is four products: Q K^T, P V, Q S^T and V^T K' (K' = K with weighted rows).
//
// Precision.  q, k, v enter the products as they are stored.  P is rounded once to bf16, as
// the probabilities of the softmax attention are, and its decays come from the approximate ex2.
// In the 2-norm, against 64 bits: with skip and gate the outputs are 1.7e-3 off, the rounding of
// the output itself; without them 1.9e-3 (1 x 8320 rows of dk 128, and 7 ragged sequences of dk 16)
// to 2.2e-3, where that rounding alone is 1.7e-3.  The state is kept in fp32 registers.  As the operand of Q S^T it
// is split in two bf16 parts (16 bits), more than the bf16 output holds; the weighted keys,
// whose errors would stay in the state, in three (24 bits, all of an fp32 product): with two
// parts the state of 8320 rows was 2.5e-6 off in the 2-norm.  A chunk's contribution is
// summed in tensor memory from zero and added to the state in fp32 by the CUDA cores.
#include <algorithm>

#include "linattn.cuh"
#include "tmap.h"

namespace hymba {

HYMBA_DEVICE_ERROR_WORD(g_err_lin);

namespace {

constexpr int C = 128;         // rows per chunk
// Warpgroups: control (TMA, MMA, decays: a warp each), scores, keys, output (two), state.
constexpr int kThreads = 768;
// Registers a thread of each takes; launched with 80 each.  The state holds dk fp32 values a
// thread.
template <int NK>
struct Regs {
  static constexpr int LAUNCH = 80, CTRL = 64, SCORES = NK == 1 ? 72 : 64, KEYS = 80;
  static constexpr int OUT = NK == 1 ? 72 : 56, STATE = NK == 1 ? 120 : 160;
  static_assert(CTRL + SCORES + KEYS + 2 * OUT + STATE == 6 * LAUNCH, "the warpgroups share the launch's registers");
};
constexpr int kAtom = C * 128;  // bytes of 128 rows x 64 bf16 columns, 128-byte swizzle

struct Decays {  // of one chunk's rows, log2 units
  float hi[C], lo[C];  // G = hi + lo, hi a multiple of 1/8: differences of hi are exact
  float s[C];          // scale * input scale
  float c[C];          // scale * input scale * exp(G_end of the row's block of 32 - G)
  float w[C];          // input scale * exp(G_end of the chunk - G)
  float e[C];          // scale * exp(G)
  float end, pad[3];   // exp(G_end of the chunk)
};

// NK, NV: 64-column atoms of dk and of the CTA's dv block.  For dk <= 64 two stages of
// (Q, K, V) tiles and a gate tile fit shared memory.  Wider keys take one stage, and read the
// gate from global memory.
template <int NK, int NV>
struct Layout {
  static constexpr int STAGES = NK == 1 ? 2 : 1;
  static constexpr bool GATE = NK == 1;
  static constexpr int Q = 0, K = NK * kAtom, V = 2 * NK * kAtom, STAGE = (2 * NK + NV) * kAtom;
  static constexpr int MID = STAGES * STAGE;            // middle parts of the weighted keys
  static constexpr int SB = MID + NK * kAtom;           // state operand: hi, then lo
  static constexpr int SB_PART = NK * NV * (kAtom / 2); // 64 NV rows of 128 bytes per dk atom
  // the state product reads 128 state rows whatever dv is: for NV = 1 up to one atom behind V
  static constexpr int Z = SB + 2 * SB_PART;            // gate tile
  static constexpr int DEC = Z + (GATE ? NV * kAtom : 0);
  static constexpr int SKIP = DEC + 2 * (int)sizeof(Decays);
  static constexpr int BAR = SKIP + NV * 64 * 4;
  static constexpr int TOTAL = BAR + 32 * 8 + 1024;  // + alignment of the base
};

// Two fp32 values cut to their high 16 bits, as a bf16 pair: what is cut off is exact in fp32,
// so three such parts hold all 24 bits of a value.
__device__ __forceinline__ uint32_t high_pair(float2 x) {
  return __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
}

// A bounded wait as in common.cuh, in few instructions, since the roles share an instruction
// cache (see the kernel).  A role that gives up leaves its loop early,
// which the end of the kernel reports; a CTA that starts after that does nothing.
__device__ __forceinline__ bool one_wait(uint64_t *bar, uint32_t parity, unsigned limit) {
  const unsigned t0 = (unsigned)clock();
  while (!mbar_try_wait(bar, parity))
    if ((unsigned)clock() - t0 > limit) return false;
  return true;
}
// ... by a whole warp: all of its lanes go on, or none.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, unsigned limit) {
  return __all_sync(0xffffffffu, one_wait(bar, parity, limit));
}

__device__ __forceinline__ unsigned load_acquire(const unsigned *p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

struct Params {
  hymba_linear_attention a;
  LinearSegments seg;
  int blocks;      // dv blocks of 64 * NV columns
  unsigned wlim;   // bounded waits: SM clock cycles
};

// One CTA takes one head's (or segment's) chunks.  A chunk c runs through warps of different
// roles, each a chunk or so ahead of the next one:
//   TMA      Q, K, V, gate tiles of c + 1, c + 2
//   decays   sums of the log decays by an fp64 scan, and the factors that come from them
//   MMA      Q K^T(c + 1) | Q S^T(c) | V^T K'(c) | P V(c) onto the scaled Q S^T, in this order
//   scores   P over Q K^T in tensor memory, as the operand of P V
//   keys     the three parts of the weighted keys, ready but for the low ones' stores before
//            Q S^T is through with the queries
//   output   exp(G) Q S^T + skip v in place (of c + 1), then gate and store (of c): two
//            accumulators, so that the loop through the state does not wait for an output
//   state    fp32 state in registers: decayed, the chunk's sum added, split for Q S^T
// What has to follow one another, chunk by chunk, is state operand -> Q S^T -> low parts ->
// V^T K' -> state: about 6300 cycles a chunk, of which the products are 1300; the rest are the
// roles' CUDA-core instructions and the waits between them.  Six warps share a scheduler that
// issues in 43 % of the cycles, stalled on shared memory (which the operands of the products
// and the tiles take for half of the time) and on each other; shortening the chain alone, by
// buffers of its own for the low parts, made nothing faster.  HBM is at half of its rate: 400
// heads of 8320 rows, dk 64, dv 128, 745 us for 401 us of bytes (853 us in long runs, in which
// the board's power holds the clock at 1.7 GHz).
//   measured, 200 heads of 4224 rows / 25 of 8320 rows with dk 128 / 400 of 8320 rows:
//     one output accumulator, 32 columns at a time                   237 / 170 / 842 us
//     16 columns at a time (less code, fewer registers)              227 / 165 / 792 us
//     scores 16 columns at a time, errors reported in one place      225 / 162 / 790 us
//     keys ahead of Q S^T, V released of its own                     227 / 147 / 788 us
//     two output accumulators, skip v ahead, rows stored directly    214 / 153 / 743 us
//     gate by cp.async in place of TMA, to free a buffer for the
//     low parts                                                      269 / 158 / 967 us
//     the tiles brought into L2 ahead                                222 / 150 / 765 us
// dk > 64 (NK = 2): one stage of tiles, so that a chunk takes about 11000 cycles, and 56 bytes a thread
// are spilled in the whole kernel (none for dk <= 64).
// The code of all roles together matters: 8 % between two builds of the same work when one
// was 5 KB above the other's 71 KB.
template <int NK, int NV>
__global__ void __launch_bounds__(kThreads, 1)
    linear_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmZ,
                        const __grid_constant__ Params prm) {
  pdl_wait();
  pdl_trigger();
  using Lay = Layout<NK, NV>;
  constexpr int ST = Lay::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::BAR);
  // [2] each: a stage's (Q, K) and V tiles, decays, scores, outputs.  A barrier of which a
  // warp may look at one phase when the next is over already has two, by the chunk's parity.
  uint64_t *full = bars + 0, *empty = bars + 2, *v_full = bars + 4, *v_empty = bars + 6;
  uint64_t *dec_full = bars + 8, *dec_empty = bars + 10;
  uint64_t *s_full = bars + 12;                          // scores ready
  uint64_t *o_full = bars + 14, *o_empty = bars + 16;    // outputs ready / read
  uint64_t *z_full = bars + 18, *z_empty = bars + 19;    // gate tile
  uint64_t *p_full = bars + 20, *x_full = bars + 21;     // P written over the scores / Q S^T scaled
  uint64_t *k_full = bars + 22;                          // weighted keys ready
  uint64_t *c_full = bars + 23, *c_empty = bars + 24;    // the chunk's state ready / read
  uint64_t *sb_full = bars + 25, *qs_done = bars + 26;   // state operand ready / Q S^T done
  uint64_t *drain = bars + 27;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 28);
  Decays *dec = reinterpret_cast<Decays *>(smem + Lay::DEC);
  float *s_skip = reinterpret_cast<float *>(smem + Lay::SKIP);

  const hymba_linear_attention &a = prm.a;
  const int warp = warp_id(), lane = lane_id();
  const unsigned wlim = prm.wlim;
  // A chain's segments are handed out in order, first the first of every chain: a CTA waits
  // only for a segment that a CTA has taken before it, so every wait ends.
  unsigned task = blockIdx.x;
  if (prm.seg.chain) {
    if (threadIdx.x == 0) tmem_slot[2] = atomicAdd(prm.seg.ticket, 1u);
    __syncthreads();
    task = tmem_slot[2];
  }
  const int blk = task % prm.blocks;
  const int bhs = task / prm.blocks;
  const int bh = bhs % (a.batch * a.n_heads), seg = bhs / (a.batch * a.n_heads);
  const int h = bh % a.n_heads, b = bh / a.n_heads;
  const int hk = h / (a.n_heads / a.n_qk_heads);
  const int p0 = blk * 64 * NV;                    // first state row (column of v and o)
  const int pn = min(64 * NV, a.dv - p0);          // and how many
  const int base = seg * prm.seg.rows;             // the segment's first row
  const int len = max(0, min(linear_length(a, b) - base, prm.seg.rows));  // and how many count
  const bool outputs = prm.seg.pass == 1;          // else the segment's state alone
  const int ksteps = (a.dk + 15) / 16;

  if (warp == 0 && lane == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&full[x], 1);
      mbar_init(&empty[x], 1);
      mbar_init(&v_full[x], 1);
      mbar_init(&v_empty[x], outputs ? 1 + 8 : 1);  // products retired, V read by the output's warps
      mbar_init(&dec_full[x], 1);
      mbar_init(&s_full[x], 1);
      mbar_init(&o_full[x], 1);
      mbar_init(&o_empty[x], 8);
      mbar_init(&dec_empty[x], outputs ? 20 : 8);
    }
    mbar_init(z_full, 1);
    mbar_init(z_empty, 8);
    mbar_init(p_full, 4);
    mbar_init(x_full, 8);
    mbar_init(k_full, 128);
    mbar_init(c_full, 1);
    mbar_init(c_empty, 4);
    mbar_init(sb_full, 128);
    mbar_init(qs_done, 1);
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
  const uint32_t tS = tmem, tO = tmem + 128, tC = tmem + 384;  // tO: two chunks' outputs
  bool gave_up = false;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<NK>::CTRL));
    if (warp == 0) {
      if (lane == 0) {
        // ---------------- TMA producer ----------------
        bool ok = true;
        int c = 0;
        for (; c < chunks; ++c) {
          const int st = c % ST;
          const uint32_t ph = uint32_t(c / ST) & 1u;
          if (!one_wait(&empty[st], ph ^ 1u, wlim)) { ok = false; break; }
          uint8_t *dst = smem + st * Lay::STAGE;
          mbar_arrive_expect_tx(&full[st], (outputs ? 2 : 1) * NK * kAtom);
          for (int x = 0; x < NK; ++x) {
            tma_load_4d(dst + Lay::K + x * kAtom, &tmK, &full[st], 64 * x, hk, base + c * C, b);
            if (outputs) tma_load_4d(dst + Lay::Q + x * kAtom, &tmQ, &full[st], 64 * x, hk, base + c * C, b);
          }
          if (!one_wait(&v_empty[st], ph ^ 1u, wlim)) { ok = false; one_wait(&full[st], ph, wlim); break; }
          mbar_arrive_expect_tx(&v_full[st], NV * kAtom);
          for (int x = 0; x < NV; ++x)
            tma_load_4d(dst + Lay::V + x * kAtom, &tmV, &v_full[st], p0 + 64 * x, h, base + c * C, b);
        }
        if (!ok)  // the copies in flight land before the CTA ends
          for (int q = c > ST ? c - ST : 0; q < c; ++q) {
            one_wait(&full[q % ST], uint32_t(q / ST) & 1u, wlim);
            one_wait(&v_full[q % ST], uint32_t(q / ST) & 1u, wlim);
          }
        gave_up = !ok;
      }
    } else if (warp == 1) {
      if (lane == 0) {
        // ---------------- MMA issuer ----------------
        // Every loop over a product's 16-wide steps is unrolled, so that each instruction has
        // descriptor registers of its own: in a rolled loop one instruction's registers are
        // free for the next only when it has run (390 cycles a step against 80).
        constexpr uint32_t idS = make_idesc(C, 1, 0, 0);
        constexpr uint32_t idPV = make_idesc(64 * NV, 1, 0, 1);
        constexpr uint32_t idQS = make_idesc(64 * NV, 1, 0, 0);
        const uint32_t idC = make_idesc(NK == 1 ? 128 : 16 * ksteps, 1, 1, 1);
        constexpr uint32_t idCl = make_idesc(64, 1, 1, 1);
        const uint32_t mid = smem_u32(smem + Lay::MID), sb = smem_u32(smem + Lay::SB);
        auto stage = [&](int c, int what) { return smem_u32(smem + (c % ST) * Lay::STAGE + what); };
        // a step of 16 columns inside a 64-column atom, or of 16 rows, on a descriptor's address
        auto cols = [](int x, int atom) { return uint64_t(((x >> 2) * atom + (x & 3) * 32) >> 4); };
        constexpr uint64_t kRows16 = 2048 >> 4;
        // Q K^T of chunk c: its columns were last read by the P V before it (in order)
        auto scores = [&](int c) -> bool {
          if (!one_wait(&full[c % ST], uint32_t(c / ST) & 1u, wlim)) return false;
          tc_fence_after();
          const uint64_t dq = make_sdesc(stage(c, Lay::Q), 16, 1024), dk = make_sdesc(stage(c, Lay::K), 16, 1024);
#pragma unroll
          for (int x = 0; x < 4 * NK; ++x)
            if (x < ksteps) mma_bf16_ss(tS, dq + cols(x, kAtom), dk + cols(x, kAtom), idS, x > 0);
          mma_commit(&s_full[c & 1]);
          return true;
        };
        bool ok = chunks == 0 || !outputs || scores(0);
        for (int c = 0; c < chunks && ok; ++c) {
          ok = false;  // until the end of the chunk
          const uint32_t ph = uint32_t(c) & 1u;
          const uint32_t q = stage(c, Lay::Q), k = stage(c, Lay::K);
          const uint64_t dv = make_sdesc(stage(c, Lay::V), kAtom, 1024);
          const uint32_t out = tO + 128 * (c & 1);
          if (outputs) {
            // Q S^T: high part, then low part
            if (!one_wait(&o_empty[c & 1], (uint32_t(c >> 1) & 1u) ^ 1u, wlim) || !one_wait(sb_full, ph, wlim)) break;
            tc_fence_after();
            const uint64_t dq = make_sdesc(q, 16, 1024), ds = make_sdesc(sb, 16, 1024);
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int x = 0; x < 4 * NK; ++x)
                if (x < ksteps)
                  mma_bf16_ss(out, dq + cols(x, kAtom), ds + cols(x, NV * kAtom / 2) + part * (Lay::SB_PART >> 4), idQS,
                              part > 0 || x > 0);
            mma_commit(qs_done);
          }
          // V^T K': high parts (over the keys), middle parts, low parts (over the queries); with
          // dk <= 64 the first two at once, as 64 columns each of one operand, and the low parts
          // added to the middle ones
          if (!one_wait(c_empty, ph ^ 1u, wlim) || !one_wait(&v_full[c % ST], uint32_t(c / ST) & 1u, wlim) ||
              !one_wait(k_full, ph, wlim))
            break;
          tc_fence_after();
          auto state_part = [&](uint64_t dk, uint32_t d, uint32_t id, bool add) {
#pragma unroll
            for (int x = 0; x < 8; ++x) mma_bf16_ss(d, dv + x * kRows16, dk + x * kRows16, id, add || x > 0);
          };
          if constexpr (NK == 1) {
            state_part(make_sdesc(k, mid - k, 1024), tC, idC, false);
            state_part(make_sdesc(q, kAtom, 1024), tC + 64, idCl, true);
          } else {
            state_part(make_sdesc(k, kAtom, 1024), tC, idC, false);
            state_part(make_sdesc(mid, kAtom, 1024), tC, idC, true);
            state_part(make_sdesc(q, kAtom, 1024), tC, idC, true);
          }
          mma_commit(c_full);
          mma_commit(&empty[c % ST]);
          if (outputs) {
            // P V onto the scaled Q S^T
            if (!one_wait(p_full, ph, wlim) || !one_wait(x_full, ph, wlim)) break;
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < 8; ++x) mma_bf16_ts(out, tS + 8 * x, dv + x * kRows16, idPV, true);
            mma_commit(&o_full[c & 1]);
          }
          mma_commit(&v_empty[c % ST]);
          if (outputs && c + 1 < chunks && !scores(c + 1)) break;
          ok = true;
        }
        // the products in flight end before tensor memory is released
        mma_commit(drain);
        gave_up = !one_wait(drain, 0, wlim) || !ok;
      }
    } else if (warp == 2) {
      // ---------------- decays: lane l takes rows 4 l .. 4 l + 3 of a chunk ----------------
      const float *gp = a.log_decay ? a.log_decay + b * a.decay_batch + h * a.decay_head : nullptr;
      const float *sp = a.in_scale ? a.in_scale + b * a.scale_batch + h * a.scale_head : nullptr;
      float g[4], s[4];
      auto fetch = [&](int c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = c * C + 4 * lane + i;
          const bool in = t < len;
          g[i] = in && gp ? gp[(long long)(base + t) * a.decay_row] : 0.f;
          s[i] = in ? (sp ? sp[(long long)(base + t) * a.scale_row] : 1.f) : 0.f;
        }
      };
      double total = 0.0;
      if (chunks > 0) fetch(0);
      int c = 0;
      for (; c < chunks; ++c) {
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
        // The sum before the lane's rows: the lane below's inclusive one.  (Not the lane's own less
        // its rows: a NaN among those would reach the ones before it.)
        double before = sum;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const double o = __shfl_up_sync(0xffffffffu, before, m);
          if (lane >= m) before += o;
        }
        before = __shfl_up_sync(0xffffffffu, before, 1);
        if (lane == 0) before = 0.0;
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
          d.s[r] = a.scale * si[i];
          d.c[r] = a.scale * si[i] * ex2_ftz((float)(blk_end - G[i]));
          d.w[r] = si[i] * ex2_ftz((float)(end - G[i]));
          d.e[r] = a.scale * ex2_ftz((float)G[i]);
        }
        if (lane == 31) d.end = exp2f((float)end);
        total += end;
        __syncwarp();
        if (lane == 0) mbar_arrive(&dec_full[c & 1]);
      }
      gave_up = c < chunks;
      if (!outputs && lane == 0 && blk == 0) prm.seg.decay[bhs] = total;  // log2 of the segment's decay
    } else if (Lay::GATE && a.gate && outputs && lane == 0) {
      // ---------------- gate producer ----------------
      bool ok = true;
      int c = 0;
      for (; c < chunks; ++c) {
        if (!one_wait(z_empty, (uint32_t(c) & 1u) ^ 1u, wlim)) { ok = false; break; }
        mbar_arrive_expect_tx(z_full, NV * kAtom);
        for (int x = 0; x < NV; ++x)
          tma_load_4d(smem + Lay::Z + x * kAtom, &tmZ, z_full, p0 + 64 * x, h, base + c * C, b);
      }
      if (!ok && c > 0) one_wait(z_full, uint32_t(c - 1) & 1u, wlim);
      gave_up = !ok;
    }
  } else if (warp < 8) {
    if constexpr (Regs<NK>::SCORES < Regs<NK>::LAUNCH)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<NK>::SCORES));
    // ---------------- scores: one row of the chunk per thread ----------------
    const int w = warp - 4, r = 32 * w + lane;
    const uint32_t lanes = uint32_t(32 * w) << 16;
    int c = 0;
    for (; outputs && c < chunks; ++c) {
      const Decays &d = dec[c & 1];
      if (!warp_wait(&dec_full[c & 1], uint32_t(c >> 1) & 1u, wlim)) break;
      const float hi = d.hi[r], lo = d.lo[r];
      if (!warp_wait(&s_full[c & 1], uint32_t(c >> 1) & 1u, wlim)) break;
      tc_fence_after();
      // Row r of warp w sees the whole blocks of 32 columns before block w, the part of its
      // own block up to its diagonal, and nothing behind.  A whole block's factors split at
      // the block's end, exp(G_r - G_end) and s_j exp(G_end - G_j), neither above one, so
      // only the diagonal block takes an exponential per element.
#pragma unroll 1
      for (int x0 = 0; x0 < C; x0 += 16) {  // 16 columns
        uint32_t pk[8];
        const int J = x0 >> 5;
        if (J > w) {
#pragma unroll
          for (int i = 0; i < 8; ++i) pk[i] = 0u;
        } else {
          uint32_t sc[16];
          tmem_ld16(tS + lanes + x0, sc);
          tmem_wait_ld();
          if (J < w) {
            const float f = ex2_ftz((hi - d.hi[32 * J + 31]) + (lo - d.lo[32 * J + 31]));
            const float2 f2 = make_float2(f, f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 cj = *reinterpret_cast<const float4 *>(&d.c[x0 + 4 * i]);
              const float2 x = fmul2(fmul2(make_float2(__uint_as_float(sc[4 * i]), __uint_as_float(sc[4 * i + 1])), f2),
                                     make_float2(cj.x, cj.y));
              const float2 y = fmul2(fmul2(make_float2(__uint_as_float(sc[4 * i + 2]), __uint_as_float(sc[4 * i + 3])), f2),
                                     make_float2(cj.z, cj.w));
              pk[2 * i] = pack_bf16x2(x.x, x.y);
              pk[2 * i + 1] = pack_bf16x2(y.x, y.y);
            }
          } else {
            const int last = r - x0;  // the diagonal
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 h4 = *reinterpret_cast<const float4 *>(&d.hi[x0 + 4 * i]);
              const float4 l4 = *reinterpret_cast<const float4 *>(&d.lo[x0 + 4 * i]);
              const float4 s4 = *reinterpret_cast<const float4 *>(&d.s[x0 + 4 * i]);
              const float hj[4] = {h4.x, h4.y, h4.z, h4.w}, lj[4] = {l4.x, l4.y, l4.z, l4.w};
              const float sj[4] = {s4.x, s4.y, s4.z, s4.w};
              float x[4];
#pragma unroll
              for (int m = 0; m < 4; ++m)
                x[m] = 4 * i + m <= last
                           ? __uint_as_float(sc[4 * i + m]) * (sj[m] * ex2_ftz((hi - hj[m]) + (lo - lj[m])))
                           : 0.f;
              pk[2 * i] = pack_bf16x2(x[0], x[1]);
              pk[2 * i + 1] = pack_bf16x2(x[2], x[3]);
            }
          }
        }
        // P over score columns that this row has read already
        tmem_st8(tS + lanes + x0 / 2, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(p_full);
        mbar_arrive(&dec_empty[c & 1]);
      }
    }
    gave_up = outputs && c < chunks;
  } else if (warp >= 12 && warp < 20) {
    if constexpr (Regs<NK>::OUT < Regs<NK>::LAUNCH)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<NK>::OUT));
    // ---------------- output: half of the columns of one row of the chunk per thread ----------------
    constexpr int kCols = 32 * NV;
    const int w = (warp - 12) & 3, r = 32 * w + lane, first = kCols * ((warp - 12) >> 2);
    const uint32_t lanes = (uint32_t(32 * w) << 16) + first;
    const float *skip = s_skip + first;
    const bool skips = a.skip != nullptr, gates = a.gate != nullptr;
    // this row's 16-byte pieces of a 128-row tile
    const uint32_t row = (first >> 6) * kAtom + r * 128, p8 = (first & 63) >> 3, swz = r & 7;
    const int cols = pn - first;  // that exist
    char *orow = reinterpret_cast<char *>(a.o) + 2 * (b * a.o_batch + h * a.o_head + (base + r) * a.o_row + p0 + first);
    const char *zrow = reinterpret_cast<const char *>(a.gate);
    if (gates) zrow += 2 * (b * a.gate_batch + h * a.gate_head + (base + r) * a.gate_row + p0 + first);
    // exp(G) Q S^T + skip v of chunk c, in place; P V is added to it
    auto scale_rows = [&](int c) -> bool {
      const int st = c % ST;
      const uint8_t *vs = smem + st * Lay::STAGE + Lay::V + row;
      if (!warp_wait(&dec_full[c & 1], uint32_t(c >> 1) & 1u, wlim)) return false;
      const float e = dec[c & 1].e[r];
      if (!warp_wait(&v_full[st], uint32_t(c / ST) & 1u, wlim) || !warp_wait(qs_done, uint32_t(c) & 1u, wlim)) return false;
      tc_fence_after();
      const float2 e2 = make_float2(e, e);
      const uint32_t acc = tO + lanes + 128 * (c & 1);
#pragma unroll 1
      for (int x = 0; x < kCols; x += 16) {
        uint32_t o[16];
        tmem_ld16(acc + x, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float2 y = fmul2(e2, make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])));
          o[i] = __float_as_uint(y.x);
          o[i + 1] = __float_as_uint(y.y);
        }
        if (skips) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 v = *reinterpret_cast<const uint4 *>(vs + (((p8 + (x >> 3) + i) ^ swz) << 4));
            const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int m = 0; m < 4; m += 2) {
              const float4 d = *reinterpret_cast<const float4 *>(&skip[x + 8 * i + 2 * m]);
              uint32_t *y = o + 8 * i + 2 * m;
              const float2 y0 = ffma2(make_float2(d.x, d.y), make_float2(bf16_lo(vw[m]), bf16_hi(vw[m])),
                                      make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])));
              const float2 y1 = ffma2(make_float2(d.z, d.w), make_float2(bf16_lo(vw[m + 1]), bf16_hi(vw[m + 1])),
                                      make_float2(__uint_as_float(y[2]), __uint_as_float(y[3])));
              y[0] = __float_as_uint(y0.x);
              y[1] = __float_as_uint(y0.y);
              y[2] = __float_as_uint(y1.x);
              y[3] = __float_as_uint(y1.y);
            }
          }
        }
        tmem_st16(acc + x, o);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(x_full);
        mbar_arrive(&v_empty[st]);
        mbar_arrive(&dec_empty[c & 1]);
      }
      return true;
    };
    int c = outputs ? -1 : chunks;
    for (; c < chunks; ++c) {
      // the next chunk's Q S^T, ahead of this one's output
      if (c + 1 < chunks && !scale_rows(c + 1)) break;
      if (c < 0) continue;
      const int rows = len - c * C - 32 * w;  // rows of this warp that count (may be none)
      if (Lay::GATE && gates && !warp_wait(z_full, uint32_t(c) & 1u, wlim)) break;
      if (!warp_wait(&o_full[c & 1], uint32_t(c >> 1) & 1u, wlim)) break;
      tc_fence_after();
      const uint32_t acc = tO + lanes + 128 * (c & 1);
#pragma unroll 1
      for (int x = 0; x < kCols; x += 16) {
        uint32_t o[16], out[8];
        tmem_ld16(acc + x, o);
        uint4 z[2];
        if (gates) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if constexpr (Lay::GATE) {
              z[i] = *reinterpret_cast<const uint4 *>(smem + Lay::Z + row + (((p8 + (x >> 3) + i) ^ swz) << 4));
            } else {
              z[i] = make_uint4(0u, 0u, 0u, 0u);
              if (lane < rows && x + 8 * i < cols) z[i] = __ldg(reinterpret_cast<const uint4 *>(zrow + 2 * x + 16 * i));
            }
          }
        }
        tmem_wait_ld();
        if (x == kCols - 16) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_empty[c & 1]);
        }
        const uint32_t zw[8] = {z[0].x, z[0].y, z[0].z, z[0].w, z[1].x, z[1].y, z[1].z, z[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // columns x + 2 i, x + 2 i + 1
          float2 y = make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
          if (gates) y = fmul2(y, make_float2(bf16_lo(zw[i]), bf16_hi(zw[i])));
          out[i] = pack_bf16x2(y.x, y.y);
        }
        if (lane < rows && x < cols) {
          char *dst = orow + 2 * x;
          if (x + 8 < cols && (reinterpret_cast<uintptr_t>(dst) & 31) == 0) {  // a whole sector
            st_global_v8(dst, out[0], out[1], out[2], out[3], out[4], out[5], out[6], out[7]);
          } else {
            st_global_v4(dst, out[0], out[1], out[2], out[3]);
            if (x + 8 < cols) st_global_v4(dst + 16, out[4], out[5], out[6], out[7]);
          }
        }
      }
      __syncwarp();
      // Only here, behind the use of what was read: an arrival does not wait for loads that are
      // still on their way, and a tile released before them was overwritten under them.
      if (lane == 0) mbar_arrive(z_empty);
      if (gates) zrow += 2 * C * a.gate_row;
      orow += 2 * C * a.o_row;
    }
    gave_up = c < chunks;
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<NK>::KEYS));
    // ---------------- weighted keys: one row of the chunk per thread ----------------
    const int r = 32 * (warp - 8) + lane;
    int c = 0;
    for (; c < chunks; ++c) {
      const int st = c % ST;
      const uint32_t ph = uint32_t(c) & 1u;
      const int rem = len - c * C;
      // Split over three buffers: the high parts over the keys, whose scores are done, the middle
      // parts beside them, the low parts over the queries.  Q S^T of this chunk reads those, so
      // the low parts of one atom wait in registers: only their stores come after it.
      if (!warp_wait(&dec_full[c & 1], uint32_t(c >> 1) & 1u, wlim) || !warp_wait(&full[st], uint32_t(c / ST) & 1u, wlim) ||
          !warp_wait(c_full, ph ^ 1u, wlim) || (outputs && !warp_wait(&s_full[c & 1], uint32_t(c >> 1) & 1u, wlim)) ||
          (rem < C && !warp_wait(&v_full[st], uint32_t(c / ST) & 1u, wlim)))
        break;
      const float wj = dec[c & 1].w[r];
      uint8_t *krow = smem + st * Lay::STAGE + Lay::K + r * 128, *mrow = smem + Lay::MID + r * 128;
      uint8_t *qrow = smem + st * Lay::STAGE + Lay::Q + r * 128;
      const float2 w2 = make_float2(wj, wj);
      auto split = [&](uint32_t off, uint32_t *lo) {
        uint4 kk = *reinterpret_cast<const uint4 *>(krow + off);
        if (r >= rem) kk = make_uint4(0u, 0u, 0u, 0u);  // rows behind the sequence, whatever they hold
        const uint32_t in[4] = {kk.x, kk.y, kk.z, kk.w};
        uint32_t hi[4], mid[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 y = fmul2(w2, make_float2(bf16_lo(in[i]), bf16_hi(in[i])));
          hi[i] = high_pair(y);
          y = fsub2(y, make_float2(bf16_lo(hi[i]), bf16_hi(hi[i])));
          mid[i] = high_pair(y);
          y = fsub2(y, make_float2(bf16_lo(mid[i]), bf16_hi(mid[i])));
          lo[i] = high_pair(y);
        }
        *reinterpret_cast<uint4 *>(krow + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(mrow + off) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
      };
      uint32_t lo[32];
#pragma unroll
      for (int x = 0; x < 8; ++x) split((x ^ (r & 7)) << 4, lo + 4 * x);
      if (outputs && !warp_wait(qs_done, ph, wlim)) break;
#pragma unroll
      for (int x = 0; x < 8; ++x)
        *reinterpret_cast<uint4 *>(qrow + ((x ^ (r & 7)) << 4)) = make_uint4(lo[4 * x], lo[4 * x + 1], lo[4 * x + 2], lo[4 * x + 3]);
      if constexpr (NK == 2) {
#pragma unroll 2
        for (int x = 0; x < 8; ++x) {
          const uint32_t off = kAtom + ((x ^ (r & 7)) << 4);
          split(off, lo);
          *reinterpret_cast<uint4 *>(qrow + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
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
    }
    gave_up = c < chunks;
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<NK>::STATE));
    // ---------------- state: one row of the state block per thread ----------------
    const int w = warp - 20, r = 32 * w + lane;
    const uint32_t lanes = uint32_t(32 * w) << 16;
    const long long dense = (long long)a.dv * a.dk;
    const bool mine = r < pn;
    float2 S[32 * NK];
#pragma unroll
    for (int n = 0; n < 32 * NK; ++n) S[n] = make_float2(0.f, 0.f);
    const long long at = (long long)(p0 + r) * a.dk;  // this row in a head's state
    // The state the segment starts from: the call's, or (outputs) the one after the segments
    // before it; a segment's own state starts from zero, the first one's from the call's.
    const long long heads = (long long)a.batch * a.n_heads;
    const float *from = a.state_in ? a.state_in + b * a.state_in_batch + h * dense : nullptr;
    if (outputs && prm.seg.n > 1 && !prm.seg.chain)
      from = a.state_in ? prm.seg.state + ((prm.seg.n - 1) * heads + bh) * dense : nullptr;
    if (seg > 0) from = outputs ? prm.seg.state + ((prm.seg.chain ? 0 : seg - 1) * heads + bh) * dense : nullptr;
    unsigned *left = prm.seg.ticket + 1 + bh * prm.blocks + blk;  // chain: four warps for each segment
    bool ok = !failed;
    if (prm.seg.chain && seg > 0) {
      if (ok && lane == 0) {
        const unsigned t0 = (unsigned)clock();
        while (load_acquire(left) < 4u * seg)
          if ((unsigned)clock() - t0 > wlim) {
            ok = false;
            break;
          }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (ok && from && mine)
#pragma unroll
      for (int n = 0; n < 64 * NK; n += 4)
        if (n < a.dk) {
          const float4 x = __ldcg(reinterpret_cast<const float4 *>(from + at + n));  // other SMs' stores among them
          S[n / 2] = make_float2(x.x, x.y);
          S[n / 2 + 1] = make_float2(x.z, x.w);
        }
    auto store_state = [&](float *dst) {
#pragma unroll
      for (int n = 0; n < 64 * NK; n += 4)
        if (mine && n < a.dk)
          *reinterpret_cast<float4 *>(dst + at + n) = make_float4(S[n / 2].x, S[n / 2].y, S[n / 2 + 1].x, S[n / 2 + 1].y);
    };
    if (!outputs && seg == 0 && a.state_in)  // a copy for the outputs' pass, which may write in place
      store_state(prm.seg.state + ((prm.seg.n - 1) * heads + bh) * dense);
    for (int c = 0; ok && c < chunks; ++c) {
      const uint32_t ph = uint32_t(c) & 1u;
      // The state as the operand of Q S^T: high and low bf16 parts.  The buffer's last reader,
      // the Q S^T before, ran ahead of the state product that c_full told of.
      if (outputs && r < 64 * NV) {
        uint8_t *sb = smem + Lay::SB + r * 128;
#pragma unroll
        for (int n = 0; n < 64 * NK; n += 8) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 x = S[n / 2 + i];
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
      if (!warp_wait(&dec_full[c & 1], uint32_t(c >> 1) & 1u, wlim)) { ok = false; break; }
      const float decay = dec[c & 1].end;
      if (!warp_wait(c_full, ph, wlim)) { ok = false; break; }
      tc_fence_after();
      const float2 d2 = make_float2(decay, decay);
#pragma unroll
      for (int n = 0; n < 64 * NK; n += 16) {
        if (n < a.dk) {  // columns from dk on stay zero
          uint32_t x[16], y[16];
          tmem_ld16(tC + lanes + n, x);
          if constexpr (NK == 1) tmem_ld16(tC + lanes + 64 + n, y);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float2 add = make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
            if constexpr (NK == 1) add = fadd2(add, make_float2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1])));
            S[n / 2 + i] = ffma2(d2, S[n / 2 + i], add);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(c_empty);
        mbar_arrive(&dec_empty[c & 1]);
      }
    }
    float *dst = !outputs ? prm.seg.state + (long long)bhs * dense
                 : a.state_out && seg == prm.seg.n - 1 ? a.state_out + (long long)bh * dense : nullptr;
    const bool hand_on = prm.seg.chain && seg < prm.seg.n - 1;
    if (hand_on) dst = prm.seg.state + bh * dense;
    if (ok && dst) store_state(dst);
    if (ok && hand_on) {
      __threadfence();
      __syncwarp();
      if (lane == 0) atomicAdd(left, 1u);
    }
    gave_up = !ok && !failed;
  }
  if (gave_up) atomicOr(&g_err_lin, kErrTimeout);

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Blocks of the state's rows (columns of v and o): a CTA takes 64 or 128 of them.
int dv_blocks(const hymba_linear_attention &a) { return a.dv > 64 ? (a.dv + 127) / 128 : 1; }

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
hymba_status chunk_launch(const hymba_linear_attention &a, LinearSegments seg, cudaStream_t s) {
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
  CUtensorMap tq, tk, tv, tz;
  if (!head_map(&tq, a.q, a.batch, a.n_rows, a.n_qk_heads, a.dk, a.q_batch, a.q_row, a.q_head) ||
      !head_map(&tk, a.k, a.batch, a.n_rows, a.n_qk_heads, a.dk, a.k_batch, a.k_row, a.k_head) ||
      !head_map(&tv, a.v, a.batch, a.n_rows, a.n_heads, a.dv, a.v_batch, a.v_row, a.v_head))
    return HYMBA_ERR_CUDA;
  tz = tv;
  if (a.gate && !head_map(&tz, a.gate, a.batch, a.n_rows, a.n_heads, a.dv, a.gate_batch, a.gate_row, a.gate_head))
    return HYMBA_ERR_CUDA;
  Params p{};
  p.a = a;
  p.seg = seg;
  p.blocks = dv_blocks(a);
  // When lengths differ, all segments of a long chain may run beside each other: the last one then
  // waits for all before it, at 50 (dk <= 64) to 90 cycles a row, and so do the other roles of its CTA.
  const long long cycles = std::max<long long>(wait_limit_cycles(), seg.chain ? 500LL * seg.rows * seg.n : 0);
  p.wlim = cycles > 0x7fffffffLL ? 0x7fffffffu : (unsigned)cycles;
  const long long ctas = (long long)a.batch * a.n_heads * p.blocks;
  if (ctas * seg.n > 0x7fffffffLL) {
    set_error("too many sequences and heads");
    return HYMBA_ERR_UNSUPPORTED;
  }
  for (p.seg.pass = seg.n > 1 && !seg.chain ? 0 : 1; p.seg.pass < 2; ++p.seg.pass) {
    if (p.seg.pass == 1) linear_prefix(a, p.seg, s);
    const long long grid = ctas * (p.seg.pass ? seg.n : seg.n - 1);
    launch_kernel(linear_chunk_kernel<NK, NV>, dim3((unsigned)grid), dim3(kThreads), (size_t)Lay::TOTAL, s, tq, tk, tv, tz, p);
    note_launch(1);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("linear attention launch failed: %s", cudaGetErrorString(e));
    return HYMBA_ERR_CUDA;
  }
  return HYMBA_OK;
}

}  // namespace

// One CTA takes a whole SM, a head's chunks one after another.  When the heads leave SMs idle
// the rows are split into segments, as many as fit beside each other: the segments' own
// states first (about 0.6 of a chunk's time each), then their outputs.  That takes 1.6 / n of
// the time in n segments, and a second launch about as long as four chunks: 25 heads of 8320
// rows 200 us whole and 88 us in five segments, with dk 128 379 and 157 us; 28 heads of 517 rows
// 24 us whole and 30 us in two.
//
// More heads than SMs run in rounds, the last of which leaves SMs idle.  Then each head's rows
// are a chain of segments that CTAs take up in turn, so that the rounds are shorter; a CTA's
// start and end cost about as much as 0.7 of a chunk.  200 heads of 4224 rows 234 us whole and
// 206 us in chains of two, 180 heads with dk 128 399 and 314 us.
LinearSegments linear_attention_tc_segments(const hymba_linear_attention &a) {
  LinearSegments g{};
  const long long ctas = (long long)a.batch * a.n_heads * dv_blocks(a);
  const int chunks = (a.n_rows + C - 1) / C;
  g.n = 1;
  g.rows = chunks * C;
  if (ctas <= 148) {
    const long long most = std::max<long long>(1, std::min<long long>(148 / std::max<long long>(1, ctas), chunks / 2));
    const int per = (chunks + (int)most - 1) / (int)most, n = (chunks + per - 1) / per;
    if (5 * chunks * (long long)n - 8 * chunks >= 20 * (long long)n) {  // chunks (1 - 1.6 / n) >= 4
      g.n = n;
      g.rows = per * C;
    }
    return g;
  }
  double best = 0.0;
  for (int want = 1; want <= std::min(32, std::max(1, chunks / 4)); ++want) {  // of at least four chunks
    const int per = (chunks + want - 1) / want, n = (chunks + per - 1) / per;
    const double cost = (double)((ctas * n + 147) / 148) * (per + 0.7);
    if (want == 1 || cost < 0.97 * best) {
      best = cost;
      g.n = n;
      g.rows = per * C;
    }
  }
  g.chain = g.n > 1;
  return g;
}

size_t linear_attention_tc_tickets(const hymba_linear_attention &a) {
  return 1 + (size_t)a.batch * a.n_heads * dv_blocks(a);
}

hymba_status linear_attention_tc(const hymba_linear_attention &a, const LinearSegments &seg, cudaStream_t s) {
  const bool wide_k = a.dk > 64, wide_v = a.dv > 64;
  if (wide_k) return wide_v ? chunk_launch<2, 2>(a, seg, s) : chunk_launch<2, 1>(a, seg, s);
  return wide_v ? chunk_launch<1, 2>(a, seg, s) : chunk_launch<1, 1>(a, seg, s);
}

unsigned take_error_linear() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_lin, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_err_lin, &zero, sizeof(zero));
  return v;
}

}  // namespace hymba
