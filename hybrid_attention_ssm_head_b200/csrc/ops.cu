// Host side of the operators of include/hymba.h (head norm/rotation, linear attention):
// argument validation, then the launchers.
#include <algorithm>
#include <cmath>

#include "kernels.h"
#include "profile.h"

using namespace hymba;

#define FAIL(code, ...)        \
  do {                         \
    set_error(__VA_ARGS__);    \
    return code;               \
  } while (0)

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
long long esize(hymba_dtype d) { return d == HYMBA_BF16 ? 2 : 4; }

// One [batch, rows, heads, dim] grid: extents and element strides, outermost first.
struct Grid {
  long long n[3], st[3], dim;
  // The elements from the first to behind the last; strides over an extent of one count zero.
  long long span() const {
    long long s = dim;
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1) s += (n[i] - 1) * st[i];
    return s;
  }
};

constexpr long long kMaxStride = 1LL << 38;  // elements: byte strides below 2^40 (TMA)

// Strides of at least one element where the extent is above one, 16-byte multiples.
hymba_status check_grid(const char *name, const void *p, const Grid &g, long long es) {
  if (!p || !aligned16(p)) FAIL(HYMBA_ERR_INVALID_ARG, "%s null or not 16-byte aligned", name);
  for (int i = 0; i < 3; ++i) {
    if (g.n[i] <= 1) continue;
    if (g.st[i] <= 0 || g.st[i] >= kMaxStride)
      FAIL(HYMBA_ERR_INVALID_ARG, "%s: stride %lld outside 1..2^38", name, g.st[i]);
    if ((g.st[i] * es) % 16) FAIL(HYMBA_ERR_INVALID_ARG, "%s: stride %lld is not a multiple of 16 bytes", name, g.st[i]);
  }
  return HYMBA_OK;
}

// No two elements of a written grid share an address: with the extents sorted by stride, each
// stride clears everything below it.
hymba_status check_written(const char *name, const Grid &g) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int x, int y) { return g.st[x] < g.st[y]; });
  long long inner = g.dim;
  for (int i : order) {
    if (g.n[i] <= 1) continue;
    if (g.st[i] < inner) FAIL(HYMBA_ERR_INVALID_ARG, "%s: rows written through these strides overlap", name);
    inner += (g.n[i] - 1) * g.st[i];
  }
  return HYMBA_OK;
}

bool ranges_overlap(const void *a, long long abytes, const void *b, long long bbytes) {
  const char *x = reinterpret_cast<const char *>(a), *y = reinterpret_cast<const char *>(b);
  return x < y + bbytes && y < x + abytes;
}

bool bad_dtype(hymba_dtype d) { return d != HYMBA_F32 && d != HYMBA_BF16; }

// ---- head norm and rotation -------------------------------------------------------------
hymba_status check_heads(const char *name, const hymba_qk_norm_rope_args &a, const hymba_head_rows &v) {
  if (v.n_heads < 0) FAIL(HYMBA_ERR_INVALID_ARG, "%s: n_heads < 0", name);
  if (v.n_heads == 0) return HYMBA_OK;
  const long long es = esize(a.dtype);
  const Grid in = {{a.batch, a.n_rows, v.n_heads}, {v.in_batch, v.in_row, v.in_head}, a.head_dim};
  const Grid out = {{a.batch, a.n_rows, v.n_heads}, {v.out_batch, v.out_row, v.out_head}, a.head_dim};
  hymba_status st;
  if ((st = check_grid(name, v.in, in, es)) != HYMBA_OK) return st;
  if ((st = check_grid(name, v.out, out, es)) != HYMBA_OK) return st;
  if ((st = check_written(name, out)) != HYMBA_OK) return st;
  if (v.weight && !aligned16(v.weight)) FAIL(HYMBA_ERR_INVALID_ARG, "%s: weight not 16-byte aligned", name);
  if (v.weight && !a.norm) FAIL(HYMBA_ERR_INVALID_ARG, "%s: a weight without the norm", name);
  bool same = v.in == v.out;
  for (int i = 0; i < 3; ++i) same = same && (in.n[i] <= 1 || in.st[i] == out.st[i]);
  if (!same && v.in == v.out) FAIL(HYMBA_ERR_INVALID_ARG, "%s: in place needs the same strides for in and out", name);
  return HYMBA_OK;
}

}  // namespace

// The rotation's own numbers; `width` is the head's dimension.
hymba_status hymba::check_rope(const hymba_rope &r, int width) {
  if (r.dim < 0 || r.dim % 2 || r.dim > width)
    FAIL(HYMBA_ERR_INVALID_ARG, "rope dim %d: even, 0..%d", r.dim, width);
  if (r.dim == 0) return HYMBA_OK;
  if (r.layout != HYMBA_ROPE_PAIRS && r.layout != HYMBA_ROPE_HALVES) FAIL(HYMBA_ERR_INVALID_ARG, "rope layout %d", r.layout);
  if (!(r.base > 1.0) || !std::isfinite(r.base)) FAIL(HYMBA_ERR_INVALID_ARG, "rope base must be above 1");
  if (!(r.attn_factor > 0.f) || !std::isfinite(r.attn_factor)) FAIL(HYMBA_ERR_INVALID_ARG, "rope attn_factor must be above 0");
  if (r.scaling == HYMBA_ROPE_SCALE_NONE) return HYMBA_OK;
  if (r.scaling != HYMBA_ROPE_SCALE_LINEAR && r.scaling != HYMBA_ROPE_SCALE_WAVELENGTH)
    FAIL(HYMBA_ERR_INVALID_ARG, "rope scaling %d", r.scaling);
  if (!(r.factor > 0.0) || !std::isfinite(r.factor)) FAIL(HYMBA_ERR_INVALID_ARG, "rope factor must be above 0");
  if (r.scaling == HYMBA_ROPE_SCALE_WAVELENGTH &&
      (!(r.orig_len > 0.0) || !std::isfinite(r.orig_len) || !(r.low_turns >= 0.0) ||
       !(r.high_turns > r.low_turns) || !std::isfinite(r.high_turns)))
    FAIL(HYMBA_ERR_INVALID_ARG, "rope by wavelength needs orig_len > 0 and 0 <= low_turns < high_turns");
  return HYMBA_OK;
}

namespace {

// ---- linear attention ---------------------------------------------------------------------
struct LinearGrids {
  Grid q, k, v, o, z;
};
LinearGrids linear_grids(const hymba_linear_attention &a) {
  const long long B = a.batch, L = a.n_rows, H = a.n_heads, K = a.n_qk_heads;
  return {{{B, L, K}, {a.q_batch, a.q_row, a.q_head}, a.dk},
          {{B, L, K}, {a.k_batch, a.k_row, a.k_head}, a.dk},
          {{B, L, H}, {a.v_batch, a.v_row, a.v_head}, a.dv},
          {{B, L, H}, {a.o_batch, a.o_row, a.o_head}, a.dv},
          {{B, L, H}, {a.gate_batch, a.gate_row, a.gate_head}, a.dv}};
}

hymba_status check_linear_sizes(const hymba_linear_attention &a) {
  if (bad_dtype(a.dtype)) FAIL(HYMBA_ERR_INVALID_ARG, "dtype %d", a.dtype);
  if (a.batch < 1 || a.n_rows < 1 || a.n_heads < 1 || a.n_qk_heads < 1 || a.dk < 1 || a.dv < 1)
    FAIL(HYMBA_ERR_INVALID_ARG, "every size must be positive");
  if (a.n_heads % a.n_qk_heads) FAIL(HYMBA_ERR_INVALID_ARG, "n_heads %% n_qk_heads != 0");
  if (a.dk % 8 || a.dk > 128) FAIL(HYMBA_ERR_UNSUPPORTED, "dk %d: a multiple of 8 up to 128", a.dk);
  if (a.dv % 8 || a.dv > 256) FAIL(HYMBA_ERR_UNSUPPORTED, "dv %d: a multiple of 8 up to 256", a.dv);
  if (a.batch > 65535 || a.n_heads > 65535) FAIL(HYMBA_ERR_UNSUPPORTED, "more than 65535 sequences or heads");
  if (a.n_rows > (1 << 30)) FAIL(HYMBA_ERR_UNSUPPORTED, "sequence too long");
  if (!std::isfinite(a.scale)) FAIL(HYMBA_ERR_INVALID_ARG, "scale is not finite");
  return HYMBA_OK;
}

hymba_status check_repeated(const char *name, const void *p, long long sb, long long sr, long long sh) {
  if (p && (reinterpret_cast<uintptr_t>(p) & 3u)) FAIL(HYMBA_ERR_INVALID_ARG, "%s misaligned", name);
  if (p && (sb < 0 || sr < 0 || sh < 0)) FAIL(HYMBA_ERR_INVALID_ARG, "%s: negative stride", name);
  return HYMBA_OK;
}

hymba_status check_linear(const hymba_linear_attention &a) {
  hymba_status st = check_linear_sizes(a);
  if (st != HYMBA_OK) return st;
  const long long es = esize(a.dtype);
  const LinearGrids g = linear_grids(a);
  if ((st = check_grid("q", a.q, g.q, es)) != HYMBA_OK) return st;
  if ((st = check_grid("k", a.k, g.k, es)) != HYMBA_OK) return st;
  if ((st = check_grid("v", a.v, g.v, es)) != HYMBA_OK) return st;
  if ((st = check_grid("o", a.o, g.o, es)) != HYMBA_OK) return st;
  if ((st = check_written("o", g.o)) != HYMBA_OK) return st;
  if (a.gate && (st = check_grid("gate", a.gate, g.z, es)) != HYMBA_OK) return st;
  if (a.o == a.q || a.o == a.k || a.o == a.v || a.o == a.gate) FAIL(HYMBA_ERR_INVALID_ARG, "o is one of the inputs");
  if ((st = check_repeated("log_decay", a.log_decay, a.decay_batch, a.decay_row, a.decay_head)) != HYMBA_OK) return st;
  if ((st = check_repeated("in_scale", a.in_scale, a.scale_batch, a.scale_row, a.scale_head)) != HYMBA_OK) return st;
  if (a.skip && !aligned16(a.skip)) FAIL(HYMBA_ERR_INVALID_ARG, "skip not 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(a.lengths) & 3u) FAIL(HYMBA_ERR_INVALID_ARG, "lengths misaligned");
  const long long one = (long long)a.n_heads * a.dv * a.dk;
  if (a.state_in) {
    if (!aligned16(a.state_in) || a.state_in_batch % 4) FAIL(HYMBA_ERR_INVALID_ARG, "state_in not 16-byte aligned");
    if (a.batch > 1 && a.state_in_batch != 0 && a.state_in_batch < one)
      FAIL(HYMBA_ERR_INVALID_ARG, "state_in_batch %lld: 0 or at least %lld", (long long)a.state_in_batch, one);
  }
  if (a.state_out && !aligned16(a.state_out)) FAIL(HYMBA_ERR_INVALID_ARG, "state_out not 16-byte aligned");
  if (a.state_in && a.state_out) {
    const bool in_place = a.state_in == a.state_out && (a.batch == 1 || a.state_in_batch == one);
    const long long in_n = (a.batch - 1) * (a.batch > 1 ? a.state_in_batch : 0) + one;
    if (!in_place && ranges_overlap(a.state_in, 4 * in_n, a.state_out, 4 * one * a.batch))
      FAIL(HYMBA_ERR_INVALID_ARG, "state_in and state_out overlap without being the same states");
  }
  return HYMBA_OK;
}

}  // namespace

extern "C" {

hymba_status hymba_qk_norm_rope(const hymba_qk_norm_rope_args *args, hymba_stream_t stream_) {
  set_error("%s", "");
  if (!args) FAIL(HYMBA_ERR_INVALID_ARG, "null arguments");
  const hymba_qk_norm_rope_args &a = *args;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (bad_dtype(a.dtype)) FAIL(HYMBA_ERR_INVALID_ARG, "dtype %d", a.dtype);
  if (a.batch < 1 || a.n_rows < 1) FAIL(HYMBA_ERR_INVALID_ARG, "batch and n_rows must be positive");
  if (a.head_dim < 8 || a.head_dim % 8 || a.head_dim > 256)
    FAIL(HYMBA_ERR_UNSUPPORTED, "head_dim %d: a multiple of 8 up to 256", a.head_dim);
  if (a.q.n_heads < 1 && a.k.n_heads < 1) FAIL(HYMBA_ERR_INVALID_ARG, "neither query nor key heads");
  hymba_status st;
  if ((st = check_heads("q", a, a.q)) != HYMBA_OK) return st;
  if ((st = check_heads("k", a, a.k)) != HYMBA_OK) return st;
  if ((long long)a.q.n_heads + a.k.n_heads > (1 << 20)) FAIL(HYMBA_ERR_UNSUPPORTED, "too many heads");
  if (a.norm && (!(a.eps >= 0.f) || !std::isfinite(a.eps))) FAIL(HYMBA_ERR_INVALID_ARG, "eps < 0");
  if ((st = check_rope(a.rope, a.head_dim)) != HYMBA_OK) return st;
  if (a.positions && (reinterpret_cast<uintptr_t>(a.positions) & 7u)) FAIL(HYMBA_ERR_INVALID_ARG, "positions misaligned");
  ProfScope prof_scope(stream, "qk_norm_rope");
  return qk_norm_rope(a, stream);
}

hymba_status hymba_linear_attention_workspace(const hymba_linear_attention *args, size_t *bytes) {
  set_error("%s", "");
  if (!args || !bytes) FAIL(HYMBA_ERR_INVALID_ARG, "null argument");
  const hymba_status st = check_linear_sizes(*args);
  if (st != HYMBA_OK) return st;
  *bytes = linear_attention_workspace_bytes(*args);
  return HYMBA_OK;
}

hymba_status hymba_linear_attention_prefill(const hymba_linear_attention *args, void *workspace,
                                            size_t workspace_bytes, hymba_stream_t stream_) {
  set_error("%s", "");
  if (!args) FAIL(HYMBA_ERR_INVALID_ARG, "null arguments");
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const hymba_status st = check_linear(*args);
  if (st != HYMBA_OK) return st;
  const size_t need = linear_attention_workspace_bytes(*args);
  if (need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)))
    FAIL(HYMBA_ERR_INVALID_ARG, "workspace null or not 256-byte aligned");
  if (workspace_bytes < need) FAIL(HYMBA_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);
  ProfScope prof_scope(stream, "linear_attention");
  return linear_attention(*args, workspace, stream);
}

hymba_status hymba_linear_attention_decode_step(const hymba_linear_attention *args, hymba_stream_t stream_) {
  set_error("%s", "");
  if (!args) FAIL(HYMBA_ERR_INVALID_ARG, "null arguments");
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const hymba_status st = check_linear(*args);
  if (st != HYMBA_OK) return st;
  if (args->n_rows != 1) FAIL(HYMBA_ERR_INVALID_ARG, "a decode step takes one row per sequence, not %d", args->n_rows);
  if (!args->state_out) FAIL(HYMBA_ERR_INVALID_ARG, "a decode step needs state_out");
  ProfScope prof_scope(stream, "linear_step");
  return linear_attention_step(*args, stream);
}

}  // extern "C"
