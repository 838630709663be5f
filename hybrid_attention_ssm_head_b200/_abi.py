"""ctypes binding of the C ABI in include/hymba.h (argument marshalling only).

Every function of the header is exposed under its own name.  Loading fails
loudly when libhymba.so is missing: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes as C
import os
import sys

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhymba.so")

HYMBA_OK = 0
HYMBA_ERR_INVALID_ARG = 1
HYMBA_ERR_UNSUPPORTED = 2
HYMBA_ERR_WORKSPACE = 3
HYMBA_ERR_NOT_BOUND = 4
HYMBA_ERR_CUDA = 5
HYMBA_ERR_TIMEOUT = 6
HYMBA_ERR_DEVICE = 7
HYMBA_F32 = 0
HYMBA_BF16 = 1
HYMBA_ROPE_PAIRS = 0
HYMBA_ROPE_HALVES = 1
HYMBA_ROPE_SCALE_NONE = 0
HYMBA_ROPE_SCALE_LINEAR = 1
HYMBA_ROPE_SCALE_WAVELENGTH = 2


class hymba_layer_config(C.Structure):
    _fields_ = [("d_model", C.c_int), ("n_heads", C.c_int), ("n_kv_heads", C.c_int),
                ("head_dim_qk", C.c_int), ("head_dim_v", C.c_int), ("d_inner", C.c_int),
                ("d_state", C.c_int), ("d_conv", C.c_int), ("dt_rank", C.c_int),
                ("n_meta", C.c_int), ("window", C.c_int), ("is_global", C.c_int),
                ("dtype", C.c_int), ("rms_eps", C.c_float), ("softmax_scale", C.c_float),
                ("rope_base", C.c_float), ("branch_chunks", C.c_int)]


class hymba_layer_weights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("w_in", "conv_w", "conv_b", "w_x", "w_dt", "b_dt",
                                          "a_log", "d_skip", "beta_attn", "beta_ssm", "w_out")]


class hymba_kv_seq(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("batch", C.c_int), ("rows", C.c_int),
                ("owner", C.c_uint64)]


class hymba_kv_cache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("batch", C.c_int), ("capacity", C.c_int),
                ("owner", C.c_uint64)]


class hymba_ssm_cache(C.Structure):
    _fields_ = [("h", C.c_void_p), ("conv", C.c_void_p)]


class hymba_meta_cache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("h", C.c_void_p), ("conv", C.c_void_p),
                ("y", C.c_void_p), ("owner", C.c_uint64)]


class hymba_block_weights(C.Structure):
    _fields_ = [("norm1", C.c_void_p), ("norm2", C.c_void_p), ("w_gate_up", C.c_void_p),
                ("w_down", C.c_void_p), ("mlp_hidden", C.c_int)]


class hymba_prefill_layout(C.Structure):
    _fields_ = [(n, C.c_size_t) for n in ("q", "x_ssm", "gate", "u", "xdbl", "delta", "y_ssm",
                                          "o_attn", "fused", "rope", "sched", "total")]


class hymba_rope(C.Structure):
    _fields_ = [("dim", C.c_int), ("layout", C.c_int), ("scaling", C.c_int), ("attn_factor", C.c_float),
                ("base", C.c_double), ("factor", C.c_double), ("orig_len", C.c_double),
                ("low_turns", C.c_double), ("high_turns", C.c_double)]


class hymba_head_rows(C.Structure):
    _fields_ = [("in_", C.c_void_p), ("out", C.c_void_p), ("weight", C.c_void_p),
                ("in_batch", C.c_int64), ("in_row", C.c_int64), ("in_head", C.c_int64),
                ("out_batch", C.c_int64), ("out_row", C.c_int64), ("out_head", C.c_int64),
                ("n_heads", C.c_int)]


class _Description(C.Structure):
    device = None         # of the tensors a maker took the addresses of
    check_device = False  # whether a call has to look at it


class hymba_qk_norm_rope_args(_Description):
    _fields_ = [("dtype", C.c_int), ("batch", C.c_int), ("n_rows", C.c_int), ("head_dim", C.c_int),
                ("q", hymba_head_rows), ("k", hymba_head_rows), ("norm", C.c_int), ("eps", C.c_float),
                ("rope", hymba_rope), ("pos0", C.c_int64), ("positions", C.c_void_p)]


class hymba_linear_attention(_Description):
    _fields_ = ([(n, C.c_int) for n in ("dtype", "batch", "n_rows", "n_heads", "n_qk_heads", "dk", "dv")] +
                [("scale", C.c_float)] +
                [f for n, s in (("q", "q"), ("k", "k"), ("v", "v"), ("o", "o"), ("gate", "gate"),
                                ("log_decay", "decay"), ("in_scale", "scale"))
                 for f in [(n, C.c_void_p)] + [(f"{s}_{x}", C.c_int64) for x in ("batch", "row", "head")]] +
                [("skip", C.c_void_p), ("state_in", C.c_void_p), ("state_in_batch", C.c_int64),
                 ("state_out", C.c_void_p), ("lengths", C.c_void_p)])


class hymba_layer_heads(C.Structure):
    _fields_ = [("norm", C.c_int), ("eps", C.c_float), ("q_weight", C.c_void_p), ("k_weight", C.c_void_p),
                ("rope", hymba_rope)]


class hymba_linear_heads(C.Structure):
    _fields_ = [("d_state", C.c_int), ("w_x", C.c_void_p), ("b_dt", C.c_void_p), ("a_log", C.c_void_p),
                ("d_skip", C.c_void_p)]


class hymba_profile_entry(C.Structure):
    _fields_ = [("name", C.c_char * 32), ("calls", C.c_int), ("kernels", C.c_int),
                ("total_ms", C.c_double)]


class HymbaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


_lib = None

# name -> (restype, argtypes)
_SIGS = {
    "hymba_layer_create": (C.c_int, [C.POINTER(hymba_layer_config), C.POINTER(hymba_layer_weights),
                                     C.POINTER(C.c_void_p)]),
    "hymba_layer_destroy": (None, [C.c_void_p]),
    "hymba_layer_is_consumer": (C.c_int, [C.c_void_p]),
    "hymba_kv_share_bind": (C.c_int, [C.c_void_p, C.c_void_p]),
    "hymba_layer_prefill_workspace": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.POINTER(C.c_size_t)]),
    "hymba_layer_prefill_layout": (C.c_int, [C.c_void_p, C.c_int, C.c_int,
                                             C.POINTER(hymba_prefill_layout)]),
    "hymba_layer_prefill": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_void_p,
                                      C.POINTER(hymba_kv_seq), C.POINTER(hymba_kv_cache),
                                      C.POINTER(hymba_ssm_cache), C.c_void_p, C.c_size_t, C.c_void_p]),
    "hymba_layer_meta_workspace": (C.c_int, [C.c_void_p, C.POINTER(C.c_size_t)]),
    "hymba_layer_meta_precompute": (C.c_int, [C.c_void_p, C.c_void_p, C.POINTER(hymba_meta_cache),
                                              C.POINTER(hymba_meta_cache), C.c_void_p, C.c_size_t,
                                              C.c_void_p]),
    "hymba_layer_prefill_cached_workspace": (C.c_int, [C.c_void_p, C.c_int, C.c_int,
                                                       C.POINTER(C.c_size_t)]),
    "hymba_layer_prefill_cached": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_void_p,
                                             C.POINTER(hymba_meta_cache), C.POINTER(hymba_kv_seq),
                                             C.POINTER(hymba_kv_cache), C.POINTER(hymba_ssm_cache),
                                             C.c_void_p, C.c_size_t, C.c_void_p]),
    "hymba_block_prefill_workspace": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int, C.POINTER(C.c_size_t)]),
    "hymba_block_prefill": (C.c_int, [C.c_void_p, C.POINTER(hymba_block_weights), C.c_int, C.c_int,
                                      C.c_void_p, C.c_void_p, C.POINTER(hymba_kv_seq),
                                      C.POINTER(hymba_kv_cache), C.POINTER(hymba_ssm_cache), C.c_void_p,
                                      C.c_size_t, C.c_void_p]),
    "hymba_block_decode_workspace": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int64, C.POINTER(C.c_size_t)]),
    "hymba_block_decode_step": (C.c_int, [C.c_void_p, C.POINTER(hymba_block_weights), C.c_int, C.c_int64,
                                          C.c_void_p, C.c_void_p, C.POINTER(hymba_kv_cache),
                                          C.POINTER(hymba_ssm_cache), C.c_void_p, C.c_size_t, C.c_void_p]),
    "hymba_layer_decode_workspace": (C.c_int, [C.c_void_p, C.c_int, C.c_int64, C.POINTER(C.c_size_t)]),
    "hymba_layer_decode_step": (C.c_int, [C.c_void_p, C.c_int, C.c_int64, C.c_void_p, C.c_void_p,
                                          C.POINTER(hymba_kv_cache), C.POINTER(hymba_ssm_cache),
                                          C.c_void_p, C.c_size_t, C.c_void_p]),
    "hymba_layer_set_heads": (C.c_int, [C.c_void_p, C.POINTER(hymba_layer_heads)]),
    "hymba_layer_set_linear_heads": (C.c_int, [C.c_void_p, C.POINTER(hymba_linear_heads)]),
    "hymba_qk_norm_rope": (C.c_int, [C.POINTER(hymba_qk_norm_rope_args), C.c_void_p]),
    "hymba_linear_attention_workspace": (C.c_int, [C.POINTER(hymba_linear_attention), C.POINTER(C.c_size_t)]),
    "hymba_linear_attention_prefill": (C.c_int, [C.POINTER(hymba_linear_attention), C.c_void_p, C.c_size_t,
                                                 C.c_void_p]),
    "hymba_linear_attention_decode_step": (C.c_int, [C.POINTER(hymba_linear_attention), C.c_void_p]),
    "hymba_stream_status": (C.c_int, [C.c_void_p]),
    "hymba_last_error": (C.c_char_p, []),
    "hymba_status_string": (C.c_char_p, [C.c_int]),
    "hymba_version": (C.c_char_p, []),
    "hymba_debug_mask_bitmap": (C.c_int, [C.c_int, C.c_int, C.c_int, C.c_int, C.c_int, C.c_void_p,
                                          C.c_void_p, C.c_void_p]),
    "hymba_debug_decode_mask": (C.c_int, [C.c_int64, C.c_int, C.c_int, C.c_int, C.c_int, C.c_void_p,
                                          C.c_void_p]),
    "hymba_debug_exp2_poly": (C.c_int, [C.c_int, C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p]),
    "hymba_layer_decode_step_static": (C.c_int, [C.c_void_p, C.c_int, C.c_int64, C.c_void_p, C.c_void_p,
                                                 C.POINTER(hymba_kv_cache), C.POINTER(hymba_ssm_cache),
                                                 C.c_void_p]),
    "hymba_set_wait_limit": (C.c_int, [C.c_int64, C.POINTER(C.c_int64)]),
    "hymba_debug_stall_next_prefill": (C.c_int, [C.c_int]),
    "hymba_profile_enable": (C.c_int, [C.c_int]),
    "hymba_profile_collect": (C.c_int, [C.POINTER(hymba_profile_entry), C.c_int, C.POINTER(C.c_int)]),
}
EXPORTED = tuple(_SIGS)


def lib():
    """The loaded libhymba.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m hybrid_attention_ssm_head_b200.build`")
        lib_ = C.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib_, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib_
    return _lib


def check(status: int, what: str = "") -> None:
    if status != HYMBA_OK:
        msg = lib().hymba_last_error().decode()
        name = lib().hymba_status_string(status).decode()
        raise HymbaError(status, f"{what}: {name}: {msg}")


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s) -> int | None:
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


# ---- the entry points, same names as the header ------------------------------------------

def hymba_layer_create(cfg: hymba_layer_config, w: hymba_layer_weights) -> int:
    out = C.c_void_p()
    check(lib().hymba_layer_create(C.byref(cfg), C.byref(w), C.byref(out)), "hymba_layer_create")
    return out.value


def hymba_layer_destroy(layer: int) -> None:
    lib().hymba_layer_destroy(layer)


def hymba_layer_is_consumer(layer: int) -> bool:
    return bool(lib().hymba_layer_is_consumer(layer))


def hymba_kv_share_bind(consumer: int, producer: int) -> None:
    check(lib().hymba_kv_share_bind(consumer, producer), "hymba_kv_share_bind")


def hymba_layer_prefill_workspace(layer: int, batch: int, n_tokens: int) -> int:
    out = C.c_size_t()
    check(lib().hymba_layer_prefill_workspace(layer, batch, n_tokens, C.byref(out)),
          "hymba_layer_prefill_workspace")
    return out.value


def hymba_layer_prefill_layout(layer: int, batch: int, n_tokens: int) -> hymba_prefill_layout:
    out = hymba_prefill_layout()
    check(lib().hymba_layer_prefill_layout(layer, batch, n_tokens, C.byref(out)),
          "hymba_layer_prefill_layout")
    return out


def hymba_layer_prefill(layer: int, batch: int, n_tokens: int, x, y, kv: hymba_kv_seq,
                        kv_cache: hymba_kv_cache | None, ssm_cache: hymba_ssm_cache | None,
                        workspace, workspace_bytes: int, stream=None) -> None:
    check(lib().hymba_layer_prefill(
        layer, batch, n_tokens, _ptr(x), _ptr(y), C.byref(kv),
        C.byref(kv_cache) if kv_cache is not None else None,
        C.byref(ssm_cache) if ssm_cache is not None else None,
        _ptr(workspace), workspace_bytes, _stream(stream)), "hymba_layer_prefill")


def hymba_layer_meta_workspace(layer: int) -> int:
    out = C.c_size_t()
    check(lib().hymba_layer_meta_workspace(layer, C.byref(out)), "hymba_layer_meta_workspace")
    return out.value


def hymba_layer_meta_precompute(layer: int, x_meta, meta: hymba_meta_cache,
                                producer_meta: hymba_meta_cache | None, workspace, workspace_bytes: int,
                                stream=None) -> None:
    check(lib().hymba_layer_meta_precompute(
        layer, _ptr(x_meta), C.byref(meta), C.byref(producer_meta) if producer_meta is not None else None,
        _ptr(workspace), workspace_bytes, _stream(stream)), "hymba_layer_meta_precompute")


def hymba_layer_prefill_cached_workspace(layer: int, batch: int, n_tokens: int) -> int:
    out = C.c_size_t()
    check(lib().hymba_layer_prefill_cached_workspace(layer, batch, n_tokens, C.byref(out)),
          "hymba_layer_prefill_cached_workspace")
    return out.value


def hymba_layer_prefill_cached(layer: int, batch: int, n_tokens: int, x, y, meta: hymba_meta_cache,
                               kv: hymba_kv_seq, kv_cache: hymba_kv_cache | None,
                               ssm_cache: hymba_ssm_cache | None, workspace, workspace_bytes: int,
                               stream=None) -> None:
    check(lib().hymba_layer_prefill_cached(
        layer, batch, n_tokens, _ptr(x), _ptr(y), C.byref(meta), C.byref(kv),
        C.byref(kv_cache) if kv_cache is not None else None,
        C.byref(ssm_cache) if ssm_cache is not None else None,
        _ptr(workspace), workspace_bytes, _stream(stream)), "hymba_layer_prefill_cached")


def make_block_weights(w: dict) -> hymba_block_weights:
    """From device tensors norm1, norm2 [d] fp32, w_gate_up [2F, d] (rows interleaved), w_down [d, F]."""
    return hymba_block_weights(_ptr(w["norm1"]), _ptr(w["norm2"]), _ptr(w["w_gate_up"]), _ptr(w["w_down"]),
                               int(w["w_down"].shape[1]))


def hymba_block_prefill_workspace(layer: int, mlp_hidden: int, batch: int, n_tokens: int) -> int:
    out = C.c_size_t()
    check(lib().hymba_block_prefill_workspace(layer, mlp_hidden, batch, n_tokens, C.byref(out)),
          "hymba_block_prefill_workspace")
    return out.value


def hymba_block_prefill(layer: int, bw: hymba_block_weights, batch: int, n_tokens: int, x, y, kv: hymba_kv_seq,
                        kv_cache: hymba_kv_cache | None, ssm_cache: hymba_ssm_cache | None, workspace,
                        workspace_bytes: int, stream=None) -> None:
    check(lib().hymba_block_prefill(
        layer, C.byref(bw), batch, n_tokens, _ptr(x), _ptr(y), C.byref(kv),
        C.byref(kv_cache) if kv_cache is not None else None,
        C.byref(ssm_cache) if ssm_cache is not None else None,
        _ptr(workspace), workspace_bytes, _stream(stream)), "hymba_block_prefill")


def hymba_block_decode_workspace(layer: int, mlp_hidden: int, batch: int, max_pos: int) -> int:
    out = C.c_size_t()
    check(lib().hymba_block_decode_workspace(layer, mlp_hidden, batch, max_pos, C.byref(out)),
          "hymba_block_decode_workspace")
    return out.value


def hymba_block_decode_step(layer: int, bw: hymba_block_weights, batch: int, pos: int, x_t, y_t,
                            kv_cache: hymba_kv_cache, ssm_cache: hymba_ssm_cache, workspace, workspace_bytes: int,
                            stream=None) -> None:
    check(lib().hymba_block_decode_step(layer, C.byref(bw), batch, pos, _ptr(x_t), _ptr(y_t), C.byref(kv_cache),
                                        C.byref(ssm_cache), _ptr(workspace), workspace_bytes, _stream(stream)),
          "hymba_block_decode_step")


def hymba_layer_decode_workspace(layer: int, batch: int, max_pos: int) -> int:
    out = C.c_size_t()
    check(lib().hymba_layer_decode_workspace(layer, batch, max_pos, C.byref(out)),
          "hymba_layer_decode_workspace")
    return out.value


def hymba_layer_decode_step(layer: int, batch: int, pos: int, x_t, y_t, kv_cache: hymba_kv_cache,
                            ssm_cache: hymba_ssm_cache, workspace, workspace_bytes: int,
                            stream=None) -> None:
    check(lib().hymba_layer_decode_step(layer, batch, pos, _ptr(x_t), _ptr(y_t), C.byref(kv_cache),
                                        C.byref(ssm_cache), _ptr(workspace), workspace_bytes,
                                        _stream(stream)), "hymba_layer_decode_step")


HYMBA_DECODE_STATIC_SCRATCH_BYTES = 40 << 20


def hymba_layer_decode_step_static(layer: int, batch: int, pos: int, x_t, y_t,
                                   kv_cache: hymba_kv_cache, ssm_cache: hymba_ssm_cache,
                                   stream=None) -> None:
    """hymba_layer_decode_step with the library's static scratch instead of a workspace."""
    check(lib().hymba_layer_decode_step_static(layer, batch, pos, _ptr(x_t), _ptr(y_t),
                                               C.byref(kv_cache), C.byref(ssm_cache),
                                               _stream(stream)), "hymba_layer_decode_step_static")


def hymba_layer_set_heads(layer: int, heads: hymba_layer_heads | None) -> None:
    check(lib().hymba_layer_set_heads(layer, C.byref(heads) if heads is not None else None), "hymba_layer_set_heads")


def hymba_layer_set_linear_heads(layer: int, heads: hymba_linear_heads | None) -> None:
    check(lib().hymba_layer_set_linear_heads(layer, C.byref(heads) if heads is not None else None),
          "hymba_layer_set_linear_heads")


def _launchable(args, what: str, workspace=None) -> None:
    """A description made from tensors runs on their GPU, which has to be the current device.  (One
    filled in by hand carries no device: its addresses are the caller's.)"""
    dev = args.device
    if dev is not None and dev.type != "cuda":
        raise ValueError(f"{what}: the tensors are on {dev}, not on a GPU")
    if dev is not None and dev.index != sys.modules["torch"].cuda.current_device():
        raise ValueError(f"{what}: the tensors are on {dev}, which is not the current device")
    on = getattr(workspace, "device", dev)
    if on is not None and (on.type != "cuda" or (dev is not None and on != dev)):
        raise ValueError(f"{what}: the workspace is on {on}, the tensors on {dev}")


def hymba_qk_norm_rope(args: hymba_qk_norm_rope_args, stream=None) -> None:
    if args.check_device:
        _launchable(args, "hymba_qk_norm_rope")
    check(lib().hymba_qk_norm_rope(C.byref(args), _stream(stream)), "hymba_qk_norm_rope")


def hymba_linear_attention_workspace(args: hymba_linear_attention) -> int:
    out = C.c_size_t()
    check(lib().hymba_linear_attention_workspace(C.byref(args), C.byref(out)), "hymba_linear_attention_workspace")
    return out.value


def hymba_linear_attention_prefill(args: hymba_linear_attention, workspace, workspace_bytes: int,
                                   stream=None) -> None:
    if args.check_device or not getattr(workspace, "is_cuda", True):
        _launchable(args, "hymba_linear_attention_prefill", workspace)
    check(lib().hymba_linear_attention_prefill(C.byref(args), _ptr(workspace), workspace_bytes, _stream(stream)),
          "hymba_linear_attention_prefill")


def hymba_linear_attention_decode_step(args: hymba_linear_attention, stream=None) -> None:
    if args.check_device:
        _launchable(args, "hymba_linear_attention_decode_step")
    check(lib().hymba_linear_attention_decode_step(C.byref(args), _stream(stream)),
          "hymba_linear_attention_decode_step")


def hymba_stream_status(stream=None) -> None:
    check(lib().hymba_stream_status(_stream(stream)), "hymba_stream_status")


def hymba_last_error() -> str:
    return lib().hymba_last_error().decode()


def hymba_status_string(s: int) -> str:
    return lib().hymba_status_string(s).decode()


def hymba_version() -> str:
    return lib().hymba_version().decode()


def hymba_debug_mask_bitmap(L: int, n_meta: int, window: int, is_global: bool, bits,
                            tile_class=None, stream=None, path: int = 0) -> None:
    check(lib().hymba_debug_mask_bitmap(L, n_meta, window, int(is_global), path, _ptr(bits),
                                        _ptr(tile_class), _stream(stream)), "hymba_debug_mask_bitmap")


def hymba_debug_decode_mask(pos: int, n_meta: int, window: int, is_global: bool, capacity: int, bits,
                            stream=None) -> None:
    check(lib().hymba_debug_decode_mask(pos, n_meta, window, int(is_global), capacity, _ptr(bits),
                                        _stream(stream)), "hymba_debug_decode_mask")


def hymba_debug_exp2_poly(degree: int, x, y, n: int, stream=None) -> None:
    check(lib().hymba_debug_exp2_poly(degree, _ptr(x), _ptr(y), n, _stream(stream)),
          "hymba_debug_exp2_poly")


def hymba_set_wait_limit(cycles: int) -> int:
    """Sets the bounded-wait limit (0: default); returns the limit now in force."""
    out = C.c_int64()
    check(lib().hymba_set_wait_limit(cycles, C.byref(out)), "hymba_set_wait_limit")
    return out.value


def hymba_debug_stall_next_prefill(count: int) -> None:
    check(lib().hymba_debug_stall_next_prefill(count), "hymba_debug_stall_next_prefill")


def hymba_profile_enable(on: bool) -> None:
    check(lib().hymba_profile_enable(int(bool(on))), "hymba_profile_enable")


def hymba_profile_collect(max_entries: int = 64) -> list[tuple[str, int, int, float]]:
    """[(step name, calls, kernels launched, total ms)] since the last collect."""
    buf = (hymba_profile_entry * max_entries)()
    n = C.c_int()
    check(lib().hymba_profile_collect(buf, max_entries, C.byref(n)), "hymba_profile_collect")
    return [(buf[i].name.decode(), buf[i].calls, buf[i].kernels, buf[i].total_ms)
            for i in range(n.value)]


# ---- marshalling helpers ---------------------------------------------------------------

def make_config(d_model, n_heads, n_kv_heads, head_dim_qk, d_inner, d_state, d_conv, dt_rank,
                n_meta, window, is_global, dtype: str, rms_eps=1e-6, softmax_scale=0.0, rope_base=0.0,
                branch_chunks=4):
    """branch_chunks: batch chunks of the concurrent prefill (0 or 1: serial order)."""
    return hymba_layer_config(d_model, n_heads, n_kv_heads, head_dim_qk, d_inner // n_heads, d_inner,
                              d_state, d_conv, dt_rank, n_meta, window if not is_global else 0,
                              int(bool(is_global)), HYMBA_BF16 if dtype == "bf16" else HYMBA_F32,
                              rms_eps, softmax_scale, rope_base, branch_chunks)


def make_weights(w: dict) -> hymba_layer_weights:
    """From a dict of contiguous device tensors (keys as in the header)."""
    for k, t in w.items():
        if not t.is_contiguous():
            raise ValueError(f"weight {k} must be contiguous")
    return hymba_layer_weights(*[_ptr(w[n]) for n, _ in hymba_layer_weights._fields_])


def _dtype_of(t) -> int:
    name = str(t.dtype)
    if name not in ("torch.bfloat16", "torch.float32"):
        raise ValueError(f"storage dtype must be bfloat16 or float32, not {name}")
    return HYMBA_BF16 if name == "torch.bfloat16" else HYMBA_F32


def _set_device(args: _Description, **tensors) -> None:
    """The device all of them are on.  It is looked at again at each call, unless there is but one GPU."""
    on = {n: t.device for n, t in tensors.items() if t is not None}
    if len(set(on.values())) > 1:
        raise ValueError("tensors on different devices: " + ", ".join(f"{n} on {d}" for n, d in on.items()))
    args.device = next(iter(on.values()))
    args.check_device = args.device.type != "cuda" or sys.modules["torch"].cuda.device_count() > 1


def _rows(name: str, t, shape, dtype: str) -> list[int]:
    """[pointer, batch, row and head stride] of a [batch, rows, heads(, dim)] tensor; checks what
    the library cannot see: shape, dtype and a contiguous last dimension."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if str(t.dtype) != dtype:
        raise ValueError(f"{name}: {t.dtype}, expected {dtype}")
    if t.ndim == 4 and shape[3] > 1 and t.stride(3) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return [t.data_ptr(), *t.stride()[:3]]


def _dense(name: str, t, shape, dtype: str) -> int | None:
    if t is None:
        return None
    if tuple(t.shape) != tuple(shape) or str(t.dtype) != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype}, expected contiguous {tuple(shape)} {dtype}")
    return t.data_ptr()


def make_rope(dim: int, layout: str = "pairs", base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
              orig_len: float = 0.0, low_turns: float = 0.0, high_turns: float = 0.0,
              attn_factor: float = 1.0) -> hymba_rope:
    """layout "pairs" or "halves"; scaling "none", "linear" or "wavelength"."""
    return hymba_rope(dim, {"pairs": HYMBA_ROPE_PAIRS, "halves": HYMBA_ROPE_HALVES}[layout],
                      {"none": HYMBA_ROPE_SCALE_NONE, "linear": HYMBA_ROPE_SCALE_LINEAR,
                       "wavelength": HYMBA_ROPE_SCALE_WAVELENGTH}[scaling],
                      attn_factor, base, factor, orig_len, low_turns, high_turns)


def make_qk_norm_rope(q, k, q_out=None, k_out=None, norm: bool = True, eps: float = 1e-6, q_weight=None,
                      k_weight=None, rope: hymba_rope | None = None, pos0: int = 0,
                      positions=None) -> hymba_qk_norm_rope_args:
    """q [batch, rows, heads, dim], k [batch, rows, kv_heads, dim] or None: device tensors of any
    strides with a contiguous head; q_out, k_out likewise (None: in place).  All on one device.  The
    description holds addresses only: the tensors must outlive its use."""
    some = q if q is not None else k
    B, R, _, d = some.shape
    a = hymba_qk_norm_rope_args(dtype=_dtype_of(some), batch=B, n_rows=R, head_dim=d, norm=int(norm), eps=eps,
                                pos0=pos0)
    for side, x, out, w in (("q", q, q_out, q_weight), ("k", k, k_out, k_weight)):
        if x is None:
            continue
        shape = (B, R, x.shape[2], d)
        i = _rows(side, x, shape, str(some.dtype))
        o = _rows(side + "_out", x if out is None else out, shape, str(some.dtype))
        setattr(a, side, hymba_head_rows(i[0], o[0], _dense(side + "_weight", w, (d,), "torch.float32"), *i[1:], *o[1:],
                                         x.shape[2]))
    if rope is not None:
        a.rope = rope
    _set_device(a, q=q, k=k, q_out=q_out, k_out=k_out, q_weight=q_weight, k_weight=k_weight, positions=positions)
    a.positions = _dense("positions", positions, (B, R), "torch.int64")
    return a


def make_linear_attention(q, k, v, o, log_decay=None, in_scale=None, skip=None, gate=None, state_in=None,
                          state_out=None, lengths=None, scale: float = 1.0) -> hymba_linear_attention:
    """q, k [batch, rows, qk_heads, dk], v, o, gate [batch, rows, heads, dv]: device tensors of any
    strides with a contiguous head; log_decay, in_scale [batch, rows, heads] fp32 of any strides
    (expand() repeats a value); skip [heads, dv]; state_in [batch, heads, dv, dk] dense per sequence
    (expand() over the batch repeats one); state_out likewise, dense; lengths [batch] int32.  All on one
    device.  The description holds addresses only: the tensors must outlive its use."""
    B, L, K, dk = q.shape
    H, dv = v.shape[2], v.shape[3]
    dt = str(q.dtype)
    a = hymba_linear_attention(dtype=_dtype_of(q), batch=B, n_rows=L, n_heads=H, n_qk_heads=K, dk=dk, dv=dv,
                               scale=scale)
    grids = (("q", "q", q, (B, L, K, dk), dt), ("k", "k", k, (B, L, K, dk), dt), ("v", "v", v, (B, L, H, dv), dt),
             ("o", "o", o, (B, L, H, dv), dt), ("gate", "gate", gate, (B, L, H, dv), dt),
             ("log_decay", "decay", log_decay, (B, L, H), "torch.float32"),
             ("in_scale", "scale", in_scale, (B, L, H), "torch.float32"))
    for name, stride, t, shape, want in grids:
        if t is not None:
            p, sb, sr, sh = _rows(name, t, shape, want)
            setattr(a, name, p)
            setattr(a, stride + "_batch", sb)
            setattr(a, stride + "_row", sr)
            setattr(a, stride + "_head", sh)
    _set_device(a, q=q, k=k, v=v, o=o, log_decay=log_decay, in_scale=in_scale, skip=skip, gate=gate,
                state_in=state_in, state_out=state_out, lengths=lengths)
    a.skip = _dense("skip", skip, (H, dv), "torch.float32")
    if state_in is not None:
        if tuple(state_in.shape) != (B, H, dv, dk):
            raise ValueError(f"state_in: shape {tuple(state_in.shape)}, expected {(B, H, dv, dk)}")
        a.state_in = _dense("state_in[0]", state_in[0], (H, dv, dk), "torch.float32")
        a.state_in_batch = state_in.stride(0)
    a.state_out = _dense("state_out", state_out, (B, H, dv, dk), "torch.float32")
    a.lengths = _dense("lengths", lengths, (B,), "torch.int32")
    return a


def _weight(name: str, t, dtype: str | None = None, shape=None) -> int | None:
    """Address of a weight.  A tensor has to be contiguous and, where given, of this dtype and shape."""
    if t is None or isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError(f"weight {name} must be contiguous")
    if (dtype and str(t.dtype) != dtype) or (shape and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"weight {name}: {tuple(t.shape)} {t.dtype}, expected {shape or 'any shape'} {dtype or ''}")
    return t.data_ptr()


def make_layer_heads(norm: bool = True, eps: float = 1e-6, q_weight=None, k_weight=None,
                     rope: hymba_rope | None = None) -> hymba_layer_heads:
    """q_weight, k_weight [head_dim_qk] fp32 device tensors or None."""
    return hymba_layer_heads(int(norm), eps, _weight("q_weight", q_weight, "torch.float32"),
                             _weight("k_weight", k_weight, "torch.float32"), rope if rope is not None else hymba_rope())


def make_linear_heads(w: dict, d_state: int) -> hymba_linear_heads:
    """From device tensors w_x [2 * d_state + n_heads, d_inner] of the layer's dtype, and fp32 b_dt and
    a_log [n_heads], d_skip [d_inner]."""
    b, x = w["b_dt"], w["w_x"]
    heads = tuple(b.shape) if hasattr(b, "shape") else None
    wide = hasattr(x, "shape")
    if wide and (x.ndim != 2 or (heads and x.shape[0] != 2 * d_state + heads[0])):
        raise ValueError(f"weight w_x: {tuple(x.shape)}, expected (2 * {d_state} + n_heads, d_inner)")
    return hymba_linear_heads(d_state, _weight("w_x", x), _weight("b_dt", b, "torch.float32"),
                              _weight("a_log", w["a_log"], "torch.float32", heads),
                              _weight("d_skip", w["d_skip"], "torch.float32", (x.shape[1],) if wide else None))
