"""ctypes binding of libdflash.so (include/dflash.h), names as in the header.

Argument marshalling only: every step of the round runs in the library's
CUDA kernels.  Importing this module loads the library and raises if it is
missing; there is no other implementation to fall back to.
"""

from __future__ import annotations

import ctypes as C
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdflash.so")

DFLASH_OK = 0
ERRORS = {-1: "CONFIG", -2: "CAPACITY", -3: "ARG", -4: "CUDA", -5: "DEVICE", -6: "TIMEOUT",
          -7: "STATE"}
DFLASH_F32, DFLASH_BF16, DFLASH_INT4G64, DFLASH_F16 = 0, 1, 2, 3
ROPE_SCALING = {"none": 0, "linear": 1, "parts": 2}
KV8_PAGE = 64
MAX_TAPS = 8
MAX_BLOCK = 16


class DFlashError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"DFLASH_ERR_{ERRORS.get(code, code)}: {msg}")
        self.code = code


class dflash_config(C.Structure):
    _fields_ = [
        ("hidden", C.c_int32), ("n_q", C.c_int32), ("n_kv", C.c_int32), ("head_dim", C.c_int32),
        ("ffn", C.c_int32), ("vocab", C.c_int32), ("tgt_layers", C.c_int32),
        ("drf_layers", C.c_int32), ("n_taps", C.c_int32), ("tap_layer", C.c_int32 * MAX_TAPS),
        ("block_max", C.c_int32), ("window", C.c_int32), ("max_seq", C.c_int32),
        ("eos_id", C.c_int32), ("dtype", C.c_int32), ("tgt_wfmt", C.c_int32),
        ("drf_wfmt", C.c_int32), ("ctx_norm", C.c_int32), ("rms_eps", C.c_float),
        ("rope_theta", C.c_float), ("lm_wfmt", C.c_int32), ("adaptive_block", C.c_int32),
    ]


class dflash_layer(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in (
        "wq", "wk", "wv", "wo", "w_gate", "w_up", "w_down",
        "sq", "sk", "sv", "so", "s_gate", "s_up", "s_down",
        "ln_attn", "ln_mlp", "q_norm", "k_norm")]


class dflash_weights(C.Structure):
    _fields_ = [
        ("embed", C.c_void_p), ("final_norm_tgt", C.c_void_p), ("final_norm_drf", C.c_void_p),
        ("fc", C.c_void_p), ("ctx_norm", C.c_void_p),
        ("tgt", C.POINTER(dflash_layer)), ("drf", C.POINTER(dflash_layer)),
        ("lm_head", C.c_void_p), ("lm_scales", C.c_void_p),
    ]


class dflash_stats_t(C.Structure):
    _fields_ = [
        ("rounds", C.c_int64), ("emitted", C.c_int64), ("accept_hist", C.c_int64 * MAX_BLOCK),
        ("n", C.c_int32), ("t_n", C.c_int32), ("block_len", C.c_int32), ("generated", C.c_int32),
        ("max_new", C.c_int32), ("ctx_len", C.c_int32), ("finished", C.c_int32),
        ("last_accept", C.c_int32), ("device_error", C.c_int32), ("pad_", C.c_int32),
    ]


class dflash_profile_t(C.Structure):
    _fields_ = [("gemm_launches", C.c_int64), ("gemm_ms", C.c_double), ("gemm_bytes", C.c_double),
                ("gemm_weight_bytes", C.c_double)]


class dflash_kv8_cache(C.Structure):
    _fields_ = [("k_codes", C.c_void_p), ("v_codes", C.c_void_p), ("k_scale", C.c_void_p),
                ("v_scale", C.c_void_p), ("n_pages", C.c_int32), ("n_kv", C.c_int32),
                ("head_dim", C.c_int32), ("pad_", C.c_int32)]


class dflash_kv8_query(C.Structure):
    _fields_ = [("q", C.c_void_p), ("out", C.c_void_p), ("lse", C.c_void_p), ("table", C.c_void_p),
                ("kv_len", C.c_void_p), ("row_start", C.c_void_p), ("q_row", C.c_int64),
                ("q_head", C.c_int64), ("out_row", C.c_int64), ("out_head", C.c_int64),
                ("rows", C.c_int32), ("n_q", C.c_int32), ("S", C.c_int32), ("max_pages", C.c_int32),
                ("dtype", C.c_int32), ("causal", C.c_int32), ("window", C.c_int32),
                ("scale", C.c_float)]


class dflash_drafts(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in (
        "probs", "draft_probs", "ids", "uniform", "row_start", "kv_len", "tokens", "n_tokens",
        "new_len")] + [
        ("probs_row", C.c_int64), ("draft_row", C.c_int64), ("rows", C.c_int32), ("vocab", C.c_int32),
        ("S", C.c_int32), ("pad_", C.c_int32)]


class dflash_evict(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in (
        "table", "kv_len", "weights", "weights_out", "budget", "new_len", "dropped", "source")] + [
        ("S", C.c_int32), ("max_pages", C.c_int32), ("keep_first", C.c_int32), ("keep_last", C.c_int32)]


class dflash_rope_config(C.Structure):
    _fields_ = [("rotary_dim", C.c_int32), ("interleaved", C.c_int32), ("scaling", C.c_int32),
                ("original_len", C.c_int32), ("theta", C.c_double), ("factor", C.c_double),
                ("alpha", C.c_double), ("beta", C.c_double), ("scale", C.c_float), ("pad_", C.c_int32)]


class dflash_heads(C.Structure):
    _fields_ = [("x", C.c_void_p), ("out", C.c_void_p), ("heads", C.c_int32), ("pad_", C.c_int32),
                ("x_row", C.c_int64), ("x_head", C.c_int64), ("out_row", C.c_int64),
                ("out_head", C.c_int64)]


def _load() -> C.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m block_diffusion_speculative_gather_gb300.build` (no fallback exists)")
    lib = C.CDLL(LIB_PATH)
    vp, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
    sig = {
        "dflash_workspace_bytes": (sz, [C.POINTER(dflash_config)]),
        "dflash_kv_target_bytes": (sz, [C.POINTER(dflash_config)]),
        "dflash_kv_draft_bytes": (sz, [C.POINTER(dflash_config)]),
        "dflash_init": (C.c_int, [C.POINTER(dflash_config), C.POINTER(dflash_weights), vp, vp,
                                  vp, sz, C.POINTER(vp)]),
        "dflash_prefill_taps": (C.c_int, [vp, vp, i32, vp, i32, i32, i32, i32, vp]),
        "dflash_draft_block": (C.c_int, [vp, vp, vp]),
        "dflash_verify_accept": (C.c_int, [vp, vp, vp, vp, vp]),
        "dflash_rollback": (C.c_int, [vp, i64, i32, vp]),
        "dflash_stats": (C.c_int, [vp, C.POINTER(dflash_stats_t), vp]),
        "dflash_check": (C.c_int, [vp, vp]),
        "dflash_set_logits_out": (C.c_int, [vp, vp, vp]),
        "dflash_destroy": (None, [vp]),
        "dflash_last_error": (C.c_char_p, []),
        "dflash_tap_reduce": (C.c_int, [C.POINTER(vp), i32, i32, i32, i32, vp, vp]),
        "dflash_quantize_int4g64": (C.c_int, [vp, i32, i32, vp, vp, vp]),
        "dflash_profile": (C.c_int, [vp, i32, C.POINTER(dflash_profile_t)]),
        "dflash_launch_count": (i64, []),
        "dflash_selftest_timeout": (C.c_int, [vp, i64, vp]),
        "dflash_adopt_kv": (C.c_int, [vp, i32, i32, i32, vp]),
        "dflash_linear_workspace_bytes": (sz, [i32, i32]),
        "dflash_linear": (C.c_int, [vp, vp, i32, i32, vp, vp, sz, vp, vp]),
        "dflash_linear_noalloc": (C.c_int, [vp, vp, i32, i32, vp, vp, vp]),
        "dflash_progress": (C.c_int, [vp, vp, vp]),
        "dflash_attention_form": (C.c_int, [vp, i32]),
        "dflash_linear_dense": (C.c_int, [vp, vp, vp, i32, i32, i32, vp, vp, vp]),
        "dflash_batch_workspace_bytes": (sz, [C.POINTER(dflash_config), i32]),
        "dflash_batch_init": (C.c_int, [C.POINTER(dflash_config), C.POINTER(dflash_weights), i32, vp,
                                        vp, vp, sz, C.POINTER(vp)]),
        "dflash_batch_context": (vp, [vp, i32]),
        "dflash_batch_draft": (C.c_int, [vp, vp, vp]),
        "dflash_batch_verify_accept": (C.c_int, [vp, vp, vp, vp, vp]),
        "dflash_batch_set_logits_out": (C.c_int, [vp, vp, vp]),
        "dflash_batch_check": (C.c_int, [vp, vp]),
        "dflash_batch_destroy": (None, [vp]),
        "dflash_pages_plan": (C.c_int, [vp, vp, i32, vp, i32, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp]),
        "dflash_pages_trim": (C.c_int, [vp, vp, i32, vp, i32, vp, vp, i32, vp]),
        "dflash_kv8_append": (C.c_int, [vp, vp, i64, i64, vp, i64, i64, i32, i32,
                                        vp, vp, vp]),
        "dflash_kv8_workspace_bytes": (sz, [i32, i32, i32, i32, i32, i32]),
        "dflash_kv8_attention": (C.c_int, [vp, vp, vp, sz,
                                           vp, vp]),
        "dflash_rope_turns": (C.c_int, [C.POINTER(dflash_rope_config), vp, vp]),
        "dflash_rope": (C.c_int, [C.POINTER(dflash_rope_config), vp, vp, i32, i32, i32,
                                  vp, vp, vp]),
        "dflash_probs": (C.c_int, [vp, i64, i32, vp, vp, i32, i32, vp, i64, vp]),
        "dflash_selftest_exchange": (C.c_int, [vp, vp, i32, i32, vp, i32, i32, i32, i64, vp]),
        "dflash_verify_workspace_bytes": (sz, [i32, i32]),
        "dflash_verify_drafts": (C.c_int, [vp, vp, sz, vp, vp]),
        "dflash_kv8_weigh": (C.c_int, [vp, vp, vp, vp, i32, i32, vp, vp]),
        "dflash_kv8_evict_workspace_bytes": (sz, [i32, i32]),
        "dflash_kv8_evict": (C.c_int, [vp, i32, vp, vp, sz, vp, vp]),
        "dflash_pages_shift": (C.c_int, [vp, vp, vp, i32, i32, vp, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = _load()

EXPORTED = ("dflash_workspace_bytes", "dflash_kv_target_bytes", "dflash_kv_draft_bytes",
            "dflash_init", "dflash_prefill_taps", "dflash_draft_block", "dflash_verify_accept",
            "dflash_rollback", "dflash_stats", "dflash_check", "dflash_set_logits_out",
            "dflash_destroy", "dflash_last_error", "dflash_tap_reduce",
            "dflash_quantize_int4g64", "dflash_profile", "dflash_launch_count",
            "dflash_selftest_timeout", "dflash_adopt_kv", "dflash_linear_workspace_bytes",
            "dflash_linear", "dflash_linear_noalloc",
            "dflash_progress", "dflash_attention_form", "dflash_linear_dense",
            "dflash_batch_workspace_bytes", "dflash_batch_init", "dflash_batch_context",
            "dflash_batch_draft", "dflash_batch_verify_accept", "dflash_batch_set_logits_out",
            "dflash_batch_check", "dflash_batch_destroy", "dflash_pages_plan", "dflash_pages_trim",
            "dflash_kv8_append", "dflash_kv8_workspace_bytes", "dflash_kv8_attention",
            "dflash_rope_turns", "dflash_rope", "dflash_probs", "dflash_selftest_exchange",
            "dflash_verify_workspace_bytes", "dflash_verify_drafts", "dflash_kv8_weigh", "dflash_kv8_evict_workspace_bytes",
            "dflash_kv8_evict", "dflash_pages_shift")


def check(rc: int) -> None:
    if rc != DFLASH_OK:
        raise DFlashError(rc, lib.dflash_last_error().decode())


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


DFLASH_ERR_ARG = -3


def _need(t, name: str, dtypes, shape) -> None:
    """Binding-side argument check of a standalone operation's tensor (the C
    ABI sees only pointers and sizes): dtype, shape (None = any extent) and
    row-major contiguity.  Raises DFlashError(ARG) before any device work."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise DFlashError(DFLASH_ERR_ARG, f"{name}: a torch tensor is required")
    if dtypes is not None and t.dtype not in dtypes:
        raise DFlashError(DFLASH_ERR_ARG, f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if shape is not None and (t.dim() != len(shape) or
                              any(e is not None and e != d for e, d in zip(shape, t.shape))):
        raise DFlashError(DFLASH_ERR_ARG, f"{name}: shape {tuple(t.shape)}, expected {shape}")
    if not t.is_contiguous():
        raise DFlashError(DFLASH_ERR_ARG, f"{name}: must be contiguous (row-major)")


def _on_gpu(**tensors) -> None:
    """Every tensor on one CUDA device: the library reads device pointers and
    has no CPU path."""
    devs = set()
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise DFlashError(DFLASH_ERR_ARG, f"{name}: a CUDA tensor is required (no CPU path)")
        devs.add(t.device)
    if len(devs) > 1:
        raise DFlashError(DFLASH_ERR_ARG, f"tensors on several devices: {sorted(map(str, devs))}")


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def dflash_workspace_bytes(cfg: dflash_config) -> int:
    return lib.dflash_workspace_bytes(C.byref(cfg))


def dflash_kv_target_bytes(cfg: dflash_config) -> int:
    return lib.dflash_kv_target_bytes(C.byref(cfg))


def dflash_kv_draft_bytes(cfg: dflash_config) -> int:
    return lib.dflash_kv_draft_bytes(C.byref(cfg))


def dflash_init(cfg, weights, kv_target, kv_draft, workspace) -> int:
    out = C.c_void_p()
    check(lib.dflash_init(C.byref(cfg), C.byref(weights), _ptr(kv_target), _ptr(kv_draft),
                          _ptr(workspace), workspace.numel() * workspace.element_size(),
                          C.byref(out)))
    return out.value


def dflash_prefill_taps(ctx, prompt_ids, ext_taps, n_ext, hc, first_token, max_new, stream=None):
    n_prompt = 0 if prompt_ids is None else prompt_ids.numel()
    check(lib.dflash_prefill_taps(ctx, _ptr(prompt_ids), n_prompt, _ptr(ext_taps), n_ext, hc,
                                  first_token, max_new, _stream(stream)))


def dflash_draft_block(ctx, draft_ids, stream=None):
    check(lib.dflash_draft_block(ctx, _ptr(draft_ids), _stream(stream)))


def dflash_verify_accept(ctx, draft_ids, tokens_out, n_emitted, stream=None):
    check(lib.dflash_verify_accept(ctx, _ptr(draft_ids), _ptr(tokens_out), _ptr(n_emitted),
                                   _stream(stream)))


def dflash_rollback(ctx, new_len: int, token: int, stream=None):
    check(lib.dflash_rollback(ctx, new_len, token, _stream(stream)))


def dflash_stats(ctx, stream=None) -> dflash_stats_t:
    out = dflash_stats_t()
    check(lib.dflash_stats(ctx, C.byref(out), _stream(stream)))
    return out


def dflash_check(ctx, stream=None):
    check(lib.dflash_check(ctx, _stream(stream)))


def dflash_set_logits_out(ctx, verify_logits, draft_logits):
    check(lib.dflash_set_logits_out(ctx, _ptr(verify_logits), _ptr(draft_logits)))


def dflash_destroy(ctx):
    lib.dflash_destroy(ctx)


def dflash_tap_reduce(layer_streams, rows: int, hc: int, hidden: int, out, stream=None):
    import torch
    for i, t in enumerate(layer_streams):
        _need(t, f"layer_streams[{i}]", (torch.bfloat16,), (rows, hc * hidden))
    _need(out, "out", (torch.float32,), (rows, len(layer_streams) * hidden))
    _on_gpu(out=out, **{f"layer_streams[{i}]": t for i, t in enumerate(layer_streams)})
    arr = (C.c_void_p * len(layer_streams))(*[t.data_ptr() for t in layer_streams])
    check(lib.dflash_tap_reduce(arr, len(layer_streams), rows, hc, hidden, _ptr(out),
                                _stream(stream)))


def dflash_quantize_int4g64(w, packed, scales, stream=None):
    import torch
    _need(w, "w", (torch.float32,), (None, None))
    n, k = w.shape
    _need(packed, "packed", (torch.uint8,), (n, k // 2))
    two_byte = tuple(d for d in (torch.int16, getattr(torch, "uint16", None)) if d is not None)
    _need(scales, "scales", two_byte, (k // 64, n))
    _on_gpu(w=w, packed=packed, scales=scales)
    check(lib.dflash_quantize_int4g64(_ptr(w), n, k, _ptr(packed), _ptr(scales), _stream(stream)))


def dflash_profile(ctx, mode: int) -> dflash_profile_t:
    """mode 1 start, 2 read, 0 read and stop (see include/dflash.h)."""
    out = dflash_profile_t()
    check(lib.dflash_profile(ctx, mode, C.byref(out)))
    return out


def dflash_launch_count() -> int:
    return lib.dflash_launch_count()


def dflash_selftest_timeout(ctx, limit_ns: int, stream=None):
    check(lib.dflash_selftest_timeout(ctx, limit_ns, _stream(stream)))


def dflash_adopt_kv(ctx, n: int, pending_token: int, max_new: int, stream=None):
    check(lib.dflash_adopt_kv(ctx, n, pending_token, max_new, _stream(stream)))


def dflash_linear_workspace_bytes(n: int, k: int) -> int:
    return lib.dflash_linear_workspace_bytes(n, k)


def _linear_operands(w, x, y):
    import torch
    _need(w, "w", (torch.bfloat16,), (None, None))
    n, k = w.shape
    _need(x, "x", (torch.bfloat16,), (MAX_BLOCK, k))
    _need(y, "y", (torch.float32,), (MAX_BLOCK, n))
    return n, k


def dflash_linear(w, x, y, workspace, err, stream=None):
    """y = x w^T (16 rows); err (int32[2] on the device) receives the GEMM's
    error words after it: {0, 0}, or {1, site} when a bounded wait ran out."""
    import torch
    n, k = _linear_operands(w, x, y)
    _need(workspace, "workspace", None, None)
    _need(err, "err", (torch.int32,), (2,))
    _on_gpu(w=w, x=x, y=y, workspace=workspace, err=err)
    check(lib.dflash_linear(_ptr(w), _ptr(x), n, k, _ptr(y), _ptr(workspace),
                            workspace.numel() * workspace.element_size(), _ptr(err),
                            _stream(stream)))


def dflash_linear_noalloc(w, x, y, err, stream=None):
    """y = x w^T like dflash_linear, with the library's fixed scratch instead
    of a caller workspace (for callers that cannot allocate device memory);
    err as in dflash_linear."""
    import torch
    n, k = _linear_operands(w, x, y)
    _need(err, "err", (torch.int32,), (2,))
    _on_gpu(w=w, x=x, y=y, err=err)
    check(lib.dflash_linear_noalloc(_ptr(w), _ptr(x), n, k, _ptr(y), _ptr(err), _stream(stream)))


def dflash_progress(ctx, out, stream=None):
    """Enqueue the progress words (finished, generated, n, emitted) into the
    int32[4] device tensor `out`."""
    check(lib.dflash_progress(ctx, _ptr(out), _stream(stream)))


def dflash_attention_form(ctx, model: int) -> int:
    """Attention form of the target (model 0) or drafter (model 1):
    2 tcgen05, 1 mma.sync split-KV, 0 separate partial/combine kernels."""
    r = lib.dflash_attention_form(ctx, model)
    check(min(r, 0))
    return r


def dflash_linear_dense(w, x, y, err, x_lo=None, stream=None):
    """y[m][n] = x[m] . w[n] (+ x_lo[m] . w[n]) on the tcgen05 dense GEMM:
    x, x_lo bf16 [M][K], w bf16 [N][K], y fp32 [M][N], err int32[2] zeros."""
    import torch
    _need(x, "x", (torch.bfloat16,), (None, None))
    m, k = x.shape
    _need(w, "w", (torch.bfloat16,), (None, k))
    n = w.shape[0]
    _need(y, "y", (torch.float32,), (m, n))
    if x_lo is not None:
        _need(x_lo, "x_lo", (torch.bfloat16,), (m, k))
    _need(err, "err", (torch.int32,), (None,))
    if err.numel() < 2:
        raise DFlashError(DFLASH_ERR_ARG, "err: int32[2] required")
    _on_gpu(w=w, x=x, x_lo=x_lo, y=y, err=err)
    check(lib.dflash_linear_dense(_ptr(w), _ptr(x), _ptr(x_lo), m, n, k, _ptr(y), _ptr(err),
                                  _stream(stream)))


# ---- several sequences in lockstep rounds

def dflash_batch_workspace_bytes(cfg, S: int) -> int:
    return lib.dflash_batch_workspace_bytes(C.byref(cfg), S)


def dflash_batch_init(cfg, weights, S: int, kv_target, kv_draft, workspace):
    out = C.c_void_p()
    check(lib.dflash_batch_init(C.byref(cfg), C.byref(weights), S, _ptr(kv_target), _ptr(kv_draft),
                                _ptr(workspace), workspace.numel() * workspace.element_size(),
                                C.byref(out)))
    return out.value


def dflash_batch_context(b, s: int):
    c = lib.dflash_batch_context(b, s)
    if not c:
        check(DFLASH_ERR_ARG)
    return c


def dflash_batch_draft(b, draft_ids, stream=None):
    check(lib.dflash_batch_draft(b, _ptr(draft_ids), _stream(stream)))


def dflash_batch_verify_accept(b, draft_ids, tokens_out, n_emitted, stream=None):
    check(lib.dflash_batch_verify_accept(b, _ptr(draft_ids), _ptr(tokens_out), _ptr(n_emitted),
                                         _stream(stream)))


def dflash_batch_set_logits_out(b, verify_logits=None, draft_logits=None):
    check(lib.dflash_batch_set_logits_out(b, _ptr(verify_logits), _ptr(draft_logits)))


def dflash_batch_check(b, stream=None):
    check(lib.dflash_batch_check(b, _stream(stream)))


def dflash_batch_destroy(b) -> None:
    lib.dflash_batch_destroy(b)


# ---- 8-bit paged KV cache and rotary positions
#
# These calls sit in a serving loop's every layer, where a few microseconds of
# checks are as long as the kernels: the common case is checked by plain
# comparisons, and only a call that fails one goes through the checks that
# name the tensor at fault.

_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32
_KINDS = {torch.float32: DFLASH_F32, torch.bfloat16: DFLASH_BF16, torch.float16: DFLASH_F16}
_HALVES = (torch.bfloat16, torch.float16)
_CODES = (torch.uint8, torch.float8_e4m3fn)
_MOST = 0x7fffffff
_CACHE = struct.Struct("4Q4i")        # dflash_kv8_cache
_QUERY = struct.Struct("6Q4q7if")     # dflash_kv8_query
_HEADS = struct.Struct("2Q2i4q")      # dflash_heads
_DRAFTS = struct.Struct("9Q2q4i")     # dflash_drafts
_EVICT = struct.Struct("8Q4i")        # dflash_evict


def _raw(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _flat(tensors, dev: int, dtype=_I32) -> bool:
    """Every tensor of dtype, contiguous, on device dev."""
    for t in tensors:
        if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
            return False
    return True


def _current(t) -> int:
    """The tensor's device where it is the current CUDA device, else -2 (no
    tensor is there)."""
    dev = t.get_device()
    return dev if dev >= 0 and dev == torch._C._cuda_getDevice() else -2


def _counts(**extents) -> None:
    """Extents that the C ABI's int32 arguments hold (a longer one would wrap)."""
    for name, n in extents.items():
        if n > _MOST:
            raise DFlashError(DFLASH_ERR_ARG, f"{name}: {n} is out of range")


def _here(**tensors) -> None:
    """Every tensor on the current CUDA device (the call is enqueued on one of
    its streams)."""
    _on_gpu(**tensors)
    cur = torch.cuda.current_device()
    for name, t in tensors.items():
        if t is not None and t.device.index != cur:
            raise DFlashError(DFLASH_ERR_ARG, f"{name}: on {t.device}, the current device is cuda:{cur}")


def _need_heads(t, name: str, dtypes, shape) -> None:
    """A [rows][heads][head_dim] tensor by strides: contiguous heads."""
    if not isinstance(t, torch.Tensor):
        raise DFlashError(DFLASH_ERR_ARG, f"{name}: a torch tensor is required")
    if t.dtype not in dtypes:
        raise DFlashError(DFLASH_ERR_ARG, f"{name}: dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if t.dim() != 3 or any(e is not None and e != d for e, d in zip(shape, t.shape)):
        raise DFlashError(DFLASH_ERR_ARG, f"{name}: shape {tuple(t.shape)}, expected {shape}")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise DFlashError(DFLASH_ERR_ARG, f"{name}: the elements of a head must be contiguous")


def dflash_pages_plan(kv_len, q_len, free_pages, n_free, table, row_start, positions, slots, kv_after,
                      n_free_out, stream=None):
    """Pages, row starts, positions and slots of the next step's rows (see
    include/dflash.h); rows = positions.numel().  int32 tensors throughout."""
    try:
        dev = _current(table)
        S, max_pages = table.shape
        one, (rows,), (pool,) = (S,), positions.shape, free_pages.shape
        fine = (kv_len.shape == one and q_len.shape == one and kv_after.shape == one and
                n_free.shape == (1,) and n_free_out.shape == (1,) and row_start.shape == (S + 1,) and
                slots.shape == (rows,) and
                _flat((table, kv_len, q_len, kv_after, free_pages, n_free, n_free_out, row_start, positions,
                       slots), dev))
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        i32 = (_I32,)
        _need(table, "table", i32, (None, None))
        S, max_pages = table.shape
        for name, t in (("kv_len", kv_len), ("q_len", q_len), ("kv_after", kv_after)):
            _need(t, name, i32, (S,))
        _need(free_pages, "free_pages", i32, (None,))
        _need(n_free, "n_free", i32, (1,))
        _need(n_free_out, "n_free_out", i32, (1,))
        _need(row_start, "row_start", i32, (S + 1,))
        _need(positions, "positions", i32, (None,))
        _need(slots, "slots", i32, (positions.shape[0],))
        _here(kv_len=kv_len, q_len=q_len, free_pages=free_pages, n_free=n_free, table=table,
              row_start=row_start, positions=positions, slots=slots, kv_after=kv_after,
              n_free_out=n_free_out)
        dev, rows, pool = table.get_device(), positions.shape[0], free_pages.shape[0]
    if S > _MOST or rows > _MOST or pool > _MOST or max_pages > _MOST:
        _counts(S=S, rows=rows, free_pages=pool, max_pages=max_pages)
    rc = lib.dflash_pages_plan(kv_len.data_ptr(), q_len.data_ptr(), S, free_pages.data_ptr(), pool,
                               n_free.data_ptr(), table.data_ptr(), max_pages, rows, row_start.data_ptr(),
                               positions.data_ptr(), slots.data_ptr(), kv_after.data_ptr(),
                               n_free_out.data_ptr(), _raw(stream, dev))
    if rc:
        check(rc)


def dflash_pages_trim(kv_len, new_len, free_pages, n_free, table, stream=None):
    """kv_len[s] = min(kv_len[s], new_len[s]); pages no longer needed go back
    onto free_pages."""
    try:
        dev = _current(table)
        S, max_pages = table.shape
        (pool,) = free_pages.shape
        fine = (kv_len.shape == (S,) and new_len.shape == (S,) and n_free.shape == (1,) and
                _flat((table, kv_len, new_len, free_pages, n_free), dev))
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        i32 = (_I32,)
        _need(table, "table", i32, (None, None))
        S, max_pages = table.shape
        _need(kv_len, "kv_len", i32, (S,))
        _need(new_len, "new_len", i32, (S,))
        _need(free_pages, "free_pages", i32, (None,))
        _need(n_free, "n_free", i32, (1,))
        _here(kv_len=kv_len, new_len=new_len, free_pages=free_pages, n_free=n_free, table=table)
        dev, pool = table.get_device(), free_pages.shape[0]
    if S > _MOST or max_pages > _MOST or pool > _MOST:
        _counts(S=S, max_pages=max_pages, free_pages=pool)
    rc = lib.dflash_pages_trim(kv_len.data_ptr(), new_len.data_ptr(), S, free_pages.data_ptr(), pool,
                               n_free.data_ptr(), table.data_ptr(), max_pages, _raw(stream, dev))
    if rc:
        check(rc)


def _cache_ok(shape, k_codes, v_codes, k_scale, v_scale, dev: int) -> bool:
    per_page = shape[:2]
    return (shape[2] == KV8_PAGE and v_codes.shape == shape and k_scale.shape == per_page and
            v_scale.shape == per_page and k_codes.dtype in _CODES and v_codes.dtype in _CODES and
            v_codes.get_device() == dev and k_codes.is_contiguous() and v_codes.is_contiguous() and
            k_scale.dtype is _F32 and v_scale.dtype is _F32 and k_scale.get_device() == dev and
            v_scale.get_device() == dev and k_scale.is_contiguous() and v_scale.is_contiguous())


def _need_cache(k_codes, v_codes, k_scale, v_scale) -> None:
    _need(k_codes, "k_codes", _CODES, (None, None, KV8_PAGE, None))
    n_pages, n_kv, _, hd = k_codes.shape
    _need(v_codes, "v_codes", _CODES, (n_pages, n_kv, KV8_PAGE, hd))
    _need(k_scale, "k_scale", (_F32,), (n_pages, n_kv))
    _need(v_scale, "v_scale", (_F32,), (n_pages, n_kv))


def dflash_kv8_append(k, v, slots, k_codes, v_codes, k_scale, v_scale, err, stream=None):
    """Quantise rows k, v [rows][n_kv][head_dim] (fp32, bf16 or f16, strided
    rows and heads) into the pool at slots [rows]; negative slots skip."""
    try:
        dev = _current(k_codes)
        shape = k_codes.shape
        n_pages, n_kv, _, hd = shape
        (rows,) = slots.shape
        kind, ks, vs = k.dtype, k.stride(), v.stride()
        fine = (kind in _KINDS and v.dtype is kind and k.shape == (rows, n_kv, hd) and v.shape == k.shape and
                ks[2] == 1 and vs[2] == 1 and k.get_device() == dev and v.get_device() == dev and
                err.shape == (2,) and _flat((slots, err), dev) and
                _cache_ok(shape, k_codes, v_codes, k_scale, v_scale, dev))
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        _need_cache(k_codes, v_codes, k_scale, v_scale)
        _need(slots, "slots", (_I32,), (None,))
        n_pages, n_kv, _, hd = k_codes.shape
        rows = slots.shape[0]
        _need_heads(k, "k", _KINDS, (rows, n_kv, hd))
        _need_heads(v, "v", (k.dtype,), (rows, n_kv, hd))
        _need(err, "err", (_I32,), (2,))
        _here(k=k, v=v, slots=slots, k_codes=k_codes, v_codes=v_codes, k_scale=k_scale, v_scale=v_scale,
              err=err)
        dev, kind, ks, vs = k.get_device(), k.dtype, k.stride(), v.stride()
    if n_pages > _MOST or rows > _MOST:
        _counts(n_pages=n_pages, rows=rows)
    cache = _CACHE.pack(k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                        n_pages, n_kv, hd, 0)
    rc = lib.dflash_kv8_append(cache, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], _KINDS[kind],
                               rows, slots.data_ptr(), err.data_ptr(), _raw(stream, dev))
    if rc:
        check(rc)


def dflash_kv8_workspace_bytes(rows: int, S: int, n_q: int, n_kv: int, head_dim: int, max_pages: int) -> int:
    return lib.dflash_kv8_workspace_bytes(rows, S, n_q, n_kv, head_dim, max_pages)


def dflash_kv8_attention(q, k_codes, v_codes, k_scale, v_scale, table, kv_len, row_start, out, workspace,
                         err, lse=None, scale=None, causal=True, window=0, stream=None):
    """out = softmax(scale q k^T + mask) v of each sequence's rows over its
    cached positions; q, out [rows][n_q][head_dim] bf16 or f16 by strides,
    lse fp32 [rows][n_q]; scale None: head_dim ** -0.5."""
    try:
        dev = _current(k_codes)
        cshape = k_codes.shape
        n_pages, n_kv, _, _ = cshape
        shape = q.shape
        rows, n_q, hd = shape
        S, max_pages = table.shape
        kind, qs, os_ = q.dtype, q.stride(), out.stride()
        fine = (kind in _HALVES and out.dtype is kind and out.shape == shape and hd == cshape[3] and
                qs[2] == 1 and os_[2] == 1 and q.get_device() == dev and out.get_device() == dev and
                kv_len.shape == (S,) and row_start.shape == (S + 1,) and err.shape == (2,) and
                _flat((table, kv_len, row_start, err), dev) and workspace.get_device() == dev and
                workspace.is_contiguous() and _cache_ok(cshape, k_codes, v_codes, k_scale, v_scale, dev) and
                (lse is None or (lse.shape == shape[:2] and _flat((lse,), dev, _F32))))
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        _need_cache(k_codes, v_codes, k_scale, v_scale)
        n_pages, n_kv, _, hd = k_codes.shape
        _need_heads(q, "q", _HALVES, (None, None, hd))
        rows, n_q, _ = q.shape
        _need_heads(out, "out", (q.dtype,), (rows, n_q, hd))
        i32 = (_I32,)
        _need(table, "table", i32, (None, None))
        S, max_pages = table.shape
        _need(kv_len, "kv_len", i32, (S,))
        _need(row_start, "row_start", i32, (S + 1,))
        if lse is not None:
            _need(lse, "lse", (_F32,), (rows, n_q))
        _need(workspace, "workspace", None, None)
        _need(err, "err", i32, (2,))
        _here(q=q, out=out, k_codes=k_codes, v_codes=v_codes, k_scale=k_scale, v_scale=v_scale, table=table,
              kv_len=kv_len, row_start=row_start, workspace=workspace, err=err, lse=lse)
        dev, kind, qs, os_ = q.get_device(), q.dtype, q.stride(), out.stride()
    if n_pages > _MOST or rows > _MOST or S > _MOST or max_pages > _MOST:
        _counts(n_pages=n_pages, rows=rows, S=S, max_pages=max_pages)
    cache = _CACHE.pack(k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                        n_pages, n_kv, hd, 0)
    try:
        args = _QUERY.pack(q.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(), table.data_ptr(),
                           kv_len.data_ptr(), row_start.data_ptr(), qs[0], qs[1], os_[0], os_[1], rows, n_q, S,
                           max_pages, _KINDS[kind], 1 if causal else 0, window,
                           hd ** -0.5 if scale is None else scale)
    except struct.error as e:
        raise DFlashError(DFLASH_ERR_ARG, f"window {window!r} (an int32), scale {scale!r} (a number): {e}") from None
    rc = lib.dflash_kv8_attention(cache, args, workspace.data_ptr(), workspace.nbytes, err.data_ptr(),
                                  _raw(stream, dev))
    if rc:
        check(rc)


def rope_config(rotary_dim: int, theta: float = 1e6, interleaved: bool = False, scaling: str = "none",
                factor: float = 1.0, original_len: int = 0, alpha: float = 1.0, beta: float = 32.0,
                scale: float = 1.0) -> dflash_rope_config:
    """Settings of dflash_rope; scaling "none", "linear" or "parts"."""
    if scaling not in ROPE_SCALING:
        raise DFlashError(DFLASH_ERR_ARG, f"scaling {scaling!r}, expected one of {tuple(ROPE_SCALING)}")
    return dflash_rope_config(rotary_dim, 1 if interleaved else 0, ROPE_SCALING[scaling], original_len,
                              theta, factor, alpha, beta, scale, 0)


def dflash_rope_turns(cfg: dflash_rope_config, turns, stream=None):
    """The frequency table of cfg: int64 [rotary_dim / 2], 2^-64 turns a position."""
    _need(turns, "turns", (torch.int64,), (cfg.rotary_dim // 2,))
    _here(turns=turns)
    check(lib.dflash_rope_turns(C.byref(cfg), turns.data_ptr(), _raw(stream, turns.get_device())))


def dflash_rope(cfg: dflash_rope_config, turns, positions, x, out, x2=None, out2=None, stream=None):
    """Rotate x (and x2) [rows][heads][head_dim] into out (out2) at positions
    [rows]; fp32, bf16 or f16, strided rows and heads, out may be x."""
    if (x2 is None) != (out2 is None):
        raise DFlashError(DFLASH_ERR_ARG, "x2 and out2 go together")
    try:
        dev = _current(x)
        shape = x.shape
        rows, heads, hd = shape
        kind, xs, os_ = x.dtype, x.stride(), out.stride()
        fine = (kind in _KINDS and out.dtype is kind and out.shape == shape and xs[2] == 1 and os_[2] == 1 and
                out.get_device() == dev and positions.shape == (rows,) and _flat((positions,), dev) and
                turns.shape == (cfg.rotary_dim // 2,) and _flat((turns,), dev, _I64))
        if x2 is not None:
            xs2, os2 = x2.stride(), out2.stride()
            r2, heads2, h2 = x2.shape
            fine = (fine and r2 == rows and h2 == hd and out2.shape == x2.shape and x2.dtype is kind and
                    out2.dtype is kind and xs2[2] == 1 and os2[2] == 1 and x2.get_device() == dev and
                    out2.get_device() == dev)
    except (AttributeError, TypeError, ValueError, IndexError):
        fine = False
    if not fine:
        _need(turns, "turns", (_I64,), (cfg.rotary_dim // 2,))
        _need(positions, "positions", (_I32,), (None,))
        rows = positions.shape[0]
        _need_heads(x, "x", _KINDS, (rows, None, None))
        _, heads, hd = x.shape
        _need_heads(out, "out", (x.dtype,), tuple(x.shape))
        if x2 is not None:
            _need_heads(x2, "x2", (x.dtype,), (rows, None, hd))
            _need_heads(out2, "out2", (x.dtype,), tuple(x2.shape))
            heads2, xs2, os2 = x2.shape[1], x2.stride(), out2.stride()
        _here(turns=turns, positions=positions, x=x, out=out, x2=x2, out2=out2)
        dev, kind, xs, os_ = x.get_device(), x.dtype, x.stride(), out.stride()
    if rows > _MOST:
        _counts(rows=rows)
    first = _HEADS.pack(x.data_ptr(), out.data_ptr(), heads, 0, xs[0], xs[1], os_[0], os_[1])
    second = None if x2 is None else _HEADS.pack(x2.data_ptr(), out2.data_ptr(), heads2, 0, xs2[0], xs2[1],
                                                 os2[0], os2[1])
    rc = lib.dflash_rope(C.byref(cfg), turns.data_ptr(), positions.data_ptr(), rows, hd, _KINDS[kind], first,
                         second, _raw(stream, dev))
    if rc:
        check(rc)


# ---- sampled tokens

def _need_rows(t, name: str, dtypes, shape) -> None:
    """A [rows][vocab] tensor by its row stride: contiguous tokens."""
    if not isinstance(t, torch.Tensor):
        raise DFlashError(DFLASH_ERR_ARG, f"{name}: a torch tensor is required")
    if t.dtype not in dtypes:
        raise DFlashError(DFLASH_ERR_ARG, f"{name}: dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if t.dim() != 2 or any(e is not None and e != d for e, d in zip(shape, t.shape)):
        raise DFlashError(DFLASH_ERR_ARG, f"{name}: shape {tuple(t.shape)}, expected {shape}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise DFlashError(DFLASH_ERR_ARG, f"{name}: the tokens of a row must be contiguous")


def dflash_probs(logits, temperature, out, min_p=None, stream=None):
    """out[r] = softmax(logits[r] / temperature[r]) over the tokens that min_p[r]
    leaves (temperature 0: 1 at the first maximum); logits [rows][vocab] fp32,
    bf16 or f16 by row stride, out fp32 (may be fp32 logits)."""
    try:
        dev = _current(logits)
        shape = logits.shape
        rows, vocab = shape
        kind, xs, ps = logits.dtype, logits.stride(), out.stride()
        fine = (kind in _KINDS and out.dtype is _F32 and out.shape == shape and xs[1] == 1 and ps[1] == 1 and
                out.get_device() == dev and temperature.shape == (rows,) and _flat((temperature,), dev, _F32) and
                (min_p is None or (min_p.shape == (rows,) and _flat((min_p,), dev, _F32))))
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        _need_rows(logits, "logits", _KINDS, (None, None))
        rows, vocab = logits.shape
        _need_rows(out, "out", (_F32,), (rows, vocab))
        _need(temperature, "temperature", (_F32,), (rows,))
        if min_p is not None:
            _need(min_p, "min_p", (_F32,), (rows,))
        _here(logits=logits, out=out, temperature=temperature, min_p=min_p)
        dev, kind, xs, ps = logits.get_device(), logits.dtype, logits.stride(), out.stride()
    if rows > _MOST or vocab > _MOST:
        _counts(rows=rows, vocab=vocab)
    rc = lib.dflash_probs(logits.data_ptr(), xs[0], _KINDS[kind], temperature.data_ptr(),
                          None if min_p is None else min_p.data_ptr(), rows, vocab, out.data_ptr(), ps[0],
                          _raw(stream, dev))
    if rc:
        check(rc)


def dflash_selftest_exchange(logits, temperature, out, stays: bool, word: int, row: int, limit_ns: int, stream=None):
    """dflash_probs of fp32 rows by clusters of two CTAs (one a row, or one that
    stays for all rows) whose second CTA keeps its word of an exchange to itself."""
    rows, vocab = logits.shape
    _need(logits, "logits", (_F32,), (None, None))
    _need(out, "out", (_F32,), (rows, vocab))
    _need(temperature, "temperature", (_F32,), (rows,))
    _here(logits=logits, out=out, temperature=temperature)
    check(lib.dflash_selftest_exchange(logits.data_ptr(), temperature.data_ptr(), rows, vocab, out.data_ptr(),
                                       1 if stays else 0, word, row, limit_ns, _raw(stream, logits.get_device())))


def dflash_verify_workspace_bytes(S: int, vocab: int) -> int:
    return lib.dflash_verify_workspace_bytes(S, vocab)


def dflash_verify_drafts(probs, ids, uniform, row_start, tokens, n_tokens, workspace, err, draft_probs=None,
                         kv_len=None, new_len=None, stream=None):
    """Accept or refuse the drafts ids[r] (rows behind each sequence's first)
    against probs [rows][vocab] and draw each sequence's last token, from
    uniform [rows]; draft_probs None: certain drafts.  Writes tokens [rows],
    n_tokens [S] and, with kv_len, new_len [S]."""
    try:
        dev = _current(probs)
        shape = probs.shape
        rows, vocab = shape
        (S,) = n_tokens.shape
        one, ps = (rows,), probs.stride()
        qs = ps if draft_probs is None else draft_probs.stride()
        fine = (probs.dtype is _F32 and ps[1] == 1 and qs[1] == 1 and ids.shape == one and tokens.shape == one and
                uniform.shape == one and row_start.shape == (S + 1,) and err.shape == (2,) and
                _flat((ids, tokens, row_start, n_tokens, err), dev) and _flat((uniform,), dev, _F32) and
                workspace.get_device() == dev and workspace.is_contiguous() and
                (draft_probs is None or (draft_probs.dtype is _F32 and draft_probs.shape == shape and
                                         draft_probs.get_device() == dev)) and
                (kv_len is None) == (new_len is None) and
                (kv_len is None or (kv_len.shape == (S,) and new_len.shape == (S,) and _flat((kv_len, new_len), dev))))
    except (AttributeError, TypeError, ValueError, IndexError):
        fine = False
    if not fine:
        _need_rows(probs, "probs", (_F32,), (None, None))
        rows, vocab = probs.shape
        i32 = (_I32,)
        _need(n_tokens, "n_tokens", i32, (None,))
        S = n_tokens.shape[0]
        if draft_probs is not None:
            _need_rows(draft_probs, "draft_probs", (_F32,), (rows, vocab))
        _need(ids, "ids", i32, (rows,))
        _need(tokens, "tokens", i32, (rows,))
        _need(uniform, "uniform", (_F32,), (rows,))
        _need(row_start, "row_start", i32, (S + 1,))
        if (kv_len is None) != (new_len is None):
            raise DFlashError(DFLASH_ERR_ARG, "kv_len and new_len go together")
        if kv_len is not None:
            _need(kv_len, "kv_len", i32, (S,))
            _need(new_len, "new_len", i32, (S,))
        _need(workspace, "workspace", None, None)
        _need(err, "err", i32, (2,))
        _here(probs=probs, draft_probs=draft_probs, ids=ids, uniform=uniform, row_start=row_start, tokens=tokens,
              n_tokens=n_tokens, workspace=workspace, err=err, kv_len=kv_len, new_len=new_len)
        dev, ps = probs.get_device(), probs.stride()
        qs = ps if draft_probs is None else draft_probs.stride()
    if rows > _MOST or vocab > _MOST or S > _MOST:
        _counts(rows=rows, vocab=vocab, S=S)
    args = _DRAFTS.pack(probs.data_ptr(), 0 if draft_probs is None else draft_probs.data_ptr(), ids.data_ptr(),
                        uniform.data_ptr(), row_start.data_ptr(), 0 if kv_len is None else kv_len.data_ptr(),
                        tokens.data_ptr(), n_tokens.data_ptr(), 0 if new_len is None else new_len.data_ptr(),
                        ps[0], qs[0], rows, vocab, S, 0)
    rc = lib.dflash_verify_drafts(args, workspace.data_ptr(), workspace.nbytes, err.data_ptr(), _raw(stream, dev))
    if rc:
        check(rc)


# ---- eviction from the 8-bit paged cache

def dflash_kv8_weigh(q, lse, k_codes, v_codes, k_scale, v_scale, table, kv_len, row_start, weights, err, count=None,
                     observe=0, fresh=False, scale=None, causal=True, window=0, stream=None):
    """weights[page][offset] += the attention weight that the counted rows of q
    [rows][n_q][head_dim] give each cached position; lse fp32 [rows][n_q] as
    dflash_kv8_attention wrote it, weights fp32 [n_pages][64]; count int32 [S]:
    the first rows that count, observe: the last of those (0: all); fresh: the
    step's own positions start from 0."""
    try:
        dev = _current(k_codes)
        cshape = k_codes.shape
        n_pages, n_kv, _, _ = cshape
        shape = q.shape
        rows, n_q, hd = shape
        S, max_pages = table.shape
        kind, qs = q.dtype, q.stride()
        fine = (kind in _HALVES and hd == cshape[3] and qs[2] == 1 and q.get_device() == dev and
                kv_len.shape == (S,) and row_start.shape == (S + 1,) and err.shape == (2,) and
                _flat((table, kv_len, row_start, err), dev) and lse.shape == shape[:2] and
                weights.shape == (n_pages, KV8_PAGE) and _flat((lse, weights), dev, _F32) and
                _cache_ok(cshape, k_codes, v_codes, k_scale, v_scale, dev) and
                (count is None or (count.shape == (S,) and _flat((count,), dev))))
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        _need_cache(k_codes, v_codes, k_scale, v_scale)
        n_pages, n_kv, _, hd = k_codes.shape
        _need_heads(q, "q", _HALVES, (None, None, hd))
        rows, n_q, _ = q.shape
        i32 = (_I32,)
        _need(table, "table", i32, (None, None))
        S, max_pages = table.shape
        _need(kv_len, "kv_len", i32, (S,))
        _need(row_start, "row_start", i32, (S + 1,))
        _need(lse, "lse", (_F32,), (rows, n_q))
        _need(weights, "weights", (_F32,), (n_pages, KV8_PAGE))
        if count is not None:
            _need(count, "count", i32, (S,))
        _need(err, "err", i32, (2,))
        _here(q=q, lse=lse, k_codes=k_codes, v_codes=v_codes, k_scale=k_scale, v_scale=v_scale, table=table,
              kv_len=kv_len, row_start=row_start, weights=weights, err=err, count=count)
        dev, kind, qs = q.get_device(), q.dtype, q.stride()
    if n_pages > _MOST or rows > _MOST or S > _MOST or max_pages > _MOST:
        _counts(n_pages=n_pages, rows=rows, S=S, max_pages=max_pages)
    if not 0 <= observe <= _MOST:
        raise DFlashError(DFLASH_ERR_ARG, f"observe {observe!r}: 0 or a number of rows (an int32)")
    cache = _CACHE.pack(k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                        n_pages, n_kv, hd, 0)
    try:
        args = _QUERY.pack(q.data_ptr(), 0, lse.data_ptr(), table.data_ptr(), kv_len.data_ptr(),
                           row_start.data_ptr(), qs[0], qs[1], 0, 0, rows, n_q, S, max_pages, _KINDS[kind],
                           1 if causal else 0, window, hd ** -0.5 if scale is None else scale)
    except struct.error as e:
        raise DFlashError(DFLASH_ERR_ARG, f"window {window!r} (an int32), scale {scale!r} (a number): {e}") from None
    rc = lib.dflash_kv8_weigh(cache, args, weights.data_ptr(), None if count is None else count.data_ptr(), observe,
                              1 if fresh else 0, err.data_ptr(), _raw(stream, dev))
    if rc:
        check(rc)


class kv8_layers:
    """The pools of a model's layers, [(k_codes, v_codes, k_scale, v_scale), ..],
    all of one shape on one device and none given twice, checked and packed once
    for dflash_kv8_evict.  Holds the tensors."""

    def __init__(self, caches):
        self.caches = [tuple(c) for c in caches]
        if not self.caches:
            raise DFlashError(DFLASH_ERR_ARG, "layers: at least one")
        shape = None
        for c in self.caches:
            if len(c) != 4:
                raise DFlashError(DFLASH_ERR_ARG, "layers: (k_codes, v_codes, k_scale, v_scale) each")
            _need_cache(*c)
            shape = shape or c[0].shape
            if c[0].shape != shape:
                raise DFlashError(DFLASH_ERR_ARG, f"layers: shapes {tuple(shape)} and {tuple(c[0].shape)}")
        _on_gpu(**{f"layer {i} {n}": t for i, c in enumerate(self.caches)
                   for n, t in zip(("k_codes", "v_codes", "k_scale", "v_scale"), c)})
        self.n_pages, self.n_kv, _, self.head_dim = shape
        _counts(n_pages=self.n_pages)
        self.device = self.caches[0][0].get_device()
        self.packed = b"".join(_CACHE.pack(*(t.data_ptr() for t in c), self.n_pages, self.n_kv, self.head_dim, 0)
                               for c in self.caches)


def dflash_kv8_evict_workspace_bytes(S: int, max_pages: int) -> int:
    return lib.dflash_kv8_evict_workspace_bytes(S, max_pages)


def dflash_kv8_evict(layers, table, kv_len, weights, budget, new_len, source, workspace, err, weights_out=None,
                     dropped=None, keep_first=0, keep_last=0, stream=None):
    """Sequences above their budget [S] keep their first and last positions and
    the heaviest of the others, moved down in order in every layer of `layers`
    (a kv8_layers) and in weights_out (None: in place); new_len [S] and source
    [S][max_pages * 64] say what stayed, dropped [S] grows by what went.
    dflash_pages_trim(kv_len, new_len, ..) takes the pages back."""
    weights_out = weights if weights_out is None else weights_out
    try:
        dev = _current(table)
        S, max_pages = table.shape
        one, plane = (S,), (layers.n_pages, KV8_PAGE)
        fine = (layers.device == dev and kv_len.shape == one and budget.shape == one and new_len.shape == one and
                source.shape == (S, max_pages * KV8_PAGE) and weights.shape == plane and weights_out.shape == plane and
                err.shape == (2,) and _flat((table, kv_len, budget, new_len, source, err), dev) and
                _flat((weights, weights_out), dev, _F32) and workspace.get_device() == dev and
                workspace.is_contiguous() and (dropped is None or (dropped.shape == one and _flat((dropped,), dev))))
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        if not isinstance(layers, kv8_layers):
            raise DFlashError(DFLASH_ERR_ARG, "layers: a kv8_layers is required")
        i32 = (_I32,)
        _need(table, "table", i32, (None, None))
        S, max_pages = table.shape
        for name, t in (("kv_len", kv_len), ("budget", budget), ("new_len", new_len)):
            _need(t, name, i32, (S,))
        if dropped is not None:
            _need(dropped, "dropped", i32, (S,))
        _need(source, "source", i32, (S, max_pages * KV8_PAGE))
        _need(weights, "weights", (_F32,), (layers.n_pages, KV8_PAGE))
        _need(weights_out, "weights_out", (_F32,), (layers.n_pages, KV8_PAGE))
        _need(workspace, "workspace", None, None)
        _need(err, "err", i32, (2,))
        _here(k_codes=layers.caches[0][0], table=table, kv_len=kv_len, budget=budget, new_len=new_len, source=source,
              weights=weights, weights_out=weights_out, workspace=workspace, err=err, dropped=dropped)
        dev = table.get_device()
    if S > _MOST or max_pages > _MOST:
        _counts(S=S, max_pages=max_pages)
    try:
        args = _EVICT.pack(table.data_ptr(), kv_len.data_ptr(), weights.data_ptr(), weights_out.data_ptr(),
                           budget.data_ptr(), new_len.data_ptr(), 0 if dropped is None else dropped.data_ptr(),
                           source.data_ptr(), S, max_pages, keep_first, keep_last)
    except struct.error as e:
        raise DFlashError(DFLASH_ERR_ARG, f"keep_first {keep_first!r}, keep_last {keep_last!r} (int32): {e}") from None
    rc = lib.dflash_kv8_evict(layers.packed, len(layers.caches), args, workspace.data_ptr(), workspace.nbytes,
                              err.data_ptr(), _raw(stream, dev))
    if rc:
        check(rc)


def dflash_pages_shift(positions, row_start, dropped, out, stream=None):
    """out[r] = positions[r] + dropped[sequence of r] (-1 stays): where to rotate
    a step's rows behind evictions; a sequence that begins at position 0 has its
    dropped set to 0."""
    try:
        dev = _current(positions)
        (rows,), (S,) = positions.shape, dropped.shape
        fine = (out.shape == (rows,) and row_start.shape == (S + 1,) and _flat((positions, row_start, dropped, out), dev))
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        i32 = (_I32,)
        _need(positions, "positions", i32, (None,))
        _need(dropped, "dropped", i32, (None,))
        rows, S = positions.shape[0], dropped.shape[0]
        _need(row_start, "row_start", i32, (S + 1,))
        _need(out, "out", i32, (rows,))
        _here(positions=positions, row_start=row_start, dropped=dropped, out=out)
        dev = positions.get_device()
    if rows > _MOST or S > _MOST:
        _counts(rows=rows, S=S)
    rc = lib.dflash_pages_shift(positions.data_ptr(), row_start.data_ptr(), dropped.data_ptr(), rows, S,
                                out.data_ptr(), _raw(stream, dev))
    if rc:
        check(rc)
