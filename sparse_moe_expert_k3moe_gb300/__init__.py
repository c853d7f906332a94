"""Routed-expert layer of a Kimi-K3-style latent MoE on GB300 (sm_103a), and the
full-width Stable LatentMoE block around it (``k3moe_full_forward``, ``MoEBlock``);
and the token mixer beside the block: linear projections with their epilogue
(``k3moe_linear``, ``Linear``) and the gated delta rule (``k3moe_delta_rule``,
``DeltaRule``); and the latent attention's layer beside both: norms around a block
(``k3moe_norm``, ``Norm``), each head's own projection (``k3moe_head_linear``,
``HeadLinear``), the latent cache's write and attention in the absorbed and the expanded form
(``k3moe_latent_write``, ``k3moe_latent_attend``, ``k3moe_latent_prompt``, ``LatentAttention``).

A thin ctypes binding over ``libk3moe.so``; every function has the name of the C
entry point it calls (``include/k3moe.h``) and only marshals arguments: torch
tensors become device pointers, the current torch stream becomes the CUDA
stream.  All computation happens in the library's CUDA kernels; there is no
CPU fallback -- importing this package without the built library raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

__all__ = [
    "K3MoEConfig", "K3MOE_OK", "K3MoEError", "lib", "k3moe_config", "k3moe_validate_config",
    "k3moe_packed_bytes", "k3moe_workspace_bytes", "k3moe_pack_mxfp4", "k3moe_unpack_mxfp4",
    "k3moe_route", "k3moe_router_scores", "k3moe_forward", "k3moe_forward_noalloc", "k3moe_device_status",
    "k3moe_check_wait_timeout", "k3moe_check_bounds", "k3moe_build_flags", "k3moe_strerror",
    "k3moe_launch_count", "k3moe_timing_enable", "k3moe_timing_read", "k3moe_timing_reset",
    "k3moe_set_prefill_gemm", "k3moe_get_prefill_gemm", "PREFILL_GEMM_F16", "PREFILL_GEMM_BLOCK_SCALED",
    "library_path", "MoELayer", "K3MoEFullDims", "k3moe_full_dims", "k3moe_full_workspace_bytes",
    "k3moe_full_forward", "MoEBlock",
    "K3MoELinearConfig", "k3moe_linear_config", "k3moe_linear_workspace_bytes", "k3moe_linear", "Linear",
    "K3MoEDeltaConfig", "k3moe_delta_config", "k3moe_delta_validate_config", "k3moe_delta_workspace_bytes",
    "k3moe_delta_rule", "DeltaRule", "ACTIVATIONS",
    "K3MoENormConfig", "k3moe_norm_config", "k3moe_norm", "Norm", "GATES",
    "K3MoEHeadLinearConfig", "k3moe_head_linear_config", "k3moe_head_linear_workspace_bytes", "k3moe_head_linear", "HeadLinear",
    "K3MoELatentConfig", "k3moe_latent_config", "k3moe_latent_validate_config", "k3moe_latent_workspace_bytes",
    "k3moe_latent_write", "k3moe_latent_attend", "k3moe_latent_prompt", "LatentAttention", "ROPES",
]

_HERE = os.path.dirname(os.path.abspath(__file__))


def _lib_file() -> str:
    """The library of the variant K3MOE_BUILD_VARIANT names (libk3moe.so by default)."""
    from .build import lib_path
    return lib_path()

K3MOE_OK = 0
STATUS_NAMES = {0: "OK", 1: "EINVAL", 2: "ESHAPE", 3: "EALIGN", 4: "EWORKSPACE", 5: "ECUDA",
                6: "EDEVICE", 7: "ETIMEOUT"}
DEV_BAD_INDEX, DEV_BAD_OFFSETS, DEV_NAN_SCALE, DEV_TIMEOUT, DEV_BOUNDS = 0x1, 0x2, 0x4, 0x8, 0x10


class K3MoEConfig(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("f", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("n_shared", ctypes.c_int32), ("group", ctypes.c_int32),
                ("situ_b1", ctypes.c_float), ("situ_b2", ctypes.c_float),
                ("renorm", ctypes.c_int32), ("routed_scale", ctypes.c_float)]


class K3MoEFullDims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("latent_norm", ctypes.c_int32), ("rms_eps", ctypes.c_float)]


class K3MoELinearConfig(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("k", ctypes.c_int32), ("act", ctypes.c_int32), ("y_f32", ctypes.c_int32)]


class K3MoEDeltaConfig(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("n_qk_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("gate_dim", ctypes.c_int32), ("qk_norm", ctypes.c_int32), ("norm_eps", ctypes.c_float),
                ("scale", ctypes.c_float)]


class K3MoENormConfig(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("group", ctypes.c_int32), ("post_norm", ctypes.c_int32), ("pre_norm", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("x_f32", ctypes.c_int32), ("sum_f32", ctypes.c_int32), ("eps", ctypes.c_float),
                ("alpha", ctypes.c_float)]


class K3MoEHeadLinearConfig(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32)]


class K3MoELatentConfig(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("rank", ctypes.c_int32), ("rope_dim", ctypes.c_int32), ("key_dim", ctypes.c_int32),
                ("value_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("rope", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("norm_eps", ctypes.c_float), ("scale", ctypes.c_float), ("causal", ctypes.c_int32)]


class K3MoEError(RuntimeError):
    def __init__(self, what: str, status: int):
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} ({k3moe_strerror(status)})")
        self.status = status


def library_path() -> str:
    return _lib_file()


_lib = None


def lib():
    """The loaded libk3moe.so.  Raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is None:
        path = _lib_file()
        if not os.path.exists(path):
            raise ImportError(f"{os.path.basename(path)} is not built ({path}); run "
                              "`python -m sparse_moe_expert_k3moe_gb300.build`")
        L = ctypes.CDLL(path)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        cp = ctypes.POINTER(K3MoEConfig)
        lp, dp = ctypes.POINTER(K3MoELinearConfig), ctypes.POINTER(K3MoEDeltaConfig)
        np, hp, ap = ctypes.POINTER(K3MoENormConfig), ctypes.POINTER(K3MoEHeadLinearConfig), ctypes.POINTER(K3MoELatentConfig)
        sig = {
            "k3moe_strerror": (ctypes.c_char_p, [ctypes.c_int]),
            "k3moe_validate_config": (ctypes.c_int, [cp]),
            "k3moe_packed_bytes": (sz, [cp]),
            "k3moe_workspace_bytes": (ctypes.c_int, [cp, i32, ctypes.POINTER(sz)]),
            "k3moe_pack_mxfp4": (ctypes.c_int, [cp, i32, i32] + [vp] * 6 + [vp, sz, vp, vp]),
            "k3moe_unpack_mxfp4": (ctypes.c_int, [cp, i32, i32, vp, sz] + [vp] * 6 + [vp]),
            "k3moe_route": (ctypes.c_int, [cp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "k3moe_router_scores": (ctypes.c_int, [cp, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
            "k3moe_forward": (ctypes.c_int, [cp, i32, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp, vp,
                                             vp, sz, vp]),
            "k3moe_device_status": (ctypes.c_int, [vp, vp, ctypes.POINTER(i32)]),
            "k3moe_check_wait_timeout": (ctypes.c_int, [vp, i64, vp]),
            "k3moe_check_bounds": (ctypes.c_int, [vp, i32, i32, vp]),
            "k3moe_build_flags": (i32, []),
            "k3moe_forward_noalloc": (ctypes.c_int, [cp, i32, vp, vp, vp, vp, vp, vp, sz, vp, vp,
                                                     vp, vp, vp, vp]),
            "k3moe_full_workspace_bytes": (ctypes.c_int, [cp, ctypes.POINTER(K3MoEFullDims), i32,
                                                          ctypes.POINTER(sz)]),
            "k3moe_full_forward": (ctypes.c_int, [cp, ctypes.POINTER(K3MoEFullDims), i32, vp, vp, vp, vp,
                                                  vp, sz, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                  sz, vp]),
            "k3moe_linear_workspace_bytes": (ctypes.c_int, [lp, i32, ctypes.POINTER(sz)]),
            "k3moe_linear": (ctypes.c_int, [lp, i32, vp, i64, vp, vp, vp, i64, vp, i64, vp, sz, vp]),
            "k3moe_delta_validate_config": (ctypes.c_int, [dp]),
            "k3moe_delta_workspace_bytes": (ctypes.c_int, [dp, i32, i32, ctypes.POINTER(sz)]),
            "k3moe_delta_rule": (ctypes.c_int, [dp, i32, i32, vp, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp,
                                                i32, vp, vp, vp, sz, vp]),
            "k3moe_norm": (ctypes.c_int, [np, i32, vp, i64, vp, i64, vp, vp, i64, vp, vp, i64, vp, vp, i64, vp]),
            "k3moe_head_linear_workspace_bytes": (ctypes.c_int, [hp, i32, ctypes.POINTER(sz)]),
            "k3moe_head_linear": (ctypes.c_int, [hp, i32, vp, i64, i64, vp, vp, i64, i64, vp, sz, vp]),
            "k3moe_latent_validate_config": (ctypes.c_int, [ap]),
            "k3moe_latent_workspace_bytes": (ctypes.c_int, [ap, i32, i32, ctypes.POINTER(sz)]),
            "k3moe_latent_write": (ctypes.c_int, [ap, i32, vp, i64, vp, vp, vp, vp, i64, vp, i32, vp, vp, i64, i64, vp, i64, i64,
                                                  vp, sz, vp]),
            "k3moe_latent_attend": (ctypes.c_int, [ap, i32, i32, vp, vp, i64, i64, vp, i32, vp, i32, vp, vp, vp, vp, sz, vp]),
            "k3moe_latent_prompt": (ctypes.c_int, [ap, i32, i32, i32, vp, vp, vp, i64, i64, vp, i64, i64, vp, i64, vp, vp, vp, sz,
                                                   vp]),
            "k3moe_call": (ctypes.c_int, [ctypes.c_char_p]),
            "k3moe_launch_count": (i64, []),
            "k3moe_set_prefill_gemm": (ctypes.c_int, [i32]),
            "k3moe_get_prefill_gemm": (i32, []),
            "k3moe_timing_enable": (None, [i32]),
            "k3moe_timing_read": (i32, [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(i64),
                                        ctypes.POINTER(ctypes.c_double), i32]),
            "k3moe_timing_reset": (None, []),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


# ----------------------------------------------------------------------------- marshalling helpers

def _ptr(t):
    """Device pointer of a tensor (or None / int passthrough)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(what, rc):
    if rc != K3MOE_OK:
        raise K3MoEError(what, rc)


def k3moe_config(d, f, n_experts, top_k, n_shared, group=32, situ_b1=4.0, situ_b2=25.0,
                 renorm=1, routed_scale=1.0) -> K3MoEConfig:
    return K3MoEConfig(d, f, n_experts, top_k, n_shared, group, situ_b1, situ_b2, renorm,
                       routed_scale)


def k3moe_strerror(status: int) -> str:
    return lib().k3moe_strerror(status).decode()


def k3moe_validate_config(cfg: K3MoEConfig) -> int:
    return lib().k3moe_validate_config(ctypes.byref(cfg))


def k3moe_packed_bytes(cfg: K3MoEConfig) -> int:
    return lib().k3moe_packed_bytes(ctypes.byref(cfg))


def k3moe_workspace_bytes(cfg: K3MoEConfig, T_max: int) -> int:
    out = ctypes.c_size_t(0)
    _check("k3moe_workspace_bytes", lib().k3moe_workspace_bytes(ctypes.byref(cfg), T_max,
                                                                ctypes.byref(out)))
    return out.value


def k3moe_pack_mxfp4(cfg, expert_lo, n_in, w1_packed, w1_scale, w3_packed, w3_scale, w2_packed,
                     w2_scale, table, table_bytes=None, ws=None, stream=None):
    tb = table_bytes if table_bytes is not None else table.numel() * table.element_size()
    _check("k3moe_pack_mxfp4", lib().k3moe_pack_mxfp4(
        ctypes.byref(cfg), expert_lo, n_in, _ptr(w1_packed), _ptr(w1_scale), _ptr(w3_packed),
        _ptr(w3_scale), _ptr(w2_packed), _ptr(w2_scale), _ptr(table), tb, _ptr(ws),
        _stream(stream)))


def k3moe_unpack_mxfp4(cfg, expert_lo, n_out, table, w1_packed, w1_scale, w3_packed, w3_scale,
                       w2_packed, w2_scale, table_bytes=None, stream=None):
    tb = table_bytes if table_bytes is not None else table.numel() * table.element_size()
    _check("k3moe_unpack_mxfp4", lib().k3moe_unpack_mxfp4(
        ctypes.byref(cfg), expert_lo, n_out, _ptr(table), tb, _ptr(w1_packed), _ptr(w1_scale),
        _ptr(w3_packed), _ptr(w3_scale), _ptr(w2_packed), _ptr(w2_scale), _stream(stream)))


def k3moe_router_scores(cfg, T, x, w_router, bias, scores, choice, ws, ws_bytes=None, stream=None):
    wb = ws_bytes if ws_bytes is not None else ws.numel() * ws.element_size()
    _check("k3moe_router_scores", lib().k3moe_router_scores(
        ctypes.byref(cfg), T, _ptr(x), _ptr(w_router), _ptr(bias), _ptr(scores), _ptr(choice),
        _ptr(ws), wb, _stream(stream)))


def k3moe_route(cfg, T, x, w_router, bias, idx, weight, offsets, perm, ws, ws_bytes=None,
                stream=None):
    wb = ws_bytes if ws_bytes is not None else ws.numel() * ws.element_size()
    _check("k3moe_route", lib().k3moe_route(
        ctypes.byref(cfg), T, _ptr(x), _ptr(w_router), _ptr(bias), _ptr(idx), _ptr(weight),
        _ptr(offsets), _ptr(perm), _ptr(ws), wb, _stream(stream)))


def k3moe_forward(cfg, T, x, idx, weight, offsets, perm, expert_table, sh_w1, sh_w3, sh_w2, out,
                  ws, ws_bytes=None, table_bytes=None, stream=None):
    wb = ws_bytes if ws_bytes is not None else ws.numel() * ws.element_size()
    tb = table_bytes if table_bytes is not None else expert_table.numel() * expert_table.element_size()
    _check("k3moe_forward", lib().k3moe_forward(
        ctypes.byref(cfg), T, _ptr(x), _ptr(idx), _ptr(weight), _ptr(offsets), _ptr(perm),
        _ptr(expert_table), tb, _ptr(sh_w1), _ptr(sh_w3), _ptr(sh_w2), _ptr(out), _ptr(ws), wb,
        _stream(stream)))


def k3moe_check_wait_timeout(ws, limit_cycles, stream=None):
    """Runs the library's bounded waits on an mbarrier nothing arrives on, each giving up
    after limit_cycles cycles: sets the timeout bit of ws's status word."""
    _check("k3moe_check_wait_timeout", lib().k3moe_check_wait_timeout(_ptr(ws), int(limit_cycles),
                                                                      _stream(stream)))


def k3moe_check_bounds(ws, index, limit, stream=None):
    """Runs one index check of the kernels' kind on index against [0, limit): a debug
    build records K3MOE_DEV_BOUNDS in ws's status word when it fails."""
    _check("k3moe_check_bounds", lib().k3moe_check_bounds(_ptr(ws), int(index), int(limit), _stream(stream)))


def k3moe_build_flags():
    """BUILD_DEBUG (0x1) when the loaded library was compiled with -DK3MOE_DEBUG."""
    return int(lib().k3moe_build_flags())


BUILD_DEBUG = 0x1


def k3moe_forward_noalloc(cfg, T, x, idx, weight, offsets, perm, expert_table, sh_w1, sh_w3,
                          sh_w2, out, status_out=None, table_bytes=None, stream=None):
    """k3moe_forward with the library's built-in scratch instead of a workspace, for
    callers that cannot allocate device memory; see include/k3moe.h."""
    tb = table_bytes if table_bytes is not None else expert_table.numel() * expert_table.element_size()
    _check("k3moe_forward_noalloc", lib().k3moe_forward_noalloc(
        ctypes.byref(cfg), T, _ptr(x), _ptr(idx), _ptr(weight), _ptr(offsets), _ptr(perm),
        _ptr(expert_table), tb, _ptr(sh_w1), _ptr(sh_w3), _ptr(sh_w2), _ptr(out),
        _ptr(status_out), _stream(stream)))


def k3moe_full_dims(hidden, latent_norm=1, rms_eps=1e-5) -> K3MoEFullDims:
    return K3MoEFullDims(hidden, latent_norm, rms_eps)


def k3moe_full_workspace_bytes(cfg: K3MoEConfig, fd: K3MoEFullDims, T_max: int) -> int:
    out = ctypes.c_size_t(0)
    _check("k3moe_full_workspace_bytes", lib().k3moe_full_workspace_bytes(
        ctypes.byref(cfg), ctypes.byref(fd), T_max, ctypes.byref(out)))
    return out.value


def k3moe_full_forward(cfg, fd, T, h, w_router, bias, w_down, expert_table, norm_gain, w_up, sh_w1,
                       sh_w3, sh_w2, idx, weight, offsets, perm, out, ws, ws_bytes=None,
                       table_bytes=None, stream=None):
    wb = ws_bytes if ws_bytes is not None else ws.numel() * ws.element_size()
    tb = table_bytes if table_bytes is not None else expert_table.numel() * expert_table.element_size()
    _check("k3moe_full_forward", lib().k3moe_full_forward(
        ctypes.byref(cfg), ctypes.byref(fd), T, _ptr(h), _ptr(w_router), _ptr(bias), _ptr(w_down),
        _ptr(expert_table), tb, _ptr(norm_gain), _ptr(w_up), _ptr(sh_w1), _ptr(sh_w3), _ptr(sh_w2),
        _ptr(idx), _ptr(weight), _ptr(offsets), _ptr(perm), _ptr(out), _ptr(ws), wb,
        _stream(stream)))


ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "sigmoid": 4, "logsigmoid": 5}


def k3moe_linear_config(n, k, act="none", y_f32=False) -> K3MoELinearConfig:
    """act: a name of ACTIVATIONS or its number."""
    return K3MoELinearConfig(n, k, ACTIVATIONS[act] if isinstance(act, str) else act, int(y_f32))


def k3moe_linear_workspace_bytes(lc: K3MoELinearConfig, T_max: int) -> int:
    out = ctypes.c_size_t(0)
    _check("k3moe_linear_workspace_bytes", lib().k3moe_linear_workspace_bytes(ctypes.byref(lc), T_max,
                                                                              ctypes.byref(out)))
    return out.value


def k3moe_linear(lc, T, x, x_stride, w, bias, residual, residual_stride, y, y_stride, ws, ws_bytes=None,
                 stream=None):
    wb = ws_bytes if ws_bytes is not None else ws.numel() * ws.element_size()
    _check("k3moe_linear", lib().k3moe_linear(
        ctypes.byref(lc), T, _ptr(x), x_stride, _ptr(w), _ptr(bias), _ptr(residual), residual_stride,
        _ptr(y), y_stride, _ptr(ws), wb, _stream(stream)))


def k3moe_delta_config(n_heads, n_qk_heads, head_dim=128, gate_dim=1, qk_norm=1, norm_eps=1e-6,
                       scale=None) -> K3MoEDeltaConfig:
    """scale: head_dim ** -0.5 when None."""
    return K3MoEDeltaConfig(n_heads, n_qk_heads, head_dim, gate_dim, int(qk_norm), norm_eps,
                            scale if scale is not None else max(head_dim, 1) ** -0.5)


def k3moe_delta_validate_config(dc: K3MoEDeltaConfig) -> int:
    return lib().k3moe_delta_validate_config(ctypes.byref(dc))


def k3moe_delta_workspace_bytes(dc: K3MoEDeltaConfig, n_seq_max: int, T_max: int) -> int:
    out = ctypes.c_size_t(0)
    _check("k3moe_delta_workspace_bytes", lib().k3moe_delta_workspace_bytes(
        ctypes.byref(dc), n_seq_max, T_max, ctypes.byref(out)))
    return out.value


def k3moe_delta_rule(dc, n_seq, T, seq_start, q, q_stride, k, k_stride, v, v_stride, g, beta, state_in,
                     state_out, n_slots, slots, out, ws, ws_bytes=None, stream=None):
    wb = ws_bytes if ws_bytes is not None else ws.numel() * ws.element_size()
    _check("k3moe_delta_rule", lib().k3moe_delta_rule(
        ctypes.byref(dc), n_seq, T, _ptr(seq_start), _ptr(q), q_stride, _ptr(k), k_stride, _ptr(v),
        v_stride, _ptr(g), _ptr(beta), _ptr(state_in), _ptr(state_out), n_slots, _ptr(slots), _ptr(out),
        _ptr(ws), wb, _stream(stream)))


GATES = {"none": 0, "sigmoid": 1, "silu": 2}


def k3moe_norm_config(n, group=0, post_norm=1, pre_norm=1, gate="none", x_f32=False, sum_f32=False, eps=1e-6,
                      alpha=1.0) -> K3MoENormConfig:
    """group: n when 0; gate: a name of GATES or its number."""
    return K3MoENormConfig(n, group or n, int(post_norm), int(pre_norm), GATES[gate] if isinstance(gate, str) else gate, int(x_f32),
                           int(sum_f32), eps, alpha)


def k3moe_norm(nc, T, x, x_stride, gate, gate_stride, post_gain, residual, residual_stride, scale, total, total_stride, pre_gain, out,
               out_stride, stream=None):
    _check("k3moe_norm", lib().k3moe_norm(
        ctypes.byref(nc), T, _ptr(x), x_stride, _ptr(gate), gate_stride, _ptr(post_gain), _ptr(residual), residual_stride, _ptr(scale),
        _ptr(total), total_stride, _ptr(pre_gain), _ptr(out), out_stride, _stream(stream)))


def k3moe_head_linear_config(n_heads, n, k) -> K3MoEHeadLinearConfig:
    return K3MoEHeadLinearConfig(n_heads, n, k)


def k3moe_head_linear_workspace_bytes(hc: K3MoEHeadLinearConfig, T_max: int) -> int:
    out = ctypes.c_size_t(0)
    _check("k3moe_head_linear_workspace_bytes", lib().k3moe_head_linear_workspace_bytes(ctypes.byref(hc), T_max, ctypes.byref(out)))
    return out.value


def k3moe_head_linear(hc, T, x, x_stride, x_head_stride, w, y, y_stride, y_head_stride, ws, ws_bytes=None, stream=None):
    wb = ws_bytes if ws_bytes is not None else ws.numel() * ws.element_size()
    _check("k3moe_head_linear", lib().k3moe_head_linear(
        ctypes.byref(hc), T, _ptr(x), x_stride, x_head_stride, _ptr(w), _ptr(y), y_stride, y_head_stride, _ptr(ws), wb, _stream(stream)))


ROPES = {"none": 0, "pairs": 1, "halves": 2}


def k3moe_latent_config(n_heads, rank=512, rope_dim=64, key_dim=128, value_dim=128, page_size=64, rope="pairs", norm=1, norm_eps=1e-6,
                        scale=None, causal=1) -> K3MoELatentConfig:
    """rope: a name of ROPES or its number; scale: (key_dim + rope_dim) ** -0.5 when None."""
    return K3MoELatentConfig(n_heads, rank, rope_dim, key_dim, value_dim, page_size, ROPES[rope] if isinstance(rope, str) else rope,
                             int(norm), norm_eps, scale if scale is not None else max(key_dim + rope_dim, 1) ** -0.5, int(causal))


def k3moe_latent_validate_config(lc: K3MoELatentConfig) -> int:
    return lib().k3moe_latent_validate_config(ctypes.byref(lc))


def k3moe_latent_workspace_bytes(lc: K3MoELatentConfig, n_seq_max: int, T_max: int) -> int:
    out = ctypes.c_size_t(0)
    _check("k3moe_latent_workspace_bytes", lib().k3moe_latent_workspace_bytes(ctypes.byref(lc), n_seq_max, T_max, ctypes.byref(out)))
    return out.value


def k3moe_latent_write(lc, T, c, c_stride, gain, positions, inv_freq, rows, rows_stride, cache, n_pages, slots, q, q_stride, q_head_stride,
                       q_rope, q_rope_stride, q_rope_head_stride, ws, ws_bytes=None, stream=None):
    wb = ws_bytes if ws_bytes is not None else ws.numel() * ws.element_size()
    _check("k3moe_latent_write", lib().k3moe_latent_write(
        ctypes.byref(lc), T, _ptr(c), c_stride, _ptr(gain), _ptr(positions), _ptr(inv_freq), _ptr(rows), rows_stride, _ptr(cache), n_pages,
        _ptr(slots), _ptr(q), q_stride, q_head_stride, _ptr(q_rope), q_rope_stride, q_rope_head_stride, _ptr(ws), wb, _stream(stream)))


def k3moe_latent_attend(lc, n_seq, T, seq_start, q, q_stride, q_head_stride, cache, n_pages, pages, max_pages, kv_len, out, lse, ws,
                        ws_bytes=None, stream=None):
    wb = ws_bytes if ws_bytes is not None else ws.numel() * ws.element_size()
    _check("k3moe_latent_attend", lib().k3moe_latent_attend(
        ctypes.byref(lc), n_seq, T, _ptr(seq_start), _ptr(q), q_stride, q_head_stride, _ptr(cache), n_pages, _ptr(pages), max_pages,
        _ptr(kv_len), _ptr(out), _ptr(lse), _ptr(ws), wb, _stream(stream)))


def k3moe_latent_prompt(lc, n_seq, T, S, seq_start, kv_start, q, q_stride, q_head_stride, kv, kv_stride, kv_head_stride, rope_key,
                        rope_stride, out, lse, ws, ws_bytes=None, stream=None):
    wb = ws_bytes if ws_bytes is not None else ws.numel() * ws.element_size()
    _check("k3moe_latent_prompt", lib().k3moe_latent_prompt(
        ctypes.byref(lc), n_seq, T, S, _ptr(seq_start), _ptr(kv_start), _ptr(q), q_stride, q_head_stride, _ptr(kv), kv_stride,
        kv_head_stride, _ptr(rope_key), rope_stride, _ptr(out), _ptr(lse), _ptr(ws), wb, _stream(stream)))


def k3moe_device_status(ws, stream=None):
    """(status, code): synchronises the stream, reads and clears the device status word."""
    code = ctypes.c_int32(0)
    rc = lib().k3moe_device_status(_ptr(ws), _stream(stream), ctypes.byref(code))
    return rc, code.value


def k3moe_launch_count() -> int:
    return lib().k3moe_launch_count()


PREFILL_GEMM_DEFAULT, PREFILL_GEMM_F16, PREFILL_GEMM_BLOCK_SCALED = 0, 1, 2


def k3moe_set_prefill_gemm(variant: int):
    """The kernel of the routed gate/up projection on the prefill path: PREFILL_GEMM_F16
    (dequantised weights), PREFILL_GEMM_BLOCK_SCALED (kind::mxf8f6f4 on the packed codes
    and scales) or PREFILL_GEMM_DEFAULT; process-wide."""
    _check("k3moe_set_prefill_gemm", lib().k3moe_set_prefill_gemm(int(variant)))


def k3moe_get_prefill_gemm() -> int:
    return int(lib().k3moe_get_prefill_gemm())


def k3moe_timing_enable(on: bool):
    lib().k3moe_timing_enable(1 if on else 0)


def k3moe_timing_read() -> dict:
    L = lib()
    n = L.k3moe_timing_read(None, None, None, 0)
    names = (ctypes.c_char_p * max(n, 1))()
    launches = (ctypes.c_int64 * max(n, 1))()
    ms = (ctypes.c_double * max(n, 1))()
    n = L.k3moe_timing_read(names, launches, ms, n)
    return {names[i].decode(): (launches[i], ms[i]) for i in range(n)}


def k3moe_timing_reset():
    lib().k3moe_timing_reset()


# ----------------------------------------------------------------------------- convenience holders

def _capture(call, x, out):
    """call(x, out) recorded as a CUDA graph on x's device.  One eager call on a side
    stream first settles the library's cached launch attributes and GEMM plans, so that
    capture itself only enqueues work.  The graph reads x and writes out, the routing
    buffers and the workspace where they are now: copy the next tokens into x, then
    replay().  The library's launches keep their programmatic dependencies as graph edges."""
    import torch
    cur = torch.cuda.current_stream(x.device)
    side = torch.cuda.Stream(device=x.device)
    side.wait_stream(cur)
    with torch.cuda.stream(side):
        call(x, out)
    cur.wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(x, out)
    return g


class MoELayer:
    """Holds one layer's device tensors (packed expert table, router, bias,
    shared experts) and a workspace, and calls k3moe_route + k3moe_forward.
    Allocation is torch's; every computation is the library's."""

    def __init__(self, cfg: K3MoEConfig, T_max: int, device="cuda"):
        import torch
        self.cfg = cfg
        self.device = torch.device(device)
        self.T_max = T_max
        self.table = torch.empty(k3moe_packed_bytes(cfg), dtype=torch.uint8, device=self.device)
        self.ws_bytes = k3moe_workspace_bytes(cfg, T_max)
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self.w_router = None
        self.bias = None
        self.sh_w1 = self.sh_w3 = self.sh_w2 = None
        E, k = cfg.n_experts, cfg.top_k
        self.idx = torch.empty((T_max, k), dtype=torch.int32, device=self.device)
        self.weight = torch.empty((T_max, k), dtype=torch.float32, device=self.device)
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device=self.device)
        self.perm = torch.empty(T_max * k, dtype=torch.int32, device=self.device)

    def pack_experts(self, expert_lo, n, w1_packed, w1_scale, w3_packed, w3_scale, w2_packed,
                     w2_scale, stream=None):
        k3moe_pack_mxfp4(self.cfg, expert_lo, n, w1_packed, w1_scale, w3_packed, w3_scale,
                         w2_packed, w2_scale, self.table, ws=self.ws, stream=stream)

    def route(self, x, stream=None):
        T = x.shape[0]
        k3moe_route(self.cfg, T, x, self.w_router, self.bias, self.idx, self.weight, self.offsets,
                    self.perm, self.ws, self.ws_bytes, stream)

    def scores(self, x, stream=None):
        """(sc, ch) [T][E] f32 device tensors: the router scores k3moe_route selects from."""
        import torch
        T = x.shape[0]
        sc = torch.empty((T, self.cfg.n_experts), dtype=torch.float32, device=self.device)
        ch = torch.empty_like(sc)
        k3moe_router_scores(self.cfg, T, x, self.w_router, self.bias, sc, ch, self.ws, self.ws_bytes,
                            stream)
        return sc, ch

    def forward(self, x, out, stream=None, routing=None):
        T = x.shape[0]
        idx, weight, offsets, perm = routing or (self.idx, self.weight, self.offsets, self.perm)
        k3moe_forward(self.cfg, T, x, idx, weight, offsets, perm, self.table, self.sh_w1,
                      self.sh_w3, self.sh_w2, out, self.ws, self.ws_bytes, stream=stream)

    def __call__(self, x, out, stream=None):
        self.route(x, stream)
        self.forward(x, out, stream)
        return out

    def capture(self, x, out):
        """Record route + forward on the fixed buffers x [T][d] bf16 and out [T][d] f32 as
        a CUDA graph and return the torch.cuda.CUDAGraph (see _capture)."""
        return _capture(self, x, out)


class MoEBlock:
    """Holds one full-width block's device tensors (the routed experts' packed table,
    the full-width router, the down and up projections, the norm gain and the fused
    shared experts) and a workspace, and calls k3moe_full_forward.  Allocation is
    torch's; every computation is the library's."""

    def __init__(self, cfg: K3MoEConfig, fd: K3MoEFullDims, T_max: int, device="cuda"):
        import torch
        self.cfg, self.fd = cfg, fd
        self.device = torch.device(device)
        self.T_max = T_max
        self.table = torch.empty(k3moe_packed_bytes(cfg), dtype=torch.uint8, device=self.device)
        self.ws_bytes = k3moe_full_workspace_bytes(cfg, fd, T_max)
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self.w_router = self.bias = self.w_down = self.w_up = self.gain = None
        self.sh_w1 = self.sh_w3 = self.sh_w2 = None
        E, k = cfg.n_experts, cfg.top_k
        self.idx = torch.empty((T_max, k), dtype=torch.int32, device=self.device)
        self.weight = torch.empty((T_max, k), dtype=torch.float32, device=self.device)
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device=self.device)
        self.perm = torch.empty(T_max * k, dtype=torch.int32, device=self.device)

    def pack_experts(self, expert_lo, n, w1_packed, w1_scale, w3_packed, w3_scale, w2_packed,
                     w2_scale, stream=None):
        k3moe_pack_mxfp4(self.cfg, expert_lo, n, w1_packed, w1_scale, w3_packed, w3_scale,
                         w2_packed, w2_scale, self.table, ws=self.ws, stream=stream)

    def forward(self, h, out, stream=None):
        T = h.shape[0]
        k3moe_full_forward(self.cfg, self.fd, T, h, self.w_router, self.bias, self.w_down,
                           self.table, self.gain, self.w_up, self.sh_w1, self.sh_w3, self.sh_w2,
                           self.idx, self.weight, self.offsets, self.perm, out, self.ws,
                           self.ws_bytes, stream=stream)
        return out

    __call__ = forward

    def capture(self, h, out):
        """k3moe_full_forward on the fixed buffers h [T][H] and out [T][H] as a CUDA graph
        (see _capture)."""
        return _capture(self, h, out)


# ----------------------------------------------------------------------------- the token mixer's holders

def _fits(t, dtypes, shape, index):
    """Whether t has this shape, one of dtypes and is on the device of this index (-1: the host)."""
    return t.dtype in dtypes and t.shape == shape and t.get_device() == index


def _require(what, t, dtypes, shape, index, rows=False):
    """Raises ValueError unless t fits and is contiguous (rows: each of its rows is, with any
    stride between them): what the entry points take on trust from a pointer.  Returns the
    elements from a row to the next."""
    if not _fits(t, dtypes, shape, index):
        raise ValueError(f"{what}: {t.dtype} {tuple(t.shape)} on {t.device}, expected "
                         f"{' or '.join(str(d) for d in dtypes)} {tuple(shape)} on "
                         f"{'the host' if index < 0 else f'cuda:{index}'}")
    row = 1
    for n, s in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if n > 1 and s != row:
            break
        row *= n
    else:
        if shape[0] <= 1 or t.is_contiguous():
            return row
        if rows:
            return t.stride(0)
    raise ValueError(f"{what}: strides {tuple(t.stride())} of shape {tuple(shape)} are not dense")


def _device(device):
    """(torch.device with its index, index or -1 for the host)."""
    import torch
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device, device.index if device.type == "cuda" else -1


def _current_stream(index):
    """A function that returns the handle of the device's current stream: torch's own one
    without the Stream object around it, where it has that."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return lambda: raw(index)
    return lambda: torch.cuda.current_stream(index).cuda_stream


def _handle(stream):
    return stream if isinstance(stream, int) else stream.cuda_stream


class Linear:
    """One projection y = act(x W^T + bias) + residual (k3moe_linear): holds the weights w
    [n][k] bf16 and the bias [n] f32 or None, both set by the caller, and a workspace."""

    def __init__(self, lc: K3MoELinearConfig, T_max: int, device="cuda"):
        import torch
        self.lc = lc
        self.device, self._index = _device(device)
        self.T_max = T_max
        self.w = self.bias = None
        self.ws_bytes = k3moe_linear_workspace_bytes(lc, T_max)
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self._bf16, self._f32 = (torch.bfloat16, torch.int16), (torch.float32,)
        self._n, self._k, self._ytype = lc.n, lc.k, self._f32 if lc.y_f32 else self._bf16
        self._lc, self._call, self._current = ctypes.byref(lc), lib().k3moe_linear, _current_stream(self._index)

    def _rows(self, what, t, types, shape):
        """The row stride of x, y or the residual."""
        if t.dtype in types and t.shape == shape and t.get_device() == self._index:
            if t.is_contiguous():
                return shape[1]
            if t.stride(1) == 1 and shape[0] > 1:
                return t.stride(0)
        return _require(what, t, types, shape, self._index, True)

    def __call__(self, x, y, residual=None, stream=None):
        """x [T][k] bf16 (rows may be slices of wider ones), y [T][n] written and returned;
        residual [T][n] of y's type, which may be y."""
        T, n, k, dev, w, bias = x.shape[0], self._n, self._k, self._index, self.w, self.bias
        if T > self.T_max:
            raise ValueError(f"x: {T} rows, the holder is for {self.T_max}")
        xs = self._rows("x", x, self._bf16, (T, k))
        ys = self._rows("y", y, self._ytype, (T, n))
        if not (w.dtype in self._bf16 and w.shape == (n, k) and w.get_device() == dev and w.is_contiguous()):
            _require("w", w, self._bf16, (n, k), dev)
        rs = 0
        if residual is not None:
            rs = ys if residual is y else self._rows("residual", residual, self._ytype, (T, n))
        if bias is not None and not (
                bias.dtype in self._f32 and bias.shape == (n,) and bias.get_device() == dev and bias.is_contiguous()):
            _require("bias", bias, self._f32, (n,), dev)
        if T:
            st = self._call(self._lc, T, x.data_ptr(), xs, w.data_ptr(), None if bias is None else bias.data_ptr(),
                            None if residual is None else residual.data_ptr(), rs, y.data_ptr(), ys, self.ws.data_ptr(),
                            self.ws_bytes, self._current() if stream is None else _handle(stream))
            if st:
                _check("k3moe_linear", st)
        return y


class DeltaRule:
    """The gated delta rule (k3moe_delta_rule) for up to n_seq_max sequences and T_max tokens
    a call: holds its workspace; the states are the caller's."""

    def __init__(self, dc: K3MoEDeltaConfig, n_seq_max: int, T_max: int, device="cuda"):
        import torch
        self.dc = dc
        self.device, self._index = _device(device)
        self.n_seq_max, self.T_max = n_seq_max, T_max
        self.ws_bytes = k3moe_delta_workspace_bytes(dc, n_seq_max, T_max)
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self._bf16, self._f32, self._i32 = (torch.bfloat16, torch.int16), (torch.float32,), (torch.int32,)
        self._H, self._Hq, self._D, self._G = dc.n_heads, dc.n_qk_heads, dc.head_dim, dc.gate_dim
        self._dc, self._call, self._current = ctypes.byref(dc), lib().k3moe_delta_rule, _current_stream(self._index)

    def new_state(self, n_slots):
        """A zeroed pool of n_slots states [n_slots][n_heads][head_dim][head_dim] f32."""
        import torch
        return torch.zeros((n_slots, self._H, self._D, self._D), dtype=torch.float32, device=self.device)

    def _rows(self, what, t, shape):
        """The row stride of q, k or v."""
        if t.dtype in self._bf16 and t.shape == shape and t.get_device() == self._index:
            s = t.stride()
            if s[2] == 1 and s[1] == self._D:
                return s[0] if shape[0] > 1 else shape[1] * self._D
        return _require(what, t, self._bf16, shape, self._index, True)

    def __call__(self, q, k, v, g, beta, out, state_in, state_out, seq_start=None, slots=None, stream=None):
        """q, k [T][n_qk_heads][D], v [T][n_heads][D] bf16, whose rows may be slices of wider
        ones; g [T][n_heads][gate_dim], beta [T][n_heads] f32; out [T][n_heads][D] bf16,
        written and returned; state_in (None: zeros) and state_out [slots][n_heads][D][D] f32,
        which may be the same; slots [n_seq] int32 or None (sequence i in slot i); seq_start
        [n_seq+1] int32, or None for one token each (with one slot: one sequence)."""
        T, H, D, dev = q.shape[0], self._H, self._D, self._index
        f32, i32 = self._f32, self._i32
        qs = self._rows("q", q, (T, self._Hq, D))
        ks = self._rows("k", k, (T, self._Hq, D))
        vs = self._rows("v", v, (T, H, D))
        n_slots = state_out.shape[0]
        pool = (n_slots, H, D, D)
        n_seq = seq_start.shape[0] - 1 if seq_start is not None else slots.shape[0] if slots is not None else T
        # one line a tensor: what _require says at length when it does not hold
        if not (g.dtype in f32 and g.shape == (T, H, self._G) and g.get_device() == dev and g.is_contiguous()):
            _require("g", g, f32, (T, H, self._G), dev)
        if not (beta.dtype in f32 and beta.shape == (T, H) and beta.get_device() == dev and beta.is_contiguous()):
            _require("beta", beta, f32, (T, H), dev)
        if not (out.dtype in self._bf16 and out.shape == (T, H, D) and out.get_device() == dev and out.is_contiguous()):
            _require("out", out, self._bf16, (T, H, D), dev)
        if not (state_out.dtype in f32 and state_out.shape == pool and state_out.get_device() == dev and state_out.is_contiguous()):
            _require("state_out", state_out, f32, pool, dev)
        if state_in is not None and state_in is not state_out and not (
                state_in.dtype in f32 and state_in.shape == pool and state_in.get_device() == dev and state_in.is_contiguous()):
            _require("state_in", state_in, f32, pool, dev)
        if seq_start is not None and not (
                seq_start.dtype in i32 and seq_start.dim() == 1 and seq_start.get_device() == dev and seq_start.is_contiguous()):
            _require("seq_start", seq_start, i32, (n_seq + 1,), dev)
        if slots is not None and not (
                slots.dtype in i32 and slots.shape == (n_seq,) and slots.get_device() == dev and slots.is_contiguous()):
            _require("slots", slots, i32, (n_seq,), dev)
        if n_seq > self.n_seq_max or T > self.T_max:
            raise ValueError(f"{n_seq} sequences of {T} tokens, the holder is for {self.n_seq_max} and {self.T_max}")
        st = self._call(
            self._dc, n_seq, T, None if seq_start is None else seq_start.data_ptr(), q.data_ptr(), qs, k.data_ptr(), ks,
            v.data_ptr(), vs, g.data_ptr(), beta.data_ptr(), None if state_in is None else state_in.data_ptr(),
            state_out.data_ptr(), n_slots, None if slots is None else slots.data_ptr(), out.data_ptr(),
            self.ws.data_ptr(), self.ws_bytes, self._current() if stream is None else _handle(stream))
        if st:
            _check("k3moe_delta_rule", st)
        return out


# ----------------------------------------------------------------------------- the latent attention's holders

# One line a tensor where it fits, in a function that returns what the entry point takes; what does not hold is said at
# length by _require.

def _dense(what, t, types, shape, index):
    """The pointer of a contiguous tensor, or 0 for None."""
    if t is None:
        return 0
    if t.dtype in types and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    _require(what, t, types, shape, index)
    return t.data_ptr()


def _rowed(what, t, types, shape, index):
    """(pointer, row stride) of a tensor whose rows may be slices of wider ones, or (0, n) for None."""
    if t is None:
        return 0, shape[1]
    if t.dtype in types and t.shape == shape and t.get_device() == index:
        if shape[0] <= 1:
            if shape[1] <= 1 or t.stride(1) == 1:
                return t.data_ptr(), shape[1]
        else:
            s0, s1 = t.stride()
            if s1 == 1:
                return t.data_ptr(), s0
    return t.data_ptr(), _require(what, t, types, shape, index, True)


def _headed(what, t, types, shape, index):
    """(pointer, stride from token to token, from head to head) of t [T][heads][columns], whose heads may be columns of
    wider ones, or (0, 0, 0) for None."""
    if t is None:
        return 0, 0, 0
    T, H, n = shape
    if t.dtype in types and t.shape == shape and t.get_device() == index:
        ts, hs, es = t.stride()
        if es == 1 or n <= 1:
            if H <= 1:
                hs = n                                     # of one head, of one token: whatever its stride says
            return t.data_ptr(), ts if T > 1 else (H - 1) * hs + (n + 7) // 8 * 8, hs
        raise ValueError(f"{what}: strides {tuple(t.stride())} of shape {tuple(shape)}: columns are not dense")
    _require(what, t, types, shape, index)                  # says what is wrong
    return t.data_ptr(), 0, 0


class _Holder:
    """What the holders below share: a device, its current stream and, where asked for, a workspace; and the config, which the
    entry point reads at each call: _read takes from it what the tensors' checks need, again whenever it has changed."""

    def _init(self, device, ws_bytes=0):
        import torch
        self.device, self._index = _device(device)
        self._bf16, self._f32, self._i32 = (torch.bfloat16, torch.int16), (torch.float32,), (torch.int32,)
        self._current, self._on = _current_stream(self._index), torch.cuda.device
        self._device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        self._words = lib().k3moe_call
        self.ws_bytes = ws_bytes
        self.ws = torch.zeros(ws_bytes, dtype=torch.uint8, device=self.device) if ws_bytes else None
        if ws_bytes and self._index >= 0 and not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self._index).synchronize()    # the zeros are there before a call on any other stream

    def _follow(self, config):
        self._config, self._at = config, ctypes.addressof(config)
        self._bytes, self._seen = (ctypes.c_char * ctypes.sizeof(config)).from_buffer(config), None

    def _entry(self, entry, name, n):
        """What _run calls: one of k3moe.h's k3moe_entry, its name and its n arguments.  They go as one string of words:
        converted one by one twenty of them took longer than the launch (4.3 us; 1.6 us packed)."""
        return struct.Struct(f"<{n + 2}q").pack, entry, n, name

    def _run(self, entry, args, stream):
        """The entry's call with args and the stream, on the holder's device, whichever is the current one."""
        pack, number, n, name = entry
        if self._index >= 0 and self._device_now() != self._index:
            with self._on(self._index):
                st = self._words(pack(number, n, *args, self._current() if stream is None else _handle(stream)))
        else:
            st = self._words(pack(number, n, *args, self._current() if stream is None else _handle(stream)))
        if st:
            _check(name, st)


class Norm(_Holder):
    """The norms after a block and before the next with the block's gate and residual scale (k3moe_norm): holds
    post_gain [group], scale [n] or None and pre_gain [n], f32, set by the caller."""

    def __init__(self, nc: K3MoENormConfig, device="cuda"):
        self._init(device)
        self.nc = nc
        self.post_gain = self.scale = self.pre_gain = None
        self._follow(nc)
        self._norm = self._entry(0, "k3moe_norm", 16)

    def _read(self):
        nc, self._seen = self._config, self._bytes.raw
        self._n, self._group = (nc.n,), (nc.group,)
        self._xtype, self._stype = self._f32 if nc.x_f32 else self._bf16, self._f32 if nc.sum_f32 else self._bf16

    def __call__(self, x, out=None, gate=None, residual=None, total=None, stream=None):
        """x [T][n] by x_f32; gate [T][n] bf16; residual and total [T][n] by sum_f32; out [T][n] bf16; rows may be
        slices of wider ones.  Returns out, or total where nothing is normed for the next block."""
        if self._bytes.raw != self._seen:
            self._read()
        dev, bf16, f32, stype = self._index, self._bf16, self._f32, self._stype
        T = x.shape[0]
        shape = (T, self._n[0])
        post, scale = _dense("post_gain", self.post_gain, f32, self._group, dev), _dense("scale", self.scale, f32, self._n, dev)
        pre = _dense("pre_gain", self.pre_gain, f32, self._n, dev)
        xp, xs = _rowed("x", x, self._xtype, shape, dev)
        gp, gs = _rowed("gate", gate, bf16, shape, dev)
        rp, rs = _rowed("residual", residual, stype, shape, dev)
        tp, ts = (rp, rs) if total is residual else _rowed("total", total, stype, shape, dev)
        op, os_ = _rowed("out", out, bf16, shape, dev)
        if T:
            self._run(self._norm, (self._at, T, xp, xs, gp, gs, post, rp, rs, scale, tp, ts, pre, op, os_), stream)
        return total if out is None else out


class HeadLinear(_Holder):
    """Every head's own projection (k3moe_head_linear): holds the weights w [n_heads][n][k] bf16, set by
    the caller, and a workspace."""

    def __init__(self, hc: K3MoEHeadLinearConfig, T_max: int, device="cuda"):
        self._init(device, k3moe_head_linear_workspace_bytes(hc, T_max))
        self.hc, self.T_max, self.w = hc, T_max, None
        self._follow(hc)
        self._linear = self._entry(1, "k3moe_head_linear", 12)

    def _read(self):
        hc, self._seen = self._config, self._bytes.raw
        self._shape = (hc.n_heads, hc.n, hc.k)

    def __call__(self, x, y, stream=None):
        """x [T][n_heads][k] bf16, y [T][n_heads][n] bf16 written and returned; heads may be columns of wider ones."""
        T, dev, bf16 = x.shape[0], self._index, self._bf16
        if self._bytes.raw != self._seen:
            self._read()
        H, n, k = self._shape
        if T > self.T_max:
            raise ValueError(f"x: {T} tokens, the holder is for {self.T_max}")
        xp, xs, xh = _headed("x", x, bf16, (T, H, k), dev)
        yp, ys, yh = _headed("y", y, bf16, (T, H, n), dev)
        w = _dense("w", self.w, bf16, self._shape, dev)
        if T:
            self._run(self._linear, (self._at, T, xp, xs, xh, w, yp, ys, yh, self.ws.data_ptr(), self.ws_bytes), stream)
        return y


class LatentAttention(_Holder):
    """The latent cache's write and attention over it (k3moe_latent_write, _attend, _prompt), for up to n_seq_max
    sequences and T_max query tokens a call: holds gain [rank] f32 and inv_freq [rope_dim / 2] f64, set by the caller, and
    a workspace; the cache is the caller's.  Calls and captured graphs of one holder share its workspace: one stream at a time has
    them, and the holder is kept until they are done."""

    def __init__(self, lc: K3MoELatentConfig, n_seq_max: int, T_max: int, device="cuda"):
        import torch
        self._init(device, k3moe_latent_workspace_bytes(lc, n_seq_max, T_max))
        self.lc, self.n_seq_max, self.T_max = lc, n_seq_max, T_max
        self.gain = self.inv_freq = None
        self._i64, self._f64 = (torch.int64,), (torch.float64,)
        # the columns are what every config has to have
        self._C, self._R, self._row = lc.rank, lc.rope_dim, lc.rank + lc.rope_dim
        self._kr, self._kv, self._v = lc.key_dim + lc.rope_dim, lc.key_dim + lc.value_dim, lc.value_dim
        self._follow(lc)
        self._write, self._attend = self._entry(2, "k3moe_latent_write", 21), self._entry(3, "k3moe_latent_attend", 17)
        self._prompt = self._entry(4, "k3moe_latent_prompt", 19)

    def _read(self):
        self._seen, self._H, self._page = self._bytes.raw, self._config.n_heads, self._config.page_size

    def new_cache(self, n_pages):
        """A zeroed cache of n_pages pages [n_pages][page_size][rank + rope_dim] bf16."""
        import torch
        self._read()
        return torch.zeros((n_pages, self._page, self._row), dtype=torch.bfloat16, device=self.device)

    def _room(self, n_seq, T):
        if n_seq > self.n_seq_max or T > self.T_max:
            raise ValueError(f"{n_seq} sequences of {T} tokens, the holder is for {self.n_seq_max} and {self.T_max}")

    def write(self, c, positions=None, cache=None, slots=None, rows=None, q=None, q_rope=None, stream=None):
        """c [T][rank + rope_dim] bf16, positions [T] int32; the rows go to slots [T] int64 of the cache and to rows
        [T][rank + rope_dim]; q [T][n_heads][rope_dim], the queries' rotated columns, to q_rope, which may be q.  Returns
        rows, or the cache where they go there alone."""
        if self._bytes.raw != self._seen:
            self._read()
        dev, bf16, T, row = self._index, self._bf16, c.shape[0], self._row
        if T > self.T_max:
            raise ValueError(f"c: {T} tokens, the holder is for {self.T_max}")
        cp, cs = _rowed("c", c, bf16, (T, row), dev)
        gain = _dense("gain", self.gain, self._f32, (self._C,), dev)
        freq = _dense("inv_freq", self.inv_freq, self._f64, (self._R // 2,), dev)
        at = _dense("positions", positions, self._i32, (T,), dev)
        rp, rs = (cp, cs) if rows is c else _rowed("rows", rows, bf16, (T, row), dev)
        n_pages = 0 if cache is None else cache.shape[0]
        pool = _dense("cache", cache, bf16, (n_pages, self._page, row), dev)
        sl = _dense("slots", slots, self._i64, (T,), dev)
        shape = (T, self._H, self._R)
        qp, qs, qh = _headed("q", q, bf16, shape, dev)
        op, os_, oh = (qp, qs, qh) if q_rope is q else _headed("q_rope", q_rope, bf16, shape, dev)
        if T:
            self._run(self._write, (self._at, T, cp, cs, gain, at, freq, rp, rs, pool, n_pages, sl, qp, qs, qh, op, os_, oh,
                      self.ws.data_ptr(), self.ws_bytes), stream)
        return cache if rows is None else rows

    def attend(self, q, cache, pages, kv_len, out, seq_start=None, lse=None, stream=None):
        """q [T][n_heads][rank + rope_dim] bf16, pages [n_seq][max_pages] int32, kv_len [n_seq] int32; out
        [T][n_heads][rank] bf16 written and returned, lse [T][n_heads] f32 or None; seq_start [n_seq+1] int32, or None for
        one token each (with one sequence: all)."""
        if self._bytes.raw != self._seen:
            self._read()
        dev, bf16, i32, T, n_seq, H = self._index, self._bf16, self._i32, q.shape[0], kv_len.shape[0], self._H
        self._room(n_seq, T)
        qp, qs, qh = _headed("q", q, bf16, (T, H, self._row), dev)
        n_pages, max_pages = cache.shape[0], pages.shape[-1]
        pool = _dense("cache", cache, bf16, (n_pages, self._page, self._row), dev)
        table, lens = _dense("pages", pages, i32, (n_seq, max_pages), dev), _dense("kv_len", kv_len, i32, (n_seq,), dev)
        o, start = _dense("out", out, bf16, (T, H, self._C), dev), _dense("seq_start", seq_start, i32, (n_seq + 1,), dev)
        ls = _dense("lse", lse, self._f32, (T, H), dev)
        if T:
            self._run(self._attend, (self._at, n_seq, T, start, qp, qs, qh, pool, n_pages, table, max_pages, lens, o, ls,
                      self.ws.data_ptr(), self.ws_bytes), stream)
        return out

    def prompt(self, q, kv, rope_key, out, seq_start=None, kv_start=None, lse=None, stream=None):
        """q [T][n_heads][key_dim + rope_dim], kv [S][n_heads][key_dim + value_dim], rope_key [S][rope_dim] bf16, the last's
        rows at any stride; out [T][n_heads][value_dim] bf16 written and returned, lse [T][n_heads] f32 or None; seq_start and
        kv_start [n_seq+1] int32, or None: one sequence, or the queries' own."""
        if self._bytes.raw != self._seen:
            self._read()
        dev, bf16, i32, T, S, H = self._index, self._bf16, self._i32, q.shape[0], kv.shape[0], self._H
        n_seq = 1 if seq_start is None else seq_start.shape[0] - 1
        self._room(n_seq, T)
        qp, qs, qh = _headed("q", q, bf16, (T, H, self._kr), dev)
        kp, ks, kh = _headed("kv", kv, bf16, (S, H, self._kv), dev)
        rp, rs = _rowed("rope_key", rope_key, bf16, (S, self._R), dev)
        o, ls = _dense("out", out, bf16, (T, H, self._v), dev), _dense("lse", lse, self._f32, (T, H), dev)
        start, keys = _dense("seq_start", seq_start, i32, (n_seq + 1,), dev), _dense("kv_start", kv_start, i32, (n_seq + 1,), dev)
        if T:
            self._run(self._prompt, (self._at, n_seq, T, S, start, keys, qp, qs, qh, kp, ks, kh, rp, rs, o, ls,
                      self.ws.data_ptr(), self.ws_bytes), stream)
        return out
