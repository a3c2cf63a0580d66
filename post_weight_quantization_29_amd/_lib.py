"""ctypes binding of libgptq.so: the C-ABI calls under the same names.

Argument marshalling only: torch tensors are passed as device pointers and the
current HIP stream; every step runs in the library's kernels.  Workspaces are
allocated through torch when the caller does not pass one.  There is no CPU
fallback: a missing library raises immediately.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("GPTQ_MI355X_LIB", os.path.join(_PKG, "libgptq.so"))

GPTQ_F32, GPTQ_F16, GPTQ_BF16 = 0, 1, 2
OK, ERR_INVALID_ARG, ERR_NOT_PD, ERR_HIP, ERR_WORKSPACE, ERR_UNSUPPORTED = 0, -1, -2, -3, -4, -5

_DTYPE = {torch.float32: GPTQ_F32, torch.float16: GPTQ_F16, torch.bfloat16: GPTQ_BF16}


class GPTQError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} (status {status})")
        self.status = status


class NotPositiveDefinite(GPTQError):
    pass


class gptq_config(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("damp_percent", ctypes.c_float),
                ("desc_act", ctypes.c_int32), ("sym", ctypes.c_int32),
                ("per_block_steps", ctypes.c_int32)]


class gptq_w4_weight(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p),
                ("perm", ctypes.c_void_p), ("d_out", ctypes.c_int32), ("d_in", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("n_groups", ctypes.c_int32)]


class gptq_kv4_cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_grid", ctypes.c_void_p),
                ("v_grid", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("n_pages", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("n_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libgptq.so not found at {LIB_PATH}; build it with "
                              f"`python -m post_weight_quantization_29_amd.build_lib`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        wt, kv = ctypes.POINTER(gptq_w4_weight), ctypes.POINTER(gptq_kv4_cache)
        sig = {
            "gptq_hessian_workspace_size": (sz, [i64, i32]),
            "gptq_hessian_accumulate": (ctypes.c_int, [vp, vp, vp, ctypes.c_int, i64, i32, vp, sz, vp]),
            "gptq_hessian_noalloc_scratch_bytes": (sz, []),
            "gptq_hessian_accumulate_noalloc": (ctypes.c_int, [vp, vp, vp, ctypes.c_int, i64, i32, vp]),
            "gptq_prepare_hinv_workspace_size": (sz, [i32]),
            "gptq_prepare_hinv": (ctypes.c_int, [vp, vp, i32, ctypes.c_float, i32, vp, vp, vp, sz, vp]),
            "gptq_quantize_workspace_size": (sz, [i32, i32, ctypes.POINTER(gptq_config)]),
            "gptq_quantize_layer": (ctypes.c_int, [vp, ctypes.c_int, i32, i32, vp, vp,
                                                   ctypes.POINTER(gptq_config), vp, vp, vp, vp, vp,
                                                   vp, sz, vp]),
            "gptq_pack_int4": (ctypes.c_int, [vp, i64, i64, vp, vp]),
            "gptq_pack_dense": (ctypes.c_int, [vp, i64, i64, i32, vp, vp]),
            "gptq_w4a16_gemm": (ctypes.c_int, [vp, ctypes.c_int, i64, i32, vp, vp, vp, vp, i32, i32,
                                               i32, vp, ctypes.c_int, vp]),
            "gptq_awq_sumsq_workspace_size": (sz, [i64, i32]),
            "gptq_awq_act_sumsq": (ctypes.c_int, [vp, vp, ctypes.c_int, i64, i32, vp, sz, vp]),
            "gptq_awq_search_workspace_size": (sz, [i32, i32, i32]),
            "gptq_awq_search": (ctypes.c_int, [vp, ctypes.c_int, i32, i32, vp, i32, i32, ctypes.c_float,
                                               ctypes.POINTER(ctypes.c_float), i32, vp, vp, vp, vp, sz,
                                               vp]),
            "gptq_awq_quantize": (ctypes.c_int, [vp, ctypes.c_int, i32, i32, vp, i32, i32, vp, vp, vp,
                                                 vp, vp]),
            "gptq_rmsnorm": (ctypes.c_int, [vp, ctypes.c_int, i64, i32, vp, ctypes.c_float, vp, vp]),
            "gptq_linear_workspace_size": (sz, [i32, i32]),
            "gptq_linear": (ctypes.c_int, [vp, i64, i32, vp, i32, vp, vp, vp, sz, vp]),
            "gptq_block_attention_workspace_size": (sz, [i64, i32, i32, i32]),
            "gptq_block_attention": (ctypes.c_int, [vp, i64, i32, i32, i32, vp, vp, vp, ctypes.c_float,
                                                    vp, vp, sz, vp]),
            "gptq_swiglu": (ctypes.c_int, [vp, vp, i64, vp, vp]),
            "gptq_w4_linear_workspace_size": (sz, [i64, wt]),
            "gptq_w4_linear": (ctypes.c_int, [vp, ctypes.c_int, i64, i64, wt, vp, ctypes.c_int, vp, i64, vp,
                                              ctypes.c_int, i64, vp, sz, vp]),
            "gptq_w4_gated_workspace_size": (sz, [i64, wt, wt]),
            "gptq_w4_gated": (ctypes.c_int, [vp, ctypes.c_int, i64, i64, wt, wt, ctypes.c_int, vp, vp, vp, vp, sz,
                                             vp]),
            "gptq_w4_gated_backward_workspace_size": (sz, [i64, wt, wt]),
            "gptq_w4_gated_backward": (ctypes.c_int, [vp, vp, vp, ctypes.c_int, i64, wt, wt, ctypes.c_int, vp, vp,
                                                      vp, vp, sz, vp]),
            "gptq_kv4_append": (ctypes.c_int, [kv, vp, vp, ctypes.c_int, i64, i64, i64, vp, vp, vp]),
            "gptq_kv4_read": (ctypes.c_int, [kv, vp, vp, ctypes.c_int, i64, vp, vp, vp]),
            "gptq_kv4_attention_workspace_size": (sz, [i64, i32, kv, i32, i32]),
            "gptq_kv4_attention": (ctypes.c_int, [vp, ctypes.c_int, i64, i32, i64, kv, vp, vp, i32, i32,
                                                  ctypes.c_float, vp, i64, vp, sz, vp]),
            "gptq_layer_error_workspace_size": (sz, [i32, i32]),
            "gptq_layer_error": (ctypes.c_int, [vp, vp, ctypes.c_int, vp, i32, i32,
                                                ctypes.POINTER(ctypes.c_double), vp, sz, vp]),
            "gptq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "gptq_abi_version": (ctypes.c_int, []),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


EXPORTED = ("gptq_hessian_workspace_size", "gptq_hessian_accumulate",
            "gptq_hessian_noalloc_scratch_bytes", "gptq_hessian_accumulate_noalloc",
            "gptq_prepare_hinv_workspace_size", "gptq_prepare_hinv",
            "gptq_quantize_workspace_size", "gptq_quantize_layer", "gptq_pack_int4",
            "gptq_pack_dense", "gptq_w4a16_gemm", "gptq_awq_sumsq_workspace_size",
            "gptq_awq_act_sumsq", "gptq_awq_search_workspace_size", "gptq_awq_search",
            "gptq_awq_quantize", "gptq_rmsnorm", "gptq_linear_workspace_size", "gptq_linear",
            "gptq_block_attention_workspace_size", "gptq_block_attention", "gptq_swiglu",
            "gptq_w4_linear_workspace_size", "gptq_w4_linear", "gptq_w4_gated_workspace_size",
            "gptq_w4_gated", "gptq_w4_gated_backward_workspace_size", "gptq_w4_gated_backward",
            "gptq_kv4_append", "gptq_kv4_read", "gptq_kv4_attention_workspace_size",
            "gptq_kv4_attention",
            "gptq_layer_error_workspace_size", "gptq_layer_error", "gptq_status_string",
            "gptq_abi_version")


def _check(st: int, what: str) -> None:
    if st == OK:
        return
    msg = f"{what}: {lib().gptq_status_string(st).decode()}"
    if st == ERR_NOT_PD:
        raise NotPositiveDefinite(st, msg)
    raise GPTQError(st, msg)


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _dev(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _ws(nbytes: int, ws: Optional[torch.Tensor], device, stream=None) -> torch.Tensor:
    """The caller's workspace, or a fresh one from torch's caching allocator.
    A fresh one is allocated on the stream the call's work goes to, so that
    the allocator reuses its memory only after that work (the call may return
    before its kernels have run)."""
    if ws is not None:
        return ws
    if stream is None:
        return torch.empty(max(1, nbytes), dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(max(1, nbytes), dtype=torch.uint8, device=device)


def make_config(bits: int = 4, group_size: int = 128, block_size: int = 128,
                damp_percent: float = 0.01, desc_act: int = 0, sym: int = 0,
                per_block_steps: int = 0) -> gptq_config:
    return gptq_config(bits, group_size, block_size, damp_percent, int(desc_act), int(sym),
                       int(per_block_steps))


# ---------------------------------------------------------------- C-ABI calls

def gptq_hessian_workspace_size(n_tokens: int, d_in: int) -> int:
    return int(lib().gptq_hessian_workspace_size(n_tokens, d_in))


def gptq_hessian_accumulate(H: torch.Tensor, X: torch.Tensor, hdiag: Optional[torch.Tensor] = None,
                            ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """H [d, d] fp32 += 2 X^T X for X [n_tokens, d] (fp32 / fp16 / bf16);
    hdiag [d] fp64 (optional) += the same diagonal summed in fp64."""
    _dev(H, "H"); _dev(X, "X")
    n, d = X.shape
    assert H.dtype == torch.float32 and tuple(H.shape) == (d, d)
    if hdiag is not None:
        _dev(hdiag, "hdiag")
        assert hdiag.dtype == torch.float64 and hdiag.numel() == d
    need = gptq_hessian_workspace_size(n, d)
    ws = _ws(need, ws, X.device, stream)
    _check(lib().gptq_hessian_accumulate(_ptr(H), _ptr(hdiag), _ptr(X), _DTYPE[X.dtype], n, d,
                                         _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "gptq_hessian_accumulate")


def gptq_hessian_noalloc_scratch_bytes() -> int:
    return int(lib().gptq_hessian_noalloc_scratch_bytes())


def gptq_hessian_accumulate_noalloc(H: torch.Tensor, X: torch.Tensor,
                                    hdiag: Optional[torch.Tensor] = None, stream=None) -> None:
    """gptq_hessian_accumulate with the partial sums in the library's static
    per-device scratch array (no allocation at all; d_in <= 11,264)."""
    _dev(H, "H"); _dev(X, "X")
    n, d = X.shape
    assert H.dtype == torch.float32 and tuple(H.shape) == (d, d)
    if hdiag is not None:
        _dev(hdiag, "hdiag")
        assert hdiag.dtype == torch.float64 and hdiag.numel() == d
    _check(lib().gptq_hessian_accumulate_noalloc(_ptr(H), _ptr(hdiag), _ptr(X), _DTYPE[X.dtype], n, d,
                                                 _stream(stream)), "gptq_hessian_accumulate_noalloc")


def gptq_prepare_hinv_workspace_size(d_in: int) -> int:
    return int(lib().gptq_prepare_hinv_workspace_size(d_in))


def gptq_prepare_hinv(H: torch.Tensor, damp_percent: float, desc_act: int, U: torch.Tensor,
                      perm: torch.Tensor, hdiag: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, stream=None) -> None:
    _dev(H, "H"); _dev(U, "U"); _dev(perm, "perm")
    d = H.shape[0]
    assert H.dtype == U.dtype == torch.float32 and perm.dtype == torch.int32
    if hdiag is not None:
        _dev(hdiag, "hdiag")
        assert hdiag.dtype == torch.float64 and hdiag.numel() == d
    ws = _ws(gptq_prepare_hinv_workspace_size(d), ws, H.device, stream)
    _check(lib().gptq_prepare_hinv(_ptr(H), _ptr(hdiag), d, float(damp_percent), int(desc_act),
                                   _ptr(U), _ptr(perm), _ptr(ws), ws.numel() * ws.element_size(),
                                   _stream(stream)), "gptq_prepare_hinv")


def gptq_quantize_workspace_size(d_out: int, d_in: int, cfg: gptq_config) -> int:
    return int(lib().gptq_quantize_workspace_size(d_out, d_in, ctypes.byref(cfg)))


def gptq_quantize_layer(W: torch.Tensor, U: torch.Tensor, perm: torch.Tensor, cfg: gptq_config,
                        codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                        g_idx: torch.Tensor, Q: Optional[torch.Tensor] = None,
                        ws: Optional[torch.Tensor] = None, stream=None) -> None:
    for t, nm in ((W, "W"), (U, "U"), (perm, "perm"), (codes, "codes"), (scales, "scales"),
                  (zeros, "zeros"), (g_idx, "g_idx")):
        _dev(t, nm)
    if Q is not None:
        _dev(Q, "Q")
    d_out, d_in = W.shape
    assert codes.dtype == torch.uint8 and scales.dtype == torch.float32
    assert zeros.dtype == torch.int32 and g_idx.dtype == torch.int32
    ws = _ws(gptq_quantize_workspace_size(d_out, d_in, cfg), ws, W.device, stream)
    _check(lib().gptq_quantize_layer(_ptr(W), _DTYPE[W.dtype], d_out, d_in, _ptr(U), _ptr(perm),
                                     ctypes.byref(cfg), _ptr(codes), _ptr(scales), _ptr(zeros),
                                     _ptr(g_idx), _ptr(Q), _ptr(ws), ws.numel() * ws.element_size(),
                                     _stream(stream)), "gptq_quantize_layer")


def gptq_pack_int4(codes: torch.Tensor, packed: torch.Tensor, stream=None) -> None:
    _dev(codes, "codes"); _dev(packed, "packed")
    rows, cols = codes.shape
    assert packed.dtype == torch.int32 or packed.dtype == torch.uint32
    _check(lib().gptq_pack_int4(_ptr(codes), rows, cols, _ptr(packed), _stream(stream)),
           "gptq_pack_int4")


def gptq_pack_dense(codes: torch.Tensor, packed: torch.Tensor, bits: int, stream=None) -> None:
    _dev(codes, "codes"); _dev(packed, "packed")
    rows, cols = codes.shape
    assert packed.dtype == torch.int32 or packed.dtype == torch.uint32
    _check(lib().gptq_pack_dense(_ptr(codes), rows, cols, int(bits), _ptr(packed), _stream(stream)),
           "gptq_pack_dense")


def gptq_w4a16_gemm(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                    Y: torch.Tensor, g_idx: Optional[torch.Tensor] = None, group_size: int = 128,
                    stream=None) -> None:
    for t, n in ((X, "X"), (packed, "packed"), (scales, "scales"), (zeros, "zeros"), (Y, "Y")):
        _dev(t, n)
    m, d_in = X.shape
    d_out, n_groups = scales.shape
    assert Y.shape == (m, d_out) and zeros.shape == scales.shape
    if g_idx is not None:
        _dev(g_idx, "g_idx")
    _check(lib().gptq_w4a16_gemm(_ptr(X), _DTYPE[X.dtype], m, d_in, _ptr(packed), _ptr(scales),
                                 _ptr(zeros), _ptr(g_idx) if g_idx is not None else None,
                                 int(group_size), n_groups, d_out, _ptr(Y), _DTYPE[Y.dtype],
                                 _stream(stream)), "gptq_w4a16_gemm")


AWQ_DEFAULT_GRID = tuple(1.0 + 0.125 * k for k in range(25))


def gptq_awq_sumsq_workspace_size(n_tokens: int, d_in: int) -> int:
    return int(lib().gptq_awq_sumsq_workspace_size(n_tokens, d_in))


def gptq_awq_act_sumsq(a: torch.Tensor, X: torch.Tensor, ws: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    _dev(a, "a"); _dev(X, "X")
    n, d_in = X.shape
    assert a.dtype == torch.float64 and a.shape == (d_in,)
    ws = _ws(gptq_awq_sumsq_workspace_size(n, d_in), ws, X.device, stream)
    _check(lib().gptq_awq_act_sumsq(_ptr(a), _ptr(X), _DTYPE[X.dtype], n, d_in, _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(stream)),
           "gptq_awq_act_sumsq")


def gptq_awq_search_workspace_size(d_out: int, d_in: int, group_size: int = 128) -> int:
    return int(lib().gptq_awq_search_workspace_size(d_out, d_in, group_size))


def gptq_awq_search(W: torch.Tensor, a: torch.Tensor, s_out: torch.Tensor, scores: torch.Tensor,
                    best: Optional[torch.Tensor] = None, bits: int = 4, group_size: int = 128,
                    top_frac: float = 0.05, grid=AWQ_DEFAULT_GRID, ws: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    for t, n in ((W, "W"), (a, "a"), (s_out, "s_out"), (scores, "scores")):
        _dev(t, n)
    d_out, d_in = W.shape
    g = (ctypes.c_float * len(grid))(*[float(v) for v in grid])
    ws = _ws(gptq_awq_search_workspace_size(d_out, d_in, group_size), ws, W.device, stream)
    _check(lib().gptq_awq_search(_ptr(W), _DTYPE[W.dtype], d_out, d_in, _ptr(a), bits, group_size,
                                 float(top_frac), g, len(grid), _ptr(s_out), _ptr(scores), _ptr(best),
                                 _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "gptq_awq_search")


def gptq_awq_quantize(W: torch.Tensor, s: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                      zeros: torch.Tensor, Qhat: Optional[torch.Tensor] = None, bits: int = 4,
                      group_size: int = 128, stream=None) -> None:
    for t, n in ((W, "W"), (s, "s"), (codes, "codes"), (scales, "scales"), (zeros, "zeros")):
        _dev(t, n)
    d_out, d_in = W.shape
    _check(lib().gptq_awq_quantize(_ptr(W), _DTYPE[W.dtype], d_out, d_in, _ptr(s), bits, group_size,
                                   _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(Qhat),
                                   _stream(stream)), "gptq_awq_quantize")


def gptq_rmsnorm(X: torch.Tensor, Y: torch.Tensor, gamma: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, stream=None) -> None:
    _dev(X, "X"); _dev(Y, "Y")
    n, d = X.shape
    assert Y.dtype == torch.float32 and Y.shape == (n, d)
    _check(lib().gptq_rmsnorm(_ptr(X), _DTYPE[X.dtype], n, d, _ptr(gamma), float(eps), _ptr(Y),
                              _stream(stream)), "gptq_rmsnorm")


def gptq_linear_workspace_size(d_out: int, d_in: int) -> int:
    return int(lib().gptq_linear_workspace_size(d_out, d_in))


def gptq_linear(X: torch.Tensor, W: torch.Tensor, Y: torch.Tensor, R: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = None, stream=None) -> None:
    _dev(X, "X"); _dev(W, "W"); _dev(Y, "Y")
    n, d_in = X.shape
    d_out = W.shape[0]
    assert W.shape == (d_out, d_in) and Y.shape == (n, d_out)
    assert X.dtype == W.dtype == Y.dtype == torch.float32
    ws = _ws(gptq_linear_workspace_size(d_out, d_in), ws, X.device, stream)
    _check(lib().gptq_linear(_ptr(X), n, d_in, _ptr(W), d_out, _ptr(R), _ptr(Y), _ptr(ws),
                             ws.numel() * ws.element_size(), _stream(stream)), "gptq_linear")


def gptq_block_attention_workspace_size(n_tokens: int, d: int, n_heads: int, seq_len: int) -> int:
    return int(lib().gptq_block_attention_workspace_size(n_tokens, d, n_heads, seq_len))


def gptq_block_attention(x1: torch.Tensor, Wq: torch.Tensor, Wk: torch.Tensor, Wv: torch.Tensor,
                         out: torch.Tensor, n_heads: int, seq_len: int, rope_base: float = 10000.0,
                         ws: Optional[torch.Tensor] = None, stream=None) -> None:
    for t, n in ((x1, "x1"), (Wq, "Wq"), (Wk, "Wk"), (Wv, "Wv"), (out, "out")):
        _dev(t, n)
    T, d = x1.shape
    ws = _ws(gptq_block_attention_workspace_size(T, d, n_heads, seq_len), ws, x1.device, stream)
    _check(lib().gptq_block_attention(_ptr(x1), T, d, n_heads, seq_len, _ptr(Wq), _ptr(Wk), _ptr(Wv),
                                      float(rope_base), _ptr(out), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream)),
           "gptq_block_attention")


def gptq_swiglu(G: torch.Tensor, U: torch.Tensor, M: torch.Tensor, stream=None) -> None:
    _dev(G, "G"); _dev(U, "U"); _dev(M, "M")
    assert G.shape == U.shape == M.shape
    _check(lib().gptq_swiglu(_ptr(G), _ptr(U), G.numel(), _ptr(M), _stream(stream)), "gptq_swiglu")


# ---------------------------------------------------------------- running the packed layer

GPTQ_ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def _on(t: Optional[torch.Tensor], name: str, index: int, dtype=None, rows: bool = False) -> None:
    """t is on device `index`, of `dtype` and contiguous (rows: only inside its rows)."""
    if t is None:
        return
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous() and not (rows and (t.stride(-1) == 1 or t.shape[-1] == 1)):
        raise ValueError(f"{name} must be contiguous" + (" inside its rows" if rows else ""))


def _shape(t: Optional[torch.Tensor], name: str, shape: tuple) -> None:
    if t is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")


def _pitch(t: torch.Tensor) -> int:
    """Elements from one row to the next; a single row counts as one whose successor would be aligned."""
    return t.stride(0) if t.shape[0] > 1 else (t.numel() + 7) & ~7


def _act(act) -> int:
    if act not in GPTQ_ACTS:
        raise ValueError(f"act must be one of {', '.join(GPTQ_ACTS)}, got {act!r}")
    return GPTQ_ACTS[act]


def _dtype16(t: torch.Tensor, name: str) -> int:
    if t.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"{name} must be float16 or bfloat16, got {t.dtype}")
    return _DTYPE[t.dtype]


def _run(name: str, index: int, stream, *args) -> None:
    """The call on `stream` (default: the tensors' device's current one), with that device current."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device.index != index:
        raise ValueError(f"{name}: the stream is on {stream.device}, the tensors are on cuda:{index}")
    else:
        raw = stream.cuda_stream
    f = getattr(lib(), name)
    if torch._C._cuda_getDevice() == index:
        st = f(*args, raw)
    else:
        with torch.cuda.device(index):
            st = f(*args, raw)
    if st != OK:
        _check(st, name)


def _scratch(nbytes: int, ws: Optional[torch.Tensor], index: int, stream) -> torch.Tensor:
    """The caller's workspace or one of nbytes (the tensor has to live until the call returns)."""
    if ws is None:
        return _ws(nbytes, None, torch.device("cuda", index), stream)
    _on(ws, "ws", index)
    return ws


class W4Weight:
    """A packed 4-bit weight (gptq_w4_weight): packed [d_out, d_in/8] (gptq_pack_int4's words, columns in
    processing order), scales and zeros [d_out, n_groups], perm [d_in] or None.  Holds the tensors; they
    may be rewritten in place between calls.  With perm the words are those of codes[:, perm]: a desc_act
    layer's `packed`, which has its columns in channel order, is not; from_codes orders them."""

    def __init__(self, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, group_size: int = 128,
                 perm: Optional[torch.Tensor] = None):
        index = packed.device.index if packed.is_cuda else 0
        _on(packed, "packed", index); _on(scales, "scales", index, torch.float32)
        _on(zeros, "zeros", index, torch.int32); _on(perm, "perm", index, torch.int32)
        if packed.dtype not in (torch.int32, torch.uint32):
            raise ValueError(f"packed must be int32 or uint32, got {packed.dtype}")
        d_out, words = packed.shape
        G = 8 * words if group_size == -1 else group_size
        if G <= 0 or G % 8:
            raise ValueError(f"group_size must be -1 or a multiple of 8, got {group_size}")
        _shape(scales, "scales", (d_out, -(-8 * words // G))); _shape(zeros, "zeros", (d_out, -(-8 * words // G)))
        _shape(perm, "perm", (8 * words,))
        self.packed, self.scales, self.zeros, self.perm, self.group_size = packed, scales, zeros, perm, group_size
        self.d_out, self.d_in, self.index = d_out, 8 * words, index
        self.c = gptq_w4_weight(_ptr(packed), _ptr(scales), _ptr(zeros), _ptr(perm), d_out, 8 * words, group_size,
                                scales.shape[1])
        self.ref = ctypes.pointer(self.c)

    @classmethod
    def from_codes(cls, codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, group_size: int = 128,
                   perm: Optional[torch.Tensor] = None) -> "W4Weight":
        """The weight of a quantized layer: codes [d_out, d_in] uint8 in channel order, scales and zeros as
        gptq_quantize_layer (or gptq_awq_quantize) writes them; perm: a desc_act layer's order, None for a layer
        quantized from left to right (entries outside it count as the nearest, as in the kernels).  Packs a copy
        of the codes, in that order."""
        index = codes.device.index if codes.is_cuda else 0
        _on(codes, "codes", index, torch.uint8)
        _on(perm, "perm", index, torch.int32)
        d_out, d_in = codes.shape
        if d_in % 8:
            raise ValueError(f"codes must have a multiple of 8 columns, got {d_in}")
        _shape(perm, "perm", (d_in,))
        ordered = codes if perm is None else codes.index_select(1, perm.clamp(0, d_in - 1))
        packed = torch.empty((d_out, d_in // 8), dtype=torch.int32, device=codes.device)
        _run("gptq_pack_int4", index, None, ordered.data_ptr(), d_out, d_in, packed.data_ptr())
        return cls(packed, scales, zeros, group_size, perm)


def gptq_w4_linear_workspace_size(m: int, w: W4Weight) -> int:
    return int(lib().gptq_w4_linear_workspace_size(m, w.ref))


def gptq_w4_linear(X: torch.Tensor, w: W4Weight, Y: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   act: str = "none", R: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    """Y [m, d_out] = act(X W^T + bias) + R.  X, Y and R may have pitched rows; R may be Y."""
    dev, m = w.index, X.shape[0]
    _on(X, "X", dev, rows=True); _on(Y, "Y", dev, rows=True)
    _shape(X, "X", (m, w.d_in)); _shape(Y, "Y", (m, w.d_out))
    if bias is not None:
        _on(bias, "bias", dev, X.dtype); _shape(bias, "bias", (w.d_out,))
    if R is not None:
        _on(R, "R", dev, Y.dtype, rows=True); _shape(R, "R", (m, w.d_out))
    xt = _dtype16(X, "X")
    if Y.dtype not in _DTYPE:
        raise ValueError(f"Y must be float32, float16 or bfloat16, got {Y.dtype}")
    ws = _scratch(0 if ws is not None else gptq_w4_linear_workspace_size(m, w), ws, dev, stream)
    _run("gptq_w4_linear", dev, stream, X.data_ptr(), xt, m, _pitch(X), w.ref, _ptr(bias), _act(act), _ptr(R),
         0 if R is None else _pitch(R), Y.data_ptr(), _DTYPE[Y.dtype], _pitch(Y), ws.data_ptr(), ws.nbytes)


def gptq_w4_gated_workspace_size(m: int, gate: W4Weight, up: W4Weight) -> int:
    return int(lib().gptq_w4_gated_workspace_size(m, gate.ref, up.ref))


def _same_device(gate: W4Weight, up: W4Weight) -> None:
    if gate.index != up.index:
        raise ValueError(f"gate is on cuda:{gate.index}, up on cuda:{up.index}")


def gptq_w4_gated(X: torch.Tensor, gate: W4Weight, up: W4Weight, M: torch.Tensor, G: Optional[torch.Tensor] = None,
                  U: Optional[torch.Tensor] = None, act: str = "silu", ws: Optional[torch.Tensor] = None,
                  stream=None) -> None:
    """M [m, f] = act(X Wg^T) * (X Wu^T); G and U, where given, take both products for the backward pass."""
    dev, m = gate.index, X.shape[0]
    _same_device(gate, up)
    _on(X, "X", dev, rows=True); _shape(X, "X", (m, gate.d_in))
    for t, n in ((M, "M"), (G, "G"), (U, "U")):
        if t is not None:
            _on(t, n, dev, X.dtype); _shape(t, n, (m, gate.d_out))
    xt = _dtype16(X, "X")
    ws = _scratch(0 if ws is not None else gptq_w4_gated_workspace_size(m, gate, up), ws, dev, stream)
    _run("gptq_w4_gated", dev, stream, X.data_ptr(), xt, m, _pitch(X), gate.ref, up.ref, _act(act), _ptr(G), _ptr(U),
         M.data_ptr(), ws.data_ptr(), ws.nbytes)


def gptq_w4_gated_backward_workspace_size(m: int, gate: W4Weight, up: W4Weight) -> int:
    return int(lib().gptq_w4_gated_backward_workspace_size(m, gate.ref, up.ref))


def gptq_w4_gated_backward(dM: torch.Tensor, G: torch.Tensor, U: torch.Tensor, gate: W4Weight, up: W4Weight,
                           dX: torch.Tensor, dG: Optional[torch.Tensor] = None, dU: Optional[torch.Tensor] = None,
                           act: str = "silu", ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """dX [m, d], dG and dU [m, f] (optional) from dM and the forward pass's G and U."""
    dev, m = gate.index, dM.shape[0]
    _same_device(gate, up)
    for t, n in ((dM, "dM"), (G, "G"), (U, "U"), (dG, "dG"), (dU, "dU")):
        if t is not None:
            _on(t, n, dev, dM.dtype); _shape(t, n, (m, gate.d_out))
    _on(dX, "dX", dev, dM.dtype); _shape(dX, "dX", (m, gate.d_in))
    dt = _dtype16(dM, "dM")
    ws = _scratch(0 if ws is not None else gptq_w4_gated_backward_workspace_size(m, gate, up), ws, dev, stream)
    _run("gptq_w4_gated_backward", dev, stream, dM.data_ptr(), G.data_ptr(), U.data_ptr(), dt, m, gate.ref, up.ref,
         _act(act), _ptr(dG), _ptr(dU), dX.data_ptr(), ws.data_ptr(), ws.nbytes)


# ---------------------------------------------------------------- a cache held in 4 bits

class KV4Cache:
    """A paged cache (gptq_kv4_cache): k_codes, v_codes [n_pages, n_kv_heads, page_size, head_dim/8] int32,
    k_grid, v_grid [n_pages, n_kv_heads, page_size, 2] float16 (step, minimum), page_table [n_seqs,
    max_pages] int32.  Holds the tensors; they may be rewritten in place between calls."""

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_grid: torch.Tensor, v_grid: torch.Tensor,
                 page_table: torch.Tensor):
        dev = k_codes.device.index if k_codes.is_cuda else 0
        for t, n in ((k_codes, "k_codes"), (v_codes, "v_codes")):
            _on(t, n, dev, torch.int32); _shape(t, n, tuple(k_codes.shape))
        for t, n in ((k_grid, "k_grid"), (v_grid, "v_grid")):
            _on(t, n, dev, torch.float16); _shape(t, n, (*k_codes.shape[:3], 2))
        _on(page_table, "page_table", dev, torch.int32)
        n_pages, n_kv, page, words = k_codes.shape
        n_seqs, max_pages = page_table.shape
        if page <= 0 or page % 16 or 8 * words not in (64, 128):
            raise ValueError(f"page_size must be a multiple of 16 and head_dim 64 or 128, got {page} and {8 * words}")
        self.k_codes, self.v_codes, self.k_grid, self.v_grid, self.page_table = k_codes, v_codes, k_grid, v_grid, page_table
        self.n_kv_heads, self.head_dim, self.page_size, self.n_seqs, self.index = n_kv, 8 * words, page, n_seqs, dev
        self.c = gptq_kv4_cache(_ptr(k_codes), _ptr(v_codes), _ptr(k_grid), _ptr(v_grid), _ptr(page_table), n_pages,
                                n_kv, page, 8 * words, n_seqs, max_pages)
        self.ref = ctypes.pointer(self.c)

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, page_size: int, head_dim: int, page_table: torch.Tensor) -> "KV4Cache":
        """A cache of its own on the page table's device."""
        dev, shape = page_table.device, (n_pages, n_kv_heads, page_size)
        codes = [torch.empty(shape + (head_dim // 8,), dtype=torch.int32, device=dev) for _ in range(2)]
        grids = [torch.empty(shape + (2,), dtype=torch.float16, device=dev) for _ in range(2)]
        return cls(*codes, *grids, page_table)


def _heads(t: torch.Tensor, name: str, index: int, heads: int, hd: int, dtype=None) -> None:
    """[tokens, heads, hd], heads side by side inside a token's row."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != hd:
        raise ValueError(f"{name} must have shape (tokens, {heads}, {hd}), got {tuple(t.shape)}")
    if t.get_device() != index or (dtype is not None and t.dtype is not dtype):
        _on(t, name, index, dtype, rows=True)
    if not t.is_contiguous() and (t.stride(2) != 1 or (heads > 1 and t.stride(1) != hd)):
        raise ValueError(f"{name}'s heads must lie side by side")


def _batch(cache: KV4Cache, q_start: torch.Tensor, kv_len: torch.Tensor) -> None:
    for t, n, name in ((q_start, cache.n_seqs + 1, "q_start"), (kv_len, cache.n_seqs, "kv_len")):
        if t.dtype is not torch.int32 or t.get_device() != cache.index or t.numel() != n or not t.is_contiguous():
            _on(t, name, cache.index, torch.int32); _shape(t, name, (n,))


def gptq_kv4_append(cache: KV4Cache, K: torch.Tensor, V: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor,
                    stream=None) -> None:
    """Quantize the new tokens' K and V [tokens, n_kv_heads, head_dim] into the cache; kv_len counts them."""
    dev = cache.index
    _batch(cache, q_start, kv_len)
    _heads(K, "K", dev, cache.n_kv_heads, cache.head_dim); _heads(V, "V", dev, cache.n_kv_heads, cache.head_dim, K.dtype)
    if V.shape[0] != K.shape[0] or K.dtype not in _DTYPE:
        raise ValueError(f"K and V must be float32, float16 or bfloat16 with as many tokens, got {K.dtype}, "
                         f"{K.shape[0]} and {V.shape[0]}")
    _run("gptq_kv4_append", dev, stream, cache.ref, K.data_ptr(), V.data_ptr(), _DTYPE[K.dtype], K.shape[0], _pitch(K),
         _pitch(V), q_start.data_ptr(), kv_len.data_ptr())


def gptq_kv4_read(cache: KV4Cache, K: Optional[torch.Tensor], V: Optional[torch.Tensor], q_start: torch.Tensor,
                  kv_len: torch.Tensor, stream=None) -> None:
    """K, V [tokens, n_kv_heads, head_dim] (each may be None): the values the cache holds for the batch's tokens."""
    dev = cache.index
    _batch(cache, q_start, kv_len)
    some = K if K is not None else V
    if some is None:
        return
    for t, n in ((K, "K"), (V, "V")):
        if t is not None:
            _heads(t, n, dev, cache.n_kv_heads, cache.head_dim, some.dtype); _on(t, n, dev)
            if t.shape[0] != some.shape[0]:
                raise ValueError("K and V must have as many tokens")
    if some.dtype not in _DTYPE:
        raise ValueError(f"K and V must be float32, float16 or bfloat16, got {some.dtype}")
    _run("gptq_kv4_read", dev, stream, cache.ref, _ptr(K), _ptr(V), _DTYPE[some.dtype], some.shape[0],
         q_start.data_ptr(), kv_len.data_ptr())


def gptq_kv4_attention_workspace_size(n_tokens: int, n_heads: int, cache: KV4Cache, max_q_len: int,
                                      max_kv_len: int) -> int:
    if max_q_len >> 31 or max_kv_len >> 31:
        raise ValueError(f"max_q_len and max_kv_len must fit 32 bits, got {max_q_len} and {max_kv_len}")
    return int(lib().gptq_kv4_attention_workspace_size(n_tokens, n_heads, cache.ref, max_q_len, max_kv_len))


def gptq_kv4_attention(Q: torch.Tensor, cache: KV4Cache, q_start: torch.Tensor, kv_len: torch.Tensor, max_q_len: int,
                       max_kv_len: int, out: torch.Tensor, scale: Optional[float] = None,
                       ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """out [tokens, n_heads, head_dim] = causal attention of Q over the cache (scale None: 1/sqrt(head_dim))."""
    dev, hd = cache.index, cache.head_dim
    _batch(cache, q_start, kv_len)
    if Q.dim() != 3:
        raise ValueError(f"Q must have shape (tokens, heads, {hd}), got {tuple(Q.shape)}")
    T, n_heads = Q.shape[0], Q.shape[1]
    _heads(Q, "Q", dev, n_heads, hd); _heads(out, "out", dev, n_heads, hd, Q.dtype)
    if out.shape[0] != T:
        raise ValueError(f"out must have {T} tokens, got {out.shape[0]}")
    qt = _dtype16(Q, "Q")
    if max_q_len >> 31 or max_kv_len >> 31:
        raise ValueError(f"max_q_len and max_kv_len must fit 32 bits, got {max_q_len} and {max_kv_len}")
    need = 0 if ws is not None else gptq_kv4_attention_workspace_size(T, n_heads, cache, max_q_len, max_kv_len)
    ws = _scratch(need, ws, dev, stream)
    _run("gptq_kv4_attention", dev, stream, Q.data_ptr(), qt, T, n_heads, _pitch(Q), cache.ref, q_start.data_ptr(),
         kv_len.data_ptr(), max_q_len, max_kv_len, hd ** -0.5 if scale is None else float(scale), out.data_ptr(),
         _pitch(out), ws.data_ptr(), ws.nbytes)


def gptq_layer_error_workspace_size(d_out: int, d_in: int) -> int:
    return int(lib().gptq_layer_error_workspace_size(d_out, d_in))


def gptq_layer_error(H: torch.Tensor, W: torch.Tensor, Q: torch.Tensor,
                     ws: Optional[torch.Tensor] = None, stream=None) -> float:
    _dev(H, "H"); _dev(W, "W"); _dev(Q, "Q")
    d_out, d_in = W.shape
    ws = _ws(gptq_layer_error_workspace_size(d_out, d_in), ws, W.device, stream)
    out = ctypes.c_double(0.0)
    _check(lib().gptq_layer_error(_ptr(H), _ptr(W), _DTYPE[W.dtype], _ptr(Q), d_out, d_in,
                                  ctypes.byref(out), _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(stream)), "gptq_layer_error")
    return float(out.value)


def gptq_status_string(status: int) -> str:
    return lib().gptq_status_string(status).decode()


def gptq_abi_version() -> int:
    return int(lib().gptq_abi_version())
