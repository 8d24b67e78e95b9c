"""Python binding of the C ABI (include/moe_gb300.h), same names.

Argument marshalling only: every step of the layer runs in the CUDA library.
PyTorch provides device memory and the current stream.  Outputs that are not
passed in are allocated with torch on the input's device.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from ._lib import (MOE_EPI_STORE_BF16, MOE_EPI_SWIGLU_BF16, MOE_EPI_SWIGLU_MX, MOE_EPI_SWIGLU_NVFP4, MOE_FMT_BF16, MOE_FMT_MXFP4,
                   MOE_FMT_MXFP8, MOE_FMT_NVFP4, check, load)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _dev(t: torch.Tensor, name: str = "tensor", dtype=None, shape=None, device=None) -> None:
    """Reject what the kernels cannot take before any launch: a tensor that
    is missing, not on a CUDA device (its address would be read by a
    kernel), not contiguous, or of the wrong dtype, shape or device."""
    if t is None:
        raise ValueError(f"{name}: required")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _opt(t: Optional[torch.Tensor], name: str, **kw) -> None:
    if t is not None:
        _dev(t, name, **kw)


def _at_least(t: torch.Tensor, name: str, nbytes: int) -> None:
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{name}: {have} bytes, needs {nbytes}")


def _ws(nbytes: int, device) -> torch.Tensor:
    # 256-byte aligned by the caching allocator (allocations are 512-byte aligned)
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def moe_version() -> int:
    return load().moe_version()


def moe_sync_status(stream=None) -> int:
    return load().moe_sync_status(_stream(stream))


def moe_set_wait_timeout_ns(ns: int) -> None:
    check(load().moe_set_wait_timeout_ns(int(ns)), "moe_set_wait_timeout_ns")


def moe_selftest_wait_timeout(timeout_ns: int, stream=None) -> None:
    check(load().moe_selftest_wait_timeout(int(timeout_ns), _stream(stream)), "moe_selftest_wait_timeout")


def moe_selftest_attention_wait_timeout(timeout_ns: int, lazy: bool = False, stream=None) -> None:
    check(load().moe_selftest_attention_wait_timeout(int(timeout_ns), 1 if lazy else 0, _stream(stream)),
          "moe_selftest_attention_wait_timeout")


def moe_route(logits: torch.Tensor, k: int, idx: Optional[torch.Tensor] = None,
              w: Optional[torch.Tensor] = None, stream=None, renorm: bool = True):
    """logits fp32 [T, E] -> (idx int32 [T, k], w fp32 [T, k]); renorm=False
    takes the full softmax over E at the picks (moe_route_ex)."""
    _dev(logits, "logits", dtype=torch.float32)
    if logits.dim() != 2:
        raise ValueError("logits: expected [T, E]")
    T, E = logits.shape
    if idx is None:
        idx = torch.empty(T, k, dtype=torch.int32, device=logits.device)
    if w is None:
        w = torch.empty(T, k, dtype=torch.float32, device=logits.device)
    _dev(idx, "idx", dtype=torch.int32, shape=(T, k), device=logits.device)
    _dev(w, "w", dtype=torch.float32, shape=(T, k), device=logits.device)
    if renorm:
        check(load().moe_route(_ptr(logits), T, E, k, _ptr(idx), _ptr(w), _stream(stream)), "moe_route")
    else:
        check(load().moe_route_ex(_ptr(logits), T, E, k, 0, _ptr(idx), _ptr(w), _stream(stream)), "moe_route_ex")
    return idx, w


def moe_permute(idx: torch.Tensor, E: int, x_rows: Optional[torch.Tensor] = None,
                x_sf: Optional[torch.Tensor] = None, stream=None):
    """Stable permutation into expert-contiguous order.

    idx int32 [T, k]; x_rows: [T, ...] any dtype (rows copied as bytes) or None;
    x_sf: uint8 [T, sf_bytes] or None.  Returns dict(counts, offsets, row_of,
    src_tok, xp, xp_sf)."""
    _dev(idx, "idx", dtype=torch.int32)
    if idx.dim() != 2:
        raise ValueError("idx: expected [T, k]")
    T, k = idx.shape
    dev = idx.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    row_of = torch.empty(T, k, dtype=torch.int32, device=dev)
    src_tok = torch.empty(T * k, dtype=torch.int32, device=dev)
    xp = xp_sf = None
    row_bytes = sf_bytes = 0
    if x_rows is not None:
        _dev(x_rows, "x_rows", device=dev)
        if x_rows.shape[0] != T:
            raise ValueError("x_rows: expected one row per token")
        row_bytes = x_rows[0].numel() * x_rows.element_size() if T else 0
        xp = torch.empty((T * k,) + tuple(x_rows.shape[1:]), dtype=x_rows.dtype, device=dev)
        if x_sf is not None:
            _dev(x_sf, "x_sf", dtype=torch.uint8, device=dev)
            if x_sf.dim() != 2 or x_sf.shape[0] != T:
                raise ValueError("x_sf: expected [T, sf_bytes]")
            sf_bytes = x_sf.shape[1]
            xp_sf = torch.empty(T * k, sf_bytes, dtype=torch.uint8, device=dev)
    lib = load()
    nbytes = lib.moe_permute_workspace_size(T, k, E)
    ws = _ws(nbytes, dev)
    check(lib.moe_permute(_ptr(idx), T, k, E, _ptr(x_rows), row_bytes, _ptr(x_sf), sf_bytes,
                          _ptr(counts), _ptr(offsets), _ptr(row_of), _ptr(src_tok), _ptr(xp),
                          _ptr(xp_sf), _ptr(ws), nbytes, _stream(stream)), "moe_permute")
    return dict(counts=counts, offsets=offsets, row_of=row_of, src_tok=src_tok, xp=xp, xp_sf=xp_sf)


def moe_permute_noalloc(idx: torch.Tensor, E: int, x_rows: Optional[torch.Tensor] = None,
                        x_sf: Optional[torch.Tensor] = None, out: Optional[dict] = None, stream=None):
    """moe_permute for callers that cannot allocate device memory when they
    dispatch: the library keeps the scratch in its own fixed device array
    (size limit ceil(T*k/1024) * E <= 131072).  Pass preallocated outputs in
    `out` (keys counts, offsets, row_of, src_tok, xp, xp_sf) to make the call
    allocation-free end to end; missing outputs are allocated here."""
    _dev(idx, "idx", dtype=torch.int32)
    if idx.dim() != 2:
        raise ValueError("idx: expected [T, k]")
    T, k = idx.shape
    dev = idx.device
    o = dict(out or {})

    def need(key, make):
        # allocate only what the caller did not pass (a setdefault would build
        # the default tensor, and so allocate, even when the key is present)
        if o.get(key) is None:
            o[key] = make()

    need("counts", lambda: torch.empty(E, dtype=torch.int32, device=dev))
    need("offsets", lambda: torch.empty(E + 1, dtype=torch.int32, device=dev))
    need("row_of", lambda: torch.empty(T, k, dtype=torch.int32, device=dev))
    need("src_tok", lambda: torch.empty(T * k, dtype=torch.int32, device=dev))
    row_bytes = sf_bytes = 0
    if x_rows is not None:
        _dev(x_rows, "x_rows", device=dev)
        if x_rows.shape[0] != T:
            raise ValueError("x_rows: expected one row per token")
        row_bytes = x_rows[0].numel() * x_rows.element_size() if T else 0
        need("xp", lambda: torch.empty((T * k,) + tuple(x_rows.shape[1:]), dtype=x_rows.dtype, device=dev))
        if x_sf is not None:
            _dev(x_sf, "x_sf", dtype=torch.uint8, device=dev)
            if x_sf.dim() != 2 or x_sf.shape[0] != T:
                raise ValueError("x_sf: expected [T, sf_bytes]")
            sf_bytes = x_sf.shape[1]
            need("xp_sf", lambda: torch.empty(T * k, sf_bytes, dtype=torch.uint8, device=dev))
    o.setdefault("xp", None)
    o.setdefault("xp_sf", None)
    # caller-given outputs are written by the kernels: check them like inputs
    _dev(o["counts"], "counts", dtype=torch.int32, shape=(E,), device=dev)
    _dev(o["offsets"], "offsets", dtype=torch.int32, shape=(E + 1,), device=dev)
    _dev(o["row_of"], "row_of", dtype=torch.int32, shape=(T, k), device=dev)
    _dev(o["src_tok"], "src_tok", dtype=torch.int32, shape=(T * k,), device=dev)
    if x_rows is not None:
        _dev(o["xp"], "xp", device=dev)
        _at_least(o["xp"], "xp", T * k * row_bytes)
        if x_sf is not None:
            _dev(o["xp_sf"], "xp_sf", device=dev)
            _at_least(o["xp_sf"], "xp_sf", T * k * sf_bytes)
    check(load().moe_permute_noalloc(_ptr(idx), T, k, E, _ptr(x_rows), row_bytes, _ptr(x_sf), sf_bytes,
                                     _ptr(o["counts"]), _ptr(o["offsets"]), _ptr(o["row_of"]), _ptr(o["src_tok"]),
                                     _ptr(o["xp"]), _ptr(o["xp_sf"]), _stream(stream)), "moe_permute_noalloc")
    return o


def moe_route_permute(logits: torch.Tensor, k: int, x_rows: Optional[torch.Tensor] = None,
                      x_sf: Optional[torch.Tensor] = None, renorm: bool = True, stream=None):
    """Fused dispatch: moe_route then moe_permute in one cooperative launch.
    logits fp32 [T, E]; x_rows / x_sf as for moe_permute.  Returns dict(idx,
    w, counts, offsets, row_of, src_tok, xp, xp_sf)."""
    _dev(logits, "logits", dtype=torch.float32)
    if logits.dim() != 2:
        raise ValueError("logits: expected [T, E]")
    T, E = logits.shape
    dev = logits.device
    o = dict(idx=torch.empty(T, k, dtype=torch.int32, device=dev), w=torch.empty(T, k, device=dev),
             counts=torch.empty(E, dtype=torch.int32, device=dev),
             offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
             row_of=torch.empty(T, k, dtype=torch.int32, device=dev),
             src_tok=torch.empty(T * k, dtype=torch.int32, device=dev), xp=None, xp_sf=None)
    row_bytes = sf_bytes = 0
    if x_rows is not None:
        _dev(x_rows, "x_rows", device=dev)
        if x_rows.shape[0] != T:
            raise ValueError("x_rows: expected one row per token")
        row_bytes = x_rows[0].numel() * x_rows.element_size() if T else 0
        o["xp"] = torch.empty((T * k,) + tuple(x_rows.shape[1:]), dtype=x_rows.dtype, device=dev)
        if x_sf is not None:
            _dev(x_sf, "x_sf", dtype=torch.uint8, device=dev)
            if x_sf.dim() != 2 or x_sf.shape[0] != T:
                raise ValueError("x_sf: expected [T, sf_bytes]")
            sf_bytes = x_sf.shape[1]
            o["xp_sf"] = torch.empty(T * k, sf_bytes, dtype=torch.uint8, device=dev)
    lib = load()
    nbytes = lib.moe_route_permute_workspace_size(T, k, E)
    ws = _ws(nbytes, dev)
    check(lib.moe_route_permute(_ptr(logits), T, E, k, 1 if renorm else 0, _ptr(o["idx"]), _ptr(o["w"]),
                                _ptr(x_rows), row_bytes, _ptr(x_sf), sf_bytes, _ptr(o["counts"]),
                                _ptr(o["offsets"]), _ptr(o["row_of"]), _ptr(o["src_tok"]), _ptr(o["xp"]),
                                _ptr(o["xp_sf"]), _ptr(ws), nbytes, _stream(stream)), "moe_route_permute")
    return o


def moe_selftest_grid_barrier_timeout(timeout_ns: int, stream=None) -> None:
    check(load().moe_selftest_grid_barrier_timeout(int(timeout_ns), _stream(stream)),
          "moe_selftest_grid_barrier_timeout")


def moe_quant_nvfp4(x: torch.Tensor, g_in: Optional[torch.Tensor] = None, stream=None):
    """x bf16 [rows, cols] or [groups, rows, cols] -> (codes uint8 [..., cols/2],
    sf uint8 [..., cols/16], g fp32 [groups])."""
    _dev(x, "x", dtype=torch.bfloat16)
    if x.dim() not in (2, 3):
        raise ValueError("x: expected [rows, cols] or [groups, rows, cols]")
    x3 = x if x.dim() == 3 else x.unsqueeze(0)
    G, R, Cc = x3.shape
    _opt(g_in, "g_in", dtype=torch.float32, shape=(G,), device=x.device)
    codes = torch.empty(x.shape[:-1] + (Cc // 2,), dtype=torch.uint8, device=x.device)
    sf = torch.empty(x.shape[:-1] + (Cc // 16,), dtype=torch.uint8, device=x.device)
    g = torch.empty(G, dtype=torch.float32, device=x.device)
    lib = load()
    nbytes = lib.moe_quant_nvfp4_workspace_size(G)
    ws = _ws(nbytes, x.device)
    check(lib.moe_quant_nvfp4(_ptr(x3), G, R, Cc, _ptr(g_in), _ptr(codes), _ptr(sf), _ptr(g),
                              _ptr(ws), nbytes, _stream(stream)), "moe_quant_nvfp4")
    return codes, sf, g


def moe_quant_mx(x: torch.Tensor, fmt: int, stream=None):
    """x bf16 [rows, cols] -> (codes, scales uint8 [rows, cols/32]): MXFP8
    codes uint8 [rows, cols], MXFP4 packed codes uint8 [rows, cols/2]."""
    _dev(x, "x", dtype=torch.bfloat16)
    if x.dim() != 2:
        raise ValueError("x: expected [rows, cols]")
    if fmt not in (MOE_FMT_MXFP8, MOE_FMT_MXFP4):
        raise ValueError("fmt: expected MOE_FMT_MXFP8 or MOE_FMT_MXFP4")
    R, Cc = x.shape
    codes = torch.empty(R, Cc if fmt == MOE_FMT_MXFP8 else Cc // 2, dtype=torch.uint8, device=x.device)
    scales = torch.empty(R, Cc // 32, dtype=torch.uint8, device=x.device)
    check(load().moe_quant_mx(_ptr(x), R, Cc, int(fmt), _ptr(codes), _ptr(scales), _stream(stream)), "moe_quant_mx")
    return codes, scales


def moe_grouped_gemm(a_fmt: int, w_fmt: int, epilogue: int, offsets: torch.Tensor, N: int, K: int,
                     A: torch.Tensor, W: torch.Tensor, A_sf=None, A_g=None, W_sf=None, W_g=None,
                     c_g=None, C=None, C_sf=None, stream=None):
    """Grouped GEMM over expert-contiguous rows; see include/moe_gb300.h.
    Every operand is checked for device, contiguity and size against
    (G, M, N, K) and the formats before the call."""
    _dev(A, "A")
    dev = A.device
    _dev(offsets, "offsets", dtype=torch.int32, device=dev)
    G = offsets.numel() - 1
    M = A.shape[0]
    wn = 2 * N if epilogue in (MOE_EPI_SWIGLU_BF16, MOE_EPI_SWIGLU_NVFP4, MOE_EPI_SWIGLU_MX) else N
    mx_c = N // 2 if a_fmt == MOE_FMT_MXFP4 else N  # bytes per row of MX-coded C
    _dev(W, "W", device=dev)
    if a_fmt == MOE_FMT_NVFP4:
        _at_least(A, "A", M * K // 2)
        _dev(A_sf, "A_sf", device=dev)
        _at_least(A_sf, "A_sf", M * K // 16)
        _dev(A_g, "A_g", dtype=torch.float32, device=dev)
        _at_least(A_g, "A_g", 4)
    elif a_fmt in (MOE_FMT_MXFP4, MOE_FMT_MXFP8):
        _at_least(A, "A", M * K // (2 if a_fmt == MOE_FMT_MXFP4 else 1))
        _dev(A_sf, "A_sf", device=dev)
        _at_least(A_sf, "A_sf", M * K // 32)
    else:
        _at_least(A, "A", M * K * 2)
    if w_fmt == MOE_FMT_NVFP4:
        _at_least(W, "W", G * wn * K // 2)
        _dev(W_sf, "W_sf", device=dev)
        _at_least(W_sf, "W_sf", G * wn * K // 16)
        _dev(W_g, "W_g", dtype=torch.float32, device=dev)
        _at_least(W_g, "W_g", 4 * G)
    elif w_fmt in (MOE_FMT_MXFP4, MOE_FMT_MXFP8):
        _at_least(W, "W", G * wn * K // (2 if w_fmt == MOE_FMT_MXFP4 else 1))
        _dev(W_sf, "W_sf", device=dev)
        _at_least(W_sf, "W_sf", G * wn * K // 32)
    else:
        _at_least(W, "W", G * wn * K * 2)
    if C is None:
        if epilogue == MOE_EPI_SWIGLU_NVFP4:
            C = torch.empty(M, N // 2, dtype=torch.uint8, device=dev)
            C_sf = torch.empty(M, N // 16, dtype=torch.uint8, device=dev)
        elif epilogue == MOE_EPI_SWIGLU_MX:
            C = torch.empty(M, mx_c, dtype=torch.uint8, device=dev)
            C_sf = torch.empty(M, N // 32, dtype=torch.uint8, device=dev)
        else:
            C = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    _dev(C, "C", device=dev)
    if epilogue == MOE_EPI_SWIGLU_NVFP4:
        _at_least(C, "C", M * N // 2)
        _dev(C_sf, "C_sf", device=dev)
        _at_least(C_sf, "C_sf", M * N // 16)
        _dev(c_g, "c_g", dtype=torch.float32, device=dev)
        _at_least(c_g, "c_g", 4)
    elif epilogue == MOE_EPI_SWIGLU_MX:
        _at_least(C, "C", M * mx_c)
        _dev(C_sf, "C_sf", device=dev)
        _at_least(C_sf, "C_sf", M * N // 32)
    else:
        _at_least(C, "C", M * N * 2)
    check(load().moe_grouped_gemm(a_fmt, w_fmt, epilogue, G, _ptr(offsets), M, N, K, _ptr(A), _ptr(A_sf),
                                  _ptr(A_g), _ptr(W), _ptr(W_sf), _ptr(W_g), _ptr(C), _ptr(C_sf), _ptr(c_g),
                                  _stream(stream)), "moe_grouped_gemm")
    return (C, C_sf) if epilogue in (MOE_EPI_SWIGLU_NVFP4, MOE_EPI_SWIGLU_MX) else C


def moe_combine(Y: torch.Tensor, row_of: torch.Tensor, w: torch.Tensor, Ys: Optional[torch.Tensor],
                T: int, k: int, H: int, out: Optional[torch.Tensor] = None, stream=None,
                ys_gate: Optional[torch.Tensor] = None):
    """ys_gate: fp32 [T] per-token factor of the shared row (moe_combine_gated)."""
    _dev(Y, "Y", dtype=torch.bfloat16)
    dev = Y.device
    _at_least(Y, "Y", T * k * H * 2)
    _dev(row_of, "row_of", dtype=torch.int32, device=dev)
    _at_least(row_of, "row_of", T * k * 4)
    _dev(w, "w", dtype=torch.float32, device=dev)
    _at_least(w, "w", T * k * 4)
    _opt(Ys, "Ys", dtype=torch.bfloat16, shape=(T, H), device=dev)
    _opt(ys_gate, "ys_gate", dtype=torch.float32, shape=(T,), device=dev)
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    _dev(out, "out", dtype=torch.bfloat16, shape=(T, H), device=dev)
    if ys_gate is None:
        check(load().moe_combine(_ptr(Y), _ptr(row_of), _ptr(w), _ptr(Ys), T, k, H, _ptr(out), _stream(stream)),
              "moe_combine")
    else:
        check(load().moe_combine_gated(_ptr(Y), _ptr(row_of), _ptr(w), _ptr(Ys), _ptr(ys_gate), T, k, H,
                                       _ptr(out), _stream(stream)), "moe_combine_gated")
    return out


def moe_shared_gate(x: torch.Tensor, g: torch.Tensor, gate: Optional[torch.Tensor] = None, stream=None):
    """x bf16 [T, H], g bf16 [H] -> gate fp32 [T] = sigmoid(x . g)."""
    _dev(x, "x", dtype=torch.bfloat16)
    if x.dim() != 2:
        raise ValueError("x: expected [T, H]")
    T, H = x.shape
    _dev(g, "g", dtype=torch.bfloat16, shape=(H,), device=x.device)
    if gate is None:
        gate = torch.empty(T, dtype=torch.float32, device=x.device)
    _dev(gate, "gate", dtype=torch.float32, shape=(T,), device=x.device)
    check(load().moe_shared_gate(_ptr(x), _ptr(g), T, H, _ptr(gate), _stream(stream)), "moe_shared_gate")
    return gate


def moe_forward_workspace_size(layer_c, T: int) -> int:
    import ctypes
    return int(load().moe_forward_workspace_size(ctypes.byref(layer_c), T))


def _host(t: torch.Tensor, name: str, dtype, shape) -> None:
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise ValueError(f"{name}: expected a host (CPU) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _forward_args(layer_c, x: torch.Tensor, logits: torch.Tensor, out: torch.Tensor, ws: torch.Tensor) -> int:
    """Checks the device buffers of a whole-layer call against the layer's
    H and E; returns T."""
    _dev(x, "x", dtype=torch.bfloat16)
    if x.dim() != 2 or x.shape[1] != layer_c.H:
        raise ValueError(f"x: expected [T, {layer_c.H}]")
    T = x.shape[0]
    dev = x.device
    _dev(logits, "logits", dtype=torch.float32, shape=(T, layer_c.E), device=dev)
    _dev(out, "out", dtype=torch.bfloat16, shape=(T, layer_c.H), device=dev)
    _dev(ws, "ws", device=dev)
    _at_least(ws, "ws", moe_forward_workspace_size(layer_c, T))
    return T


def moe_forward(layer_c, x: torch.Tensor, logits: torch.Tensor, out: torch.Tensor, ws: torch.Tensor,
                stream=None) -> torch.Tensor:
    import ctypes
    T = _forward_args(layer_c, x, logits, out, ws)
    check(load().moe_forward(ctypes.byref(layer_c), _ptr(x), _ptr(logits), T, _ptr(out), _ptr(ws),
                             ws.numel(), _stream(stream)), "moe_forward")
    return out


def moe_forward_profiled(layer_c, x: torch.Tensor, logits: torch.Tensor, out: torch.Tensor, ws: torch.Tensor,
                         events, stream=None) -> torch.Tensor:
    """moe_forward recording 6 torch.cuda.Event objects at the stage
    boundaries: start, after the activation quantisation, after the router
    top-k and permutation, after each grouped GEMM, after the combine (see
    include/moe_gb300.h)."""
    import ctypes
    if len(events) != 6:
        raise ValueError("events: expected 6 torch.cuda.Event objects")
    T = _forward_args(layer_c, x, logits, out, ws)
    handles = (ctypes.c_void_p * 6)(*[ev.cuda_event for ev in events])
    check(load().moe_forward_profiled(ctypes.byref(layer_c), _ptr(x), _ptr(logits), T, _ptr(out), _ptr(ws),
                                      ws.numel(), handles, _stream(stream)), "moe_forward_profiled")
    return out


def moe_forward_host(layer_c, x_host: torch.Tensor, logits_host: torch.Tensor, out_host: torch.Tensor,
                     x_dev: torch.Tensor, logits_dev: torch.Tensor, out_dev: torch.Tensor,
                     ws: torch.Tensor, stream=None) -> torch.Tensor:
    import ctypes
    T = _forward_args(layer_c, x_dev, logits_dev, out_dev, ws)
    _host(x_host, "x_host", torch.bfloat16, (T, layer_c.H))
    _host(logits_host, "logits_host", torch.float32, (T, layer_c.E))
    _host(out_host, "out_host", torch.bfloat16, (T, layer_c.H))
    check(load().moe_forward_host(ctypes.byref(layer_c), _ptr(x_host), _ptr(logits_host), T, _ptr(out_host),
                                  _ptr(x_dev), _ptr(logits_dev), _ptr(out_dev), _ptr(ws), ws.numel(),
                                  _stream(stream)), "moe_forward_host")
    return out_host


def moe_forward_host_pipelined(layer_c, x_host, logits_host, out_host, x_dev: torch.Tensor,
                               logits_dev: torch.Tensor, out_dev: torch.Tensor, ws: torch.Tensor, stream=None,
                               copy_stream=None):
    """n batches of T tokens through moe_forward_host_pipelined: x_host,
    logits_host, out_host are lists of n pinned host tensors (bf16 [T,H],
    fp32 [T,E], bf16 [T,H]); x_dev / logits_dev / out_dev hold two batches
    ([2,T,H], [2,T,E], [2,T,H]).  The layer runs on `stream`, the copies on
    `copy_stream` (a torch.cuda.Stream other than `stream`)."""
    import ctypes
    n = len(x_host)
    if n < 1 or len(logits_host) != n or len(out_host) != n:
        raise ValueError("x_host, logits_host, out_host: n >= 1 host tensors each")
    for nm, t, dt in (("x_dev", x_dev, torch.bfloat16), ("logits_dev", logits_dev, torch.float32),
                      ("out_dev", out_dev, torch.bfloat16)):
        _dev(t, nm, dtype=dt)
        if t.dim() != 3 or t.shape[0] != 2:
            raise ValueError(f"{nm}: expected two batches [2, T, ...]")
    T = _forward_args(layer_c, x_dev[0], logits_dev[0], out_dev[0], ws)
    for i in range(n):
        _host(x_host[i], f"x_host[{i}]", torch.bfloat16, (T, layer_c.H))
        _host(logits_host[i], f"logits_host[{i}]", torch.float32, (T, layer_c.E))
        _host(out_host[i], f"out_host[{i}]", torch.bfloat16, (T, layer_c.H))
    if copy_stream is None:
        raise ValueError("copy_stream: required (a stream other than the compute stream)")
    if stream is None:
        stream = torch.cuda.current_stream()
    if copy_stream.cuda_stream == stream.cuda_stream:
        raise ValueError("copy_stream: must differ from the compute stream")
    ptrs = lambda ts: (ctypes.c_void_p * n)(*[t.data_ptr() for t in ts])
    check(load().moe_forward_host_pipelined(ctypes.byref(layer_c), n, ptrs(x_host), ptrs(logits_host), T,
                                            ptrs(out_host), _ptr(x_dev), _ptr(logits_dev), _ptr(out_dev),
                                            _ptr(ws), ws.numel(), stream.cuda_stream, copy_stream.cuda_stream),
          "moe_forward_host_pipelined")
    return out_host


def _empty(shape, dtype, device, stream=None) -> torch.Tensor:
    """An output or scratch tensor from the memory of the stream that will
    write it (another stream's free blocks may still be in use there)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _raw_stream(stream, t: torch.Tensor) -> int:
    """The cudaStream_t of `stream`, or of the current stream of t's device
    (without building a torch.cuda.Stream, which costs as much as a launch)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if stream is None else stream.cuda_stream


# The cache calls run once or more per layer and token, where the host's time is
# what counts: each looks at its tensors with these predicates (half the cost of
# the checks that name what is wrong) and falls back to those checks, which
# raise, only where one of them says no.
_INT_MAX = 2 ** 31 - 1  # a longer window is as good as none; ctypes would cut it off silently
_BF16, _F32, _I32, _I64, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


def _is(t, dtype, shape, device: int) -> bool:
    return t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous()


def _is_heads(t, T: int, D: int, device: int) -> bool:
    if t.dtype is not _BF16 or t.get_device() != device:
        return False
    n, h, d = t.shape
    _, sh, sd = t.stride()
    return n == T and d == D and sd == 1 and (sh == d or h == 1)


def _is_rows(t, dtype, rows: int, cols: int, device: int) -> bool:
    """[rows, cols] whose rows may be apart."""
    return (t.dtype is dtype and t.shape == (rows, cols) and t.get_device() == device
            and (t.stride(1) == 1 or cols == 1))


def _rows(t: torch.Tensor, name: str, dtype, rows=None, cols=None, device=None) -> None:
    """A matrix whose rows may be apart (a slice of another's columns)."""
    if t is None:
        raise ValueError(f"{name}: required")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name}: expected [{'rows' if rows is None else rows}, {'columns' if cols is None else cols}], "
                         f"got {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: each row must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _row_stride(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def moe_linear_nvfp4(x: torch.Tensor, codes: torch.Tensor, sf: torch.Tensor, g: torch.Tensor,
                     add: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                     out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Up to 32 tokens times a matrix in NVFP4 (see include/moe_gb300.h): x bf16
    [T, K] (rows on 16-byte boundaries), codes uint8 [N, K/2], sf uint8 [N, K/16], g fp32 [1]
    as moe_quant_nvfp4 gives them; add bf16 [T, N] (any row stride) is added
    before the one rounding.  Returns out [T, N], bf16 or fp32."""
    try:
        T, K = x.shape
        N, di = codes.shape[0], x.get_device()
        ok = (di >= 0 and _is_rows(x, _BF16, T, K, di) and _is(codes, _U8, (N, K // 2), di)
              and _is(sf, _U8, (N, K // 16), di) and _is(g, _F32, (1,), di) and K % 32 == 0
              and (add is None or _is_rows(add, _BF16, T, N, di)) and (out_dtype is _BF16 or out_dtype is _F32)
              and (out is None or _is(out, out_dtype, (T, N), di)) and (ws is None or _is(ws, ws.dtype, ws.shape, di)))
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        _rows(x, "x", torch.bfloat16)
        T, K = x.shape
        dev = x.device
        if K < 32 or K % 32:
            raise ValueError(f"x: expected a multiple of 32 columns, got {K}")
        _dev(codes, "codes", dtype=torch.uint8, device=dev)
        if codes.dim() != 2 or codes.shape[1] != K // 2:
            raise ValueError(f"codes: expected [N, {K // 2}], got {tuple(codes.shape)}")
        N = codes.shape[0]
        _dev(sf, "sf", dtype=torch.uint8, shape=(N, K // 16), device=dev)
        _dev(g, "g", dtype=torch.float32, shape=(1,), device=dev)
        if add is not None:
            _rows(add, "add", torch.bfloat16, T, N, dev)
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"out_dtype: expected torch.bfloat16 or torch.float32, got {out_dtype}")
        _opt(out, "out", dtype=out_dtype, shape=(T, N), device=dev)
        _opt(ws, "ws", device=dev)
    lib = load()
    if out is None:
        out = _empty((T, N), out_dtype, x.device, stream)
    nbytes = lib.moe_linear_nvfp4_workspace_size(T, K)
    if ws is None and nbytes:
        ws = _empty((nbytes,), _U8, x.device, stream)
    check(lib.moe_linear_nvfp4(x.data_ptr(), _row_stride(x), T, codes.data_ptr(), sf.data_ptr(), g.data_ptr(), N, K,
                               None if add is None else add.data_ptr(), 0 if add is None else _row_stride(add),
                               out.data_ptr(), 1 if out_dtype is _F32 else 0, None if ws is None else ws.data_ptr(),
                               0 if ws is None else ws.numel() * ws.element_size(), _raw_stream(stream, x)), "moe_linear_nvfp4")
    return out


def moe_verify_draft(logits: torch.Tensor, tokens: torch.Tensor, q_offsets: torch.Tensor, u: torch.Tensor,
                     u_next: torch.Tensor, draft_probs: Optional[torch.Tensor] = None,
                     temperature: Optional[torch.Tensor] = None, out: Optional[dict] = None,
                     ws: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Drafted tokens against the target's probabilities (see include/moe_gb300.h):
    logits bf16 or fp32 [T, V] and draft_probs fp32 [T, V] or None (any row stride),
    tokens int32 [T], q_offsets int32 [B + 1], u fp32 [T] and u_next fp32 [B] in
    [0, 1), temperature fp32 [B] or None.  Returns dict(accepted, token, refused),
    int32 [B]."""
    o = out or {}
    r = [o.get("accepted"), o.get("token"), o.get("refused")]
    try:
        T, V = logits.shape
        (B1,) = q_offsets.shape
        B, di = B1 - 1, logits.get_device()
        ok = (di >= 0 and B >= 0 and (logits.dtype is _BF16 or logits.dtype is _F32) and _is_rows(logits, logits.dtype, T, V, di)
              and _is(tokens, _I32, (T,), di) and _is(q_offsets, _I32, (B + 1,), di) and _is(u, _F32, (T,), di)
              and _is(u_next, _F32, (B,), di) and (draft_probs is None or _is_rows(draft_probs, _F32, T, V, di))
              and (temperature is None or _is(temperature, _F32, (B,), di))
              and all(t is None or _is(t, _I32, (B,), di) for t in r) and (ws is None or _is(ws, ws.dtype, ws.shape, di)))
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        if isinstance(logits, torch.Tensor) and logits.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"logits: expected torch.bfloat16 or torch.float32, got {logits.dtype}")
        _rows(logits, "logits", getattr(logits, "dtype", None))
        T, V = logits.shape
        dev = logits.device
        _dev(q_offsets, "q_offsets", dtype=torch.int32, device=dev)
        if q_offsets.dim() != 1 or q_offsets.numel() < 1:
            raise ValueError("q_offsets: expected [B + 1]")
        B = q_offsets.numel() - 1
        _dev(tokens, "tokens", dtype=torch.int32, shape=(T,), device=dev)
        _dev(u, "u", dtype=torch.float32, shape=(T,), device=dev)
        _dev(u_next, "u_next", dtype=torch.float32, shape=(B,), device=dev)
        if draft_probs is not None:
            _rows(draft_probs, "draft_probs", torch.float32, T, V, dev)
        _opt(temperature, "temperature", dtype=torch.float32, shape=(B,), device=dev)
        for name, t in zip(("accepted", "token", "refused"), r):
            _opt(t, name, dtype=torch.int32, shape=(B,), device=dev)
        _opt(ws, "ws", device=dev)
    lib, dev = load(), logits.device
    r = [_empty((B,), _I32, dev, stream) if t is None else t for t in r]
    if ws is None:
        ws = _empty(lib.moe_verify_draft_workspace_size(T, V, B), _U8, dev, stream)
    check(lib.moe_verify_draft(
        logits.data_ptr(), 1 if logits.dtype is _F32 else 0, _row_stride(logits), T, V, tokens.data_ptr(), q_offsets.data_ptr(), B,
        u.data_ptr(), u_next.data_ptr(), None if draft_probs is None else draft_probs.data_ptr(),
        0 if draft_probs is None else _row_stride(draft_probs), None if temperature is None else temperature.data_ptr(),
        r[0].data_ptr(), r[1].data_ptr(), r[2].data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
        _raw_stream(stream, logits)), "moe_verify_draft")
    return dict(accepted=r[0], token=r[1], refused=r[2])


def _heads(t: torch.Tensor, name: str, T=None, D=None, device=None) -> None:
    """bf16 [T, heads, D] whose tokens may be apart (a slice of a projection's
    output): heads and D contiguous, any token stride."""
    if t is None:
        raise ValueError(f"{name}: required")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name}: expected torch.bfloat16, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name}: expected [T, heads, D]")
    s, h, d = t.stride(), t.shape[1], t.shape[2]
    if (d > 1 and s[2] != 1) or (h > 1 and s[1] != d):
        raise ValueError(f"{name}: heads must be contiguous within a token")
    if T is not None and t.shape[0] != T:
        raise ValueError(f"{name}: expected {T} tokens, got {t.shape[0]}")
    if D is not None and d != D:
        raise ValueError(f"{name}: expected head size {D}, got {d}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _token_stride(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def _pool_page_size(pool: torch.Tensor, Hkv: int, D: int, device) -> int:
    """The page size of a layer's pool uint8 [num_pages, Hkv, page_size*D*9/8]."""
    _dev(pool, "pool", dtype=torch.uint8, device=device)
    if pool.dim() != 3 or pool.shape[1] != Hkv or pool.shape[2] * 8 % (9 * D):
        raise ValueError(f"pool: expected [num_pages, {Hkv}, page_size * {D} * 9 / 8], got {tuple(pool.shape)}")
    return pool.shape[2] * 8 // (9 * D)


def moe_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, cos_sin: Optional[torch.Tensor] = None,
                     pos: Optional[torch.Tensor] = None, wq: Optional[torch.Tensor] = None,
                     wk: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
                     v: Optional[torch.Tensor] = None, pool: Optional[torch.Tensor] = None,
                     g_k: Optional[torch.Tensor] = None, g_v: Optional[torch.Tensor] = None,
                     slots: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                     k_out: Optional[torch.Tensor] = None, stream=None):
    """Per-head RMS norms of q and k, the rotation, and the NVFP4 write of k and
    v into the cache (see include/moe_gb300.h).  q bf16 [T, Hq, D], k and v
    bf16 [T, Hkv, D] (any token stride); wq / wk bf16 [D] or None; cos_sin fp32
    [max_pos, rot] with pos int32 [T], or None for no rotation; pool uint8
    [num_pages, Hkv, record] with g_k, g_v fp32 [Hkv] and slots int64 [T].
    Returns (q_out, k_out); k_out is allocated only where there is no pool."""
    try:
        T, Hq, D = q.shape
        di, Hkv, page_bytes = q.get_device(), k.shape[1], 0
        ok = (di >= 0 and D > 0 and _is_heads(q, T, D, di) and _is_heads(k, T, D, di)
              and (wq is None or _is(wq, _BF16, (D,), di)) and (wk is None or _is(wk, _BF16, (D,), di)))
        if ok and cos_sin is not None:
            max_pos, rot = cos_sin.shape
            ok = _is(cos_sin, _F32, (max_pos, rot), di) and _is(pos, _I32, (T,), di)
        if ok and pool is not None:
            num_pages, _, page_bytes = pool.shape
            ok = (_is(pool, _U8, (num_pages, Hkv, page_bytes), di) and page_bytes * 8 % (9 * D) == 0
                  and _is_heads(v, T, D, di) and v.shape[1] == Hkv and _is(g_k, _F32, (Hkv,), di)
                  and _is(g_v, _F32, (Hkv,), di) and _is(slots, _I64, (T,), di))
        ok = ok and (q_out is None or _is(q_out, _BF16, (T, Hq, D), di)) and (
            k_out is None or _is(k_out, _BF16, (T, Hkv, D), di))
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        _check_qk_norm_rope(q, k, cos_sin, pos, wq, wk, v, pool, g_k, g_v, slots, q_out, k_out)
        T, Hq, D = q.shape
        Hkv, page_bytes = k.shape[1], 0 if pool is None else pool.shape[2]
    if cos_sin is None:
        max_pos = rot = 0
    else:
        max_pos, rot = cos_sin.shape
    dev = q.device
    if q_out is None:
        q_out = _empty((T, Hq, D), _BF16, dev, stream)
    if k_out is None and pool is None:
        k_out = _empty((T, Hkv, D), _BF16, dev, stream)
    cache = pool is not None
    check(load().moe_qk_norm_rope(
        q.data_ptr(), _token_stride(q), k.data_ptr(), _token_stride(k), v.data_ptr() if cache else None,
        _token_stride(v) if cache else 0, T, Hq, Hkv, D, None if wq is None else wq.data_ptr(),
        None if wk is None else wk.data_ptr(), eps, None if cos_sin is None else cos_sin.data_ptr(), max_pos, rot,
        1 if interleaved else 0, None if pos is None else pos.data_ptr(), q_out.data_ptr(),
        None if k_out is None else k_out.data_ptr(), pool.data_ptr() if cache else None, pool.shape[0] if cache else 0,
        page_bytes * 8 // (9 * D) if cache else 0, g_k.data_ptr() if cache else None, g_v.data_ptr() if cache else None,
        slots.data_ptr() if cache else None, _raw_stream(stream, q)), "moe_qk_norm_rope")
    return q_out, k_out


def _check_qk_norm_rope(q, k, cos_sin, pos, wq, wk, v, pool, g_k, g_v, slots, q_out, k_out) -> None:
    """Raises what is wrong with moe_qk_norm_rope's arguments."""
    _heads(q, "q")
    T, Hq, D = q.shape
    dev = q.device
    _heads(k, "k", T, D, dev)
    Hkv = k.shape[1]
    _opt(wq, "wq", dtype=torch.bfloat16, shape=(D,), device=dev)
    _opt(wk, "wk", dtype=torch.bfloat16, shape=(D,), device=dev)
    if cos_sin is not None:
        _dev(cos_sin, "cos_sin", dtype=torch.float32, device=dev)
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin: expected [max_pos, rot]")
        _dev(pos, "pos", dtype=torch.int32, shape=(T,), device=dev)
    if pool is not None:
        _pool_page_size(pool, Hkv, D, dev)
        _heads(v, "v", T, D, dev)
        if v.shape[1] != Hkv:
            raise ValueError(f"v: expected {Hkv} heads, got {v.shape[1]}")
        _dev(g_k, "g_k", dtype=torch.float32, shape=(Hkv,), device=dev)
        _dev(g_v, "g_v", dtype=torch.float32, shape=(Hkv,), device=dev)
        _dev(slots, "slots", dtype=torch.int64, shape=(T,), device=dev)
    _opt(q_out, "q_out", dtype=torch.bfloat16, shape=(T, Hq, D), device=dev)
    _opt(k_out, "k_out", dtype=torch.bfloat16, shape=(T, Hkv, D), device=dev)


def moe_kv4_attention(q: torch.Tensor, pool: torch.Tensor, g_k: torch.Tensor, g_v: torch.Tensor,
                      q_offsets: torch.Tensor, kv_lens: torch.Tensor, table: torch.Tensor,
                      scale: Optional[float] = None, causal: bool = True, window: int = 0,
                      out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of a ragged batch over the paged NVFP4 cache (see
    include/moe_gb300.h).  q bf16 [T, Hq, D] (any token stride), pool uint8
    [num_pages, Hkv, record], q_offsets int32 [B + 1], kv_lens int32 [B],
    table int32 [B, max_pages]; scale defaults to D ** -0.5; lse fp32 [T, Hq]
    is written where given.  Returns out bf16 [T, Hq, D]."""
    try:
        T, Hq, D = q.shape
        num_pages, Hkv, page_bytes = pool.shape
        B, max_pages = table.shape
        di = q.get_device()
        ok = (di >= 0 and D > 0 and _is_heads(q, T, D, di) and _is(pool, _U8, (num_pages, Hkv, page_bytes), di)
              and page_bytes * 8 % (9 * D) == 0 and _is(g_k, _F32, (Hkv,), di) and _is(g_v, _F32, (Hkv,), di)
              and _is(table, _I32, (B, max_pages), di) and _is(q_offsets, _I32, (B + 1,), di)
              and _is(kv_lens, _I32, (B,), di) and (out is None or _is(out, _BF16, (T, Hq, D), di))
              and (lse is None or _is(lse, _F32, (T, Hq), di)) and (ws is None or _is(ws, ws.dtype, ws.shape, di)))
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        _check_kv4_attention(q, pool, g_k, g_v, q_offsets, kv_lens, table, out, lse, ws)
        T, Hq, D = q.shape
        num_pages, Hkv, page_bytes = pool.shape
        B, max_pages = table.shape
    lib, dev = load(), q.device
    if out is None:
        out = _empty((T, Hq, D), _BF16, dev, stream)
    if ws is None:
        ws = _empty(lib.moe_kv4_attention_workspace_size(T, B, Hq, Hkv, D), _U8, dev, stream)
    check(lib.moe_kv4_attention(
        q.data_ptr(), _token_stride(q), T, Hq, pool.data_ptr(), num_pages, page_bytes * 8 // (9 * D), Hkv, D,
        g_k.data_ptr(), g_v.data_ptr(), q_offsets.data_ptr(), kv_lens.data_ptr(), table.data_ptr(), B, max_pages,
        D ** -0.5 if scale is None else scale, 1 if causal else 0, min(window, _INT_MAX), out.data_ptr(),
        None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(), _raw_stream(stream, q)),
        "moe_kv4_attention")
    return out


def _check_kv4_attention(q, pool, g_k, g_v, q_offsets, kv_lens, table, out, lse, ws) -> None:
    """Raises what is wrong with moe_kv4_attention's arguments."""
    _heads(q, "q")
    T, Hq, D = q.shape
    dev = q.device
    _dev(g_k, "g_k", dtype=torch.float32, device=dev)
    Hkv = g_k.numel()
    _dev(g_v, "g_v", dtype=torch.float32, shape=(Hkv,), device=dev)
    _pool_page_size(pool, Hkv, D, dev)
    _dev(table, "table", dtype=torch.int32, device=dev)
    if table.dim() != 2:
        raise ValueError("table: expected [B, max_pages]")
    B = table.shape[0]
    _dev(q_offsets, "q_offsets", dtype=torch.int32, shape=(B + 1,), device=dev)
    _dev(kv_lens, "kv_lens", dtype=torch.int32, shape=(B,), device=dev)
    _opt(out, "out", dtype=torch.bfloat16, shape=(T, Hq, D), device=dev)
    _opt(lse, "lse", dtype=torch.float32, shape=(T, Hq), device=dev)
    _opt(ws, "ws", device=dev)


def moe_kv4_weights(q: torch.Tensor, pool: torch.Tensor, g_k: torch.Tensor, lse: torch.Tensor, q_offsets: torch.Tensor,
                    kv_lens: torch.Tensor, table: torch.Tensor, score: torch.Tensor, scale: Optional[float] = None,
                    causal: bool = True, window: int = 0, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Adds the weights that a step's attention gave to each key to score fp32
    [B, Hkv, cap], cap >= max_pages * page_size (see include/moe_gb300.h).  lse fp32
    [T, Hq] as moe_kv4_attention wrote it, the other arguments as it took them.
    Returns score."""
    try:
        T, Hq, D = q.shape
        num_pages, Hkv, page_bytes = pool.shape
        B, max_pages = table.shape
        di, cap = q.get_device(), score.shape[2]
        ok = (di >= 0 and D > 0 and _is_heads(q, T, D, di) and _is(pool, _U8, (num_pages, Hkv, page_bytes), di)
              and page_bytes * 8 % (9 * D) == 0 and _is(g_k, _F32, (Hkv,), di) and _is(lse, _F32, (T, Hq), di)
              and _is(table, _I32, (B, max_pages), di) and _is(q_offsets, _I32, (B + 1,), di)
              and _is(kv_lens, _I32, (B,), di) and _is(score, _F32, (B, Hkv, cap), di)
              and cap >= max_pages * (page_bytes * 8 // (9 * D)) and (ws is None or _is(ws, ws.dtype, ws.shape, di)))
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok:
        _check_kv4_weights(q, pool, g_k, lse, q_offsets, kv_lens, table, score, ws)
        T, Hq, D = q.shape
        num_pages, Hkv, page_bytes = pool.shape
        B, max_pages = table.shape
        cap = score.shape[2]
    lib = load()
    if ws is None:
        ws = _empty(lib.moe_kv4_weights_workspace_size(T, B, Hq, Hkv, D), _U8, q.device, stream)
    check(lib.moe_kv4_weights(
        q.data_ptr(), _token_stride(q), T, Hq, pool.data_ptr(), num_pages, page_bytes * 8 // (9 * D), Hkv, D,
        g_k.data_ptr(), lse.data_ptr(), q_offsets.data_ptr(), kv_lens.data_ptr(), table.data_ptr(), B, max_pages,
        D ** -0.5 if scale is None else scale, 1 if causal else 0, min(window, _INT_MAX), score.data_ptr(), cap,
        ws.data_ptr(), ws.numel() * ws.element_size(), _raw_stream(stream, q)), "moe_kv4_weights")
    return score


def _check_kv4_weights(q, pool, g_k, lse, q_offsets, kv_lens, table, score, ws) -> None:
    """Raises what is wrong with moe_kv4_weights' arguments."""
    _heads(q, "q")
    T, Hq, D = q.shape
    dev = q.device
    _dev(g_k, "g_k", dtype=torch.float32, device=dev)
    Hkv = g_k.numel()
    page = _pool_page_size(pool, Hkv, D, dev)
    _dev(lse, "lse", dtype=torch.float32, shape=(T, Hq), device=dev)
    _dev(table, "table", dtype=torch.int32, device=dev)
    if table.dim() != 2:
        raise ValueError("table: expected [B, max_pages]")
    B = table.shape[0]
    _dev(q_offsets, "q_offsets", dtype=torch.int32, shape=(B + 1,), device=dev)
    _dev(kv_lens, "kv_lens", dtype=torch.int32, shape=(B,), device=dev)
    _dev(score, "score", dtype=torch.float32, device=dev)
    if score.dim() != 3 or score.shape[:2] != (B, Hkv) or score.shape[2] < table.shape[1] * page:
        raise ValueError(f"score: expected [{B}, {Hkv}, >= {table.shape[1] * page}], got {tuple(score.shape)}")
    _opt(ws, "ws", device=dev)


def _kv_state(table, refs, lens=None):
    """Checks the arrays of the page operations; returns rows, max_pages, num_pages."""
    try:
        S, M = table.shape
        (N,) = refs.shape
        di = table.get_device()
        if (di >= 0 and _is(table, _I32, (S, M), di) and _is(refs, _I32, (N,), di)
                and (lens is None or _is(lens, _I32, (S,), di))):
            return S, M, N
    except (AttributeError, ValueError):
        pass
    _dev(table, "table", dtype=torch.int32)
    if table.dim() != 2:
        raise ValueError("table: expected [rows, max_pages]")
    _dev(refs, "refs", dtype=torch.int32, device=table.device)
    if refs.dim() != 1:
        raise ValueError("refs: expected [num_pages]")
    if lens is not None:
        _dev(lens, "lens", dtype=torch.int32, shape=(table.shape[0],), device=table.device)
    return table.shape[0], table.shape[1], refs.numel()


def _kv_pools(pool: Optional[torch.Tensor], num_pages: int, device):
    """(pointer, layers, bytes between layers, bytes of a page) of uint8 [layers, num_pages, ...] or None."""
    if pool is None:
        return None, 0, 0, 16
    try:
        ok = pool.dtype is _U8 and pool.device == device and pool.is_contiguous()
    except AttributeError:
        ok = False
    if not ok:
        _dev(pool, "pool", dtype=torch.uint8, device=device)
    if pool.dim() < 3 or pool.shape[1] != num_pages:
        raise ValueError(f"pool: expected [layers, {num_pages}, ...], got {tuple(pool.shape)}")
    layers = pool.shape[0]
    page = pool.numel() // (layers * num_pages) if layers and num_pages else 16
    return pool.data_ptr(), layers, page * num_pages, page


def _index(t: torch.Tensor, name: str, device) -> int:
    try:
        if t.dtype is _I32 and t.dim() == 1 and t.device == device and t.is_contiguous():
            return t.numel()
    except AttributeError:
        pass
    _dev(t, name, dtype=torch.int32, device=device)
    if t.dim() != 1:
        raise ValueError(f"{name}: expected one dimension")
    return t.numel()


def _like(out, name, t, inplace, stream):
    """The output of a page operation: the given one, the input in place, or a new one."""
    if out is not None:
        _dev(out, name, dtype=t.dtype, shape=t.shape, device=t.device)
        return out
    if inplace:
        return t
    return torch.empty_like(t) if stream is None else _empty(t.shape, t.dtype, t.device, stream)


def moe_kv_extend(q_offsets: torch.Tensor, T: int, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                  page_size: int, inplace: bool = False, out: Optional[dict] = None, stream=None) -> dict:
    """Room for new tokens: row r gets tokens q_offsets[r] .. q_offsets[r+1]
    (int32 [rows + 1], T tokens in all).  Returns dict(table, lens, refs,
    slots int64 [T], pos int32 [T]); inplace=True writes the state back into
    the arguments, `out` may hold any of the outputs."""
    return _kv_extend(q_offsets, T, table, lens, refs, page_size, inplace, out, None, stream)


def moe_kv_extend_ex(q_offsets: torch.Tensor, T: int, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                     page_size: int, inplace: bool = False, out: Optional[dict] = None, stream=None) -> dict:
    """moe_kv_extend, and kv_lens int32 [rows]: the lengths for this step's
    attention, 0 for a row that found no room (a new tensor, or out's)."""
    kv_lens = (out or {}).get("kv_lens")
    if kv_lens is None:
        kv_lens = torch.empty_like(lens) if stream is None else _empty(lens.shape, lens.dtype, lens.device, stream)
    r = _kv_extend(q_offsets, T, table, lens, refs, page_size, inplace, out, kv_lens, stream)
    r["kv_lens"] = kv_lens
    return r


def _kv_extend(q_offsets, T, table, lens, refs, page_size, inplace, out, kv_lens, stream) -> dict:
    S, M, N = _kv_state(table, refs, lens)
    dev = table.device
    try:
        di = table.get_device()
        ok = _is(q_offsets, _I32, (S + 1,), di) and (kv_lens is None or _is(kv_lens, _I32, (S,), di))
    except AttributeError:
        ok = False
    if not ok:
        _dev(q_offsets, "q_offsets", dtype=torch.int32, shape=(S + 1,), device=dev)
        _opt(kv_lens, "kv_lens", dtype=torch.int32, shape=(S,), device=dev)
    o = out or {}
    r = dict(table=_like(o.get("table"), "table", table, inplace, stream),
             lens=_like(o.get("lens"), "lens", lens, inplace, stream),
             refs=_like(o.get("refs"), "refs", refs, inplace, stream), slots=o.get("slots"), pos=o.get("pos"))
    for name, dt in (("slots", torch.int64), ("pos", torch.int32)):
        if r[name] is None:
            r[name] = _empty((T,), dt, dev, stream)
        else:
            _dev(r[name], name, dtype=dt, shape=(T,), device=dev)
    if S == 0:  # no row has the tokens
        with torch.cuda.stream(stream):
            r["slots"].fill_(-1)
            r["pos"].zero_()
    lib = load()
    ws = _empty(lib.moe_kv_pages_workspace_size(N, S), torch.uint8, dev, stream)
    check(lib.moe_kv_extend_ex(_ptr(q_offsets), T, _ptr(table), _ptr(lens), _ptr(refs), S, M, N, page_size,
                               _ptr(r["table"]), _ptr(r["lens"]), _ptr(r["refs"]), _ptr(r["slots"]), _ptr(r["pos"]),
                               _ptr(kv_lens), _ptr(ws), ws.numel(), _raw_stream(stream, table)), "moe_kv_extend")
    return r


def moe_kv_fork(src: torch.Tensor, dst: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                pool: Optional[torch.Tensor] = None, page_size: int = 64, inplace: bool = False,
                out: Optional[dict] = None, stream=None) -> dict:
    """Rows dst (empty, distinct) become forks of rows src (int32 [n] both).
    pool uint8 [layers, num_pages, ...] gets the copies of the partial pages.
    Returns dict(table, lens, refs)."""
    S, M, N = _kv_state(table, refs, lens)
    dev = table.device
    n = _index(src, "src", dev)
    if _index(dst, "dst", dev) != n:
        raise ValueError("dst: expected as many rows as src")
    if n > 0 and S == 0:
        raise ValueError("src: the table has no rows")
    base, layers, layer_stride, page_bytes = _kv_pools(pool, N, dev)
    o = out or {}
    r = dict(table=_like(o.get("table"), "table", table, inplace, stream),
             lens=_like(o.get("lens"), "lens", lens, inplace, stream),
             refs=_like(o.get("refs"), "refs", refs, inplace, stream))
    lib = load()
    ws = _empty(lib.moe_kv_pages_workspace_size(N, max(S, n)), torch.uint8, dev, stream)
    check(lib.moe_kv_fork(_ptr(src), _ptr(dst), n, _ptr(table), _ptr(lens), _ptr(refs), S, M, N, page_size,
                          _ptr(r["table"]), _ptr(r["lens"]), _ptr(r["refs"]), base, layers, layer_stride, page_bytes,
                          _ptr(ws), ws.numel(), _raw_stream(stream, table)), "moe_kv_fork")
    return r


def moe_kv_free(rows: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, page_size: int = 64,
                inplace: bool = False, out: Optional[dict] = None, stream=None) -> dict:
    """Rows (int32 [n]) become empty.  Returns dict(table, lens, refs)."""
    S, M, N = _kv_state(table, refs, lens)
    n = _index(rows, "rows", table.device)
    if n > 0 and S == 0:
        raise ValueError("rows: the table has no rows")
    o = out or {}
    r = dict(table=_like(o.get("table"), "table", table, inplace, stream),
             lens=_like(o.get("lens"), "lens", lens, inplace, stream),
             refs=_like(o.get("refs"), "refs", refs, inplace, stream))
    check(load().moe_kv_free(_ptr(rows), n, _ptr(table), _ptr(lens), _ptr(refs), S, M, N, page_size,
                             _ptr(r["table"]), _ptr(r["lens"]), _ptr(r["refs"]), _raw_stream(stream, table)), "moe_kv_free")
    return r


def moe_kv_drop(drop: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                pool: Optional[torch.Tensor] = None, page_size: int = 64, inplace: bool = False,
                out: Optional[dict] = None, stream=None) -> dict:
    """Each row loses its last drop[row] tokens (int32 [rows]).  pool uint8
    [layers, num_pages, ...] gets a copy of a page that a row then ends inside of
    and shares with another.  Returns dict(table, lens, refs)."""
    S, M, N = _kv_state(table, refs, lens)
    dev = table.device
    if _index(drop, "drop", dev) != S:
        raise ValueError(f"drop: expected {S} numbers, one per row")
    base, layers, layer_stride, page_bytes = _kv_pools(pool, N, dev)
    o = out or {}
    r = dict(table=_like(o.get("table"), "table", table, inplace, stream),
             lens=_like(o.get("lens"), "lens", lens, inplace, stream),
             refs=_like(o.get("refs"), "refs", refs, inplace, stream))
    lib = load()
    ws = _empty(lib.moe_kv_pages_workspace_size(N, S), torch.uint8, dev, stream)
    check(lib.moe_kv_drop(_ptr(drop), _ptr(table), _ptr(lens), _ptr(refs), S, M, N, page_size, _ptr(r["table"]),
                          _ptr(r["lens"]), _ptr(r["refs"]), base, layers, layer_stride, page_bytes, _ptr(ws), ws.numel(),
                          _raw_stream(stream, table)), "moe_kv_drop")
    return r


def moe_kv4_evict(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, pool: torch.Tensor,
                  score: Optional[torch.Tensor], keep: int, limit: Optional[int] = None, sinks: int = 0, recent: int = 0,
                  D: int = 128, inplace: bool = False, out: Optional[dict] = None, stream=None) -> dict:
    """Rows with more than `limit` (default: keep) tokens keep `keep`: the first
    `sinks`, the last `recent`, and the ones with the largest sums between them,
    chosen by every layer and kv head for itself (see include/moe_gb300.h).  pool
    uint8 [layers, num_pages, Hkv, record] and score fp32 [layers, rows, Hkv, cap],
    cap >= max_pages * page_size, are moved in place; score may be None where
    sinks + recent == keep.  Returns dict(table, lens, refs, dropped int32 [rows])."""
    S, M, N = _kv_state(table, refs, lens)
    dev = table.device
    _dev(pool, "pool", dtype=torch.uint8, device=dev)
    if pool.dim() != 4 or pool.shape[1] != N or D < 1 or pool.shape[3] * 8 % (9 * D):
        raise ValueError(f"pool: expected [layers, {N}, Hkv, page_size * {D} * 9 / 8], got {tuple(pool.shape)}")
    layers, _, Hkv, record = pool.shape
    page_size = record * 8 // (9 * D)
    cap = 0
    if score is not None:
        _dev(score, "score", dtype=torch.float32, device=dev)
        if score.dim() != 4 or score.shape[:3] != (layers, S, Hkv) or score.shape[3] < M * page_size:
            raise ValueError(f"score: expected [{layers}, {S}, {Hkv}, >= {M * page_size}], got {tuple(score.shape)}")
        cap = score.shape[3]
    # more tokens than any row has; ctypes would cut such numbers off silently
    keep, limit, sinks, recent = (max(-1, min(n, _INT_MAX)) for n in (keep, keep if limit is None else limit, sinks, recent))
    o = out or {}
    r = dict(table=_like(o.get("table"), "table", table, inplace, stream),
             lens=_like(o.get("lens"), "lens", lens, inplace, stream),
             refs=_like(o.get("refs"), "refs", refs, inplace, stream),
             dropped=_like(o.get("dropped"), "dropped", lens, False, stream))
    lib = load()
    ws = _empty(lib.moe_kv4_evict_workspace_size(layers, S, M, N, Hkv, max(keep, 1)), _U8, dev, stream)
    check(lib.moe_kv4_evict(_ptr(table), _ptr(lens), _ptr(refs), S, M, N, page_size, _ptr(r["table"]), _ptr(r["lens"]),
                            _ptr(r["refs"]), _ptr(r["dropped"]), _ptr(pool), layers, N * Hkv * record, Hkv, D, _ptr(score), cap,
                            keep, limit, sinks, recent, _ptr(ws), ws.numel(), _raw_stream(stream, table)),
          "moe_kv4_evict")
    return r


def moe_kv_compact(table: torch.Tensor, refs: torch.Tensor, pool: Optional[torch.Tensor] = None,
                   inplace: bool = False, out: Optional[dict] = None, stream=None) -> dict:
    """Moves the pages in use to the lowest ids (in pool uint8 [layers,
    num_pages, ...] too).  Returns dict(table, refs, remap int32 [num_pages])."""
    S, M, N = _kv_state(table, refs)
    dev = table.device
    base, layers, layer_stride, page_bytes = _kv_pools(pool, N, dev)
    o = out or {}
    r = dict(table=_like(o.get("table"), "table", table, inplace, stream),
             refs=_like(o.get("refs"), "refs", refs, inplace, stream), remap=_like(o.get("remap"), "remap", refs, False, stream))
    lib = load()
    ws = _empty(lib.moe_kv_pages_workspace_size(N, 0), torch.uint8, dev, stream)
    check(lib.moe_kv_compact(_ptr(table), _ptr(refs), S, M, N, _ptr(r["table"]), _ptr(r["refs"]), _ptr(r["remap"]),
                             base, layers, layer_stride, page_bytes, _ptr(ws), ws.numel(), _raw_stream(stream, table)),
          "moe_kv_compact")
    return r


def moe_kv_copy_pages(pool: torch.Tensor, src: torch.Tensor, dst: torch.Tensor, stream=None) -> torch.Tensor:
    """Copies pages src to pages dst (int32 [n]) in every layer of pool uint8 [layers, num_pages, ...]."""
    if pool is None or not isinstance(pool, torch.Tensor) or not pool.is_cuda or pool.dim() < 3:
        raise ValueError("pool: expected a CUDA tensor [layers, num_pages, ...]")
    base, layers, layer_stride, page_bytes = _kv_pools(pool, pool.shape[1], pool.device)
    n = _index(src, "src", pool.device)
    if _index(dst, "dst", pool.device) != n:
        raise ValueError("dst: expected as many pages as src")
    check(load().moe_kv_copy_pages(base, layers, layer_stride, page_bytes, pool.shape[1], _ptr(src), _ptr(dst), n,
                                   _raw_stream(stream, pool)), "moe_kv_copy_pages")
    return pool


__all__ = ["MOE_FMT_BF16", "MOE_FMT_NVFP4", "MOE_FMT_MXFP8", "MOE_FMT_MXFP4", "moe_quant_mx", "MOE_EPI_STORE_BF16", "MOE_EPI_SWIGLU_BF16",
           "MOE_EPI_SWIGLU_NVFP4", "moe_version", "moe_sync_status", "moe_set_wait_timeout_ns",
           "moe_selftest_wait_timeout", "moe_selftest_attention_wait_timeout", "moe_selftest_grid_barrier_timeout", "moe_route", "moe_permute",
           "moe_route_permute", "moe_quant_nvfp4", "MOE_EPI_SWIGLU_MX",
           "moe_permute_noalloc", "moe_grouped_gemm", "moe_combine", "moe_shared_gate",
           "moe_forward_workspace_size", "moe_forward", "moe_forward_profiled", "moe_forward_host",
           "moe_forward_host_pipelined", "moe_linear_nvfp4", "moe_verify_draft", "moe_qk_norm_rope", "moe_kv4_attention", "moe_kv4_weights", "moe_kv_extend", "moe_kv_extend_ex", "moe_kv_fork",
           "moe_kv_free", "moe_kv_drop", "moe_kv4_evict", "moe_kv_compact", "moe_kv_copy_pages",
           "ForwardGraph"]


class ForwardGraph:
    """moe_forward captured as a CUDA graph on fixed buffers
    (moe_forward_graph_create): launch() replays the layer with one launch;
    the contents of x / logits may change between replays, the buffers may
    not.  Creating it runs the forward once."""

    def __init__(self, layer_c, x: torch.Tensor, logits: torch.Tensor, out: torch.Tensor, ws: torch.Tensor,
                 stream=None):
        import ctypes
        self._h = None
        T = _forward_args(layer_c, x, logits, out, ws)
        self._keep = (layer_c, x, logits, out, ws)
        h = ctypes.c_void_p()
        check(load().moe_forward_graph_create(ctypes.byref(layer_c), _ptr(x), _ptr(logits), T, _ptr(out),
                                              _ptr(ws), ws.numel(), _stream(stream), ctypes.byref(h)),
              "moe_forward_graph_create")
        self._h = h

    def launch(self, stream=None) -> None:
        check(load().moe_graph_launch(self._h, _stream(stream)), "moe_graph_launch")

    def close(self) -> None:
        if getattr(self, "_h", None) is not None and self._h.value:
            load().moe_graph_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
