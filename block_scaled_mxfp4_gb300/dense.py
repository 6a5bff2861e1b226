"""A transformer's dense layer from the residual stream back to it, and its gradients.

    out = x + W2 act(W1 norm(x) + b1) + b2

``dense_block`` and ``dense_block_backward`` take tensors, allocate with torch on
the given stream and call the C entry points; every step of the computation is
one of the library's kernels.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import block_scaled_mxfp4_gb300 as mx

# The types that the codes and scales of a form stand for.
_CODES = {mx.MXFP8_E4M3: "torch.float8_e4m3fn", mx.MXFP8_E5M2: "torch.float8_e5m2"}
_PACKED, _SCALES = "torch.float4_e2m1fn_x2", "torch.float8_e8m0fnu"
_MAX_NORM = 32768                                        # the layer norm's longest row
_PARAMS = {"torch.bfloat16": mx.MXFP4_PARAM_BF16, "torch.float32": mx.MXFP4_PARAM_FP32}


class Mxfp8Forms(NamedTuple):
    """A matrix [rows, cols] as MXFP8 codes and scales along its rows (q, s), the
    same of its transpose (qt, st), and its columns' sums; None what was not asked for."""
    q: Optional["torch.Tensor"]
    s: Optional["torch.Tensor"]
    qt: Optional["torch.Tensor"]
    st: Optional["torch.Tensor"]
    sums: Optional["torch.Tensor"]


class DenseKept(NamedTuple):
    """What ``dense_block`` keeps for ``dense_block_backward``: its input and the
    norm's weight (the caller's tensors, unchanged until then), the rows' statistics,
    the normed rows along the tokens and z, both MXFP8."""
    x: "torch.Tensor"
    norm_w: Optional["torch.Tensor"]
    mean: "torch.Tensor"
    rstd: "torch.Tensor"
    yt: "torch.Tensor"
    syt: "torch.Tensor"
    z: "torch.Tensor"
    sz: "torch.Tensor"
    act: int
    fmt: int


class DenseGrads(NamedTuple):
    """dx bf16 [T, K], dw1 bf16 [F, K], dw2 bf16 [K, F]; fp32 sums db1 [F], db2,
    dnorm_w and dnorm_b [K]."""
    dx: "torch.Tensor"
    dw1: "torch.Tensor"
    dw2: "torch.Tensor"
    db1: "torch.Tensor"
    db2: "torch.Tensor"
    dnorm_w: "torch.Tensor"
    dnorm_b: "torch.Tensor"


def _up32(n):
    return -(-n // 32) * 32


def _ld(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]    # (a lone row's stride can be anything)


def _check_rows(where, name, t, shape, aligned=False):
    import torch
    if t.dtype != torch.bfloat16:
        mx._refuse(f"{where}: {name} of type torch.bfloat16", TypeError)
    if t.dim() != 2 or shape is not None and tuple(t.shape) != tuple(shape):
        mx._refuse(f"{where}: {name} of shape {'[rows, cols]' if shape is None else tuple(shape)}")
    if t.numel() and (t.stride(1) != 1 and t.shape[1] != 1 or _ld(t) < t.shape[1]):
        mx._refuse(f"{where}: {name} with neighbouring elements side by side, its rows one after the other")
    if aligned and t.numel() and (t.data_ptr() % 16 or _ld(t) % 8):
        mx._refuse(f"{where}: {name} of 16-byte aligned rows")


def _check_bytes(where, name, t, shape, means):
    """`means`: the type of 8 or 4 bits whose codes these are; other such types are refused, bytes are not."""
    if t.element_size() != 1 or t.dtype.is_floating_point and str(t.dtype) != means:
        mx._refuse(f"{where}: {name} of bytes or type {means}", TypeError)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        mx._refuse(f"{where}: {name} contiguous, of shape {tuple(shape)}")


def _check_params(where, pairs):
    """[(name, tensor or None, length)] of one type; its MXFP4_PARAM_* code."""
    kinds = set()
    for name, t, n in pairs:
        if t is None:
            continue
        if str(t.dtype) not in _PARAMS:
            mx._refuse(f"{where}: {name} of type torch.bfloat16 or torch.float32", TypeError)
        if tuple(t.shape) != (n,) or not t.is_contiguous():
            mx._refuse(f"{where}: {name} contiguous, of shape ({n},)")
        kinds.add(str(t.dtype))
    if len(kinds) > 1:
        mx._refuse(f"{where}: {' and '.join(p[0] for p in pairs)} of one type", TypeError)
    return _PARAMS[kinds.pop()] if kinds else mx.MXFP4_PARAM_BF16


def _check_codes(where, act, *fmts):
    if act not in range(mx.MXFP4_ACT_SILU + 1):
        mx._refuse(f"{where}: act one of MXFP4_ACT_*")
    if any(f not in (mx.MXFP8_E4M3, mx.MXFP8_E5M2) for f in fmts):
        mx._refuse(f"{where}: formats MXFP8_E4M3 or MXFP8_E5M2")


def _check_place(where, stream, x, *others):
    """One GPU, and the one that the kernels are launched on: that of a stream other than the current one
    (as _on_stream takes it), or else the current one."""
    import torch
    if not x.is_cuda or any(t is not None and t.device != x.device for t in others):
        mx._refuse(f"{where}: everything on one GPU")
    device = torch.cuda.current_device()
    if isinstance(stream, torch.cuda.Stream) and stream.cuda_stream != torch.cuda.current_stream().cuda_stream:
        device = stream.device.index
    if x.device.index != device:
        mx._refuse(f"{where}: tensors on the device of the current stream, or of the one given,")


def mxfp8_forms(x, fmt=mx.MXFP8_E4M3, rows=True, columns=True, sums=False, stream=None) -> Mxfp8Forms:
    """bf16 [rows, cols] of 16-byte aligned rows -> its Mxfp8Forms, from one reading
    (mxfp8_checkpoint).  q uint8 [rows, cols up to 32], s uint8 [rows, cols / 32 up],
    qt and st the same of the transpose, sums fp32 [cols]."""
    import torch
    where = "mxfp8_forms"
    _check_rows(where, "x", x, None, aligned=True)
    _check_codes(where, 0, fmt)
    M, N = x.shape
    if M < 1 or N < 1:
        mx._refuse(f"{where}: x of at least one element")
    if not (rows or columns or sums):
        mx._refuse(f"{where}: at least one form")
    _check_place(where, stream, x)
    made = []
    with mx._on_stream(stream, [x], made):
        u8 = lambda want, *shape: torch.empty(shape, dtype=torch.uint8, device=x.device) if want else None
        out = Mxfp8Forms(u8(rows, M, _up32(N)), u8(rows, M, _up32(N) // 32), u8(columns, N, _up32(M)),
                         u8(columns, N, _up32(M) // 32),
                         torch.empty(N, dtype=torch.float32, device=x.device) if sums else None)
        made += [t for t in out if t is not None]
        need = mx.mxfp8_checkpoint_workspace_size(M, N) if sums else 0
        ws = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
        mx.mxfp8_checkpoint(out.q, _up32(N), out.s, _up32(N) // 32, out.qt, _up32(M), out.st, _up32(M) // 32,
                            out.sums, x, _ld(x), M, N, fmt, ws, need)
    return out


def dense_block(x, w1, s1, w2, s2, b1=None, b2=None, norm_w=None, norm_b=None, act=mx.MXFP4_ACT_GELU,
                fmt=mx.MXFP8_E4M3, eps=1e-5, keep=False, stream=None):
    """A dense layer with its norm and residual, on MXFP4 or MXFP8 weights.

    x bf16 [T, K].  MXFP4: w1 uint8 [F, K / 2], w2 uint8 [K, F / 2] as
    mxfp4_quantize writes them; MXFP8 (codes of `fmt`): w1 [F, K], w2 [K, F] as in
    mxfp8_forms; s1 [F, K / 32], s2 [K, F / 32] either way, K and F multiples of 32,
    K up to 32768.
    Codes and scales are bytes, or of torch's own types for them (float8_e4m3fn for
    MXFP8_E4M3 and so on; another format's are refused).
    What the products read is quantised in the weights' form: the normed rows, which the
    norm rounds to bf16 first, and h, from fp32.  b1 [F] and b2 [K],
    norm_w and norm_b [K]: bf16 or fp32, each pair of one type, None for none.

    Returns out bf16 [T, K], or with keep=True (MXFP8 weights) (out, DenseKept).
    On another `stream` than the current one the block's own memory belongs to that
    stream; the caller orders the two.  Rows of x may be apart; other types or layouts
    raise TypeError or ValueError.
    """
    import torch
    where = "dense_block"
    _check_rows(where, "x", x, None)
    T, K = x.shape
    if w1.dim() != 2 or w2.dim() != 2:
        mx._refuse(f"{where}: w1 and w2 of two dimensions")
    F, packed = w1.shape[0], w1.shape[1] * 2 == K
    if K % 32 or F % 32 or not K or not F:
        mx._refuse(f"{where}: K and F multiples of 32")
    if K > _MAX_NORM:
        mx._refuse(f"{where}: K of at most {_MAX_NORM}")
    if not eps >= 0:
        mx._refuse(f"{where}: eps of at least 0")
    _check_codes(where, act, fmt)
    per, codes = (2, _PACKED) if packed else (1, _CODES[fmt])
    for name, t, shape, means in (("w1", w1, (F, K // per), codes), ("w2", w2, (K, F // per), codes),
                                  ("s1", s1, (F, K // 32), _SCALES), ("s2", s2, (K, F // 32), _SCALES)):
        _check_bytes(where, name, t, shape, means)
    bias1, bias2 = _check_params(where, [("b1", b1, F)]), _check_params(where, [("b2", b2, K)])
    norm = _check_params(where, [("norm_w", norm_w, K), ("norm_b", norm_b, K)])
    if keep and packed:
        mx._refuse(f"{where}: MXFP8 weights with keep=True")
    inputs = [x, w1, s1, w2, s2, b1, b2, norm_w, norm_b]
    _check_place(where, stream, *inputs)
    made = []
    with mx._on_stream(stream, inputs, made):
        u8 = lambda *shape: torch.empty(shape, dtype=torch.uint8, device=x.device)
        f32 = lambda *shape: torch.empty(shape, dtype=torch.float32, device=x.device)
        out = torch.empty((T, K), dtype=torch.bfloat16, device=x.device)
        made.append(out)
        kept = None
        if keep:
            kept = DenseKept(x, norm_w, f32(T), f32(T), u8(K, _up32(T)), u8(K, _up32(T) // 32), u8(T, F),
                             u8(T, F // 32), act, fmt)
            made += kept[2:8]
        if T:
            size = mx.mxfp4_gemm_workspace_size if packed else mx.mxfp8_gemm_workspace_size
            need = max(size(T, F, K, 0), size(T, K, F, 0))
            ws = u8(max(need, 256))
            y, q, sq = torch.empty_like(out), u8(T, K // per), u8(T, K // 32)
            h, sh = u8(T, F // per), u8(T, F // 32)
            mx.mxfp4_layer_norm(y, K, kept and kept.mean, kept and kept.rstd, x, _ld(x), norm_w, norm_b, norm,
                                float(eps), T, K)
            back = (b2, bias2, mx.MXFP4_ACT_NONE, x, _ld(x), 1.0, T, K, F, 0, 0, ws, need)
            if packed:
                mx.mxfp4_quantize(q, K, sq, K // 32, y, K, T, K)
                mx.mxfp4_gemm_act(None, 0, h, F, sh, F // 32, None, 0, None, 0, q, K, w1, K, sq, K // 32, s1,
                                  K // 32, 0, 1.0, b1, bias1, act, None, 0, 0.0, T, F, K, 0, 0, ws, need)
                mx.mxfp4_gemm_act(out, K, None, 0, None, 0, None, 0, None, 0, h, F, w2, F, sh, F // 32, s2,
                                  F // 32, 0, 1.0, *back)
            else:
                z, sz, yt, syt = (kept.z, kept.sz, kept.yt, kept.syt) if keep else (None,) * 4
                mx.mxfp8_checkpoint(q, K, sq, K // 32, yt, _up32(T), syt, _up32(T) // 32, None, y, K, T, K, fmt,
                                    None, 0)
                mx.mxfp8_gemm_act(None, 0, h, F, sh, F // 32, z, F, sz, F // 32, q, K, w1, K, sq, K // 32, s1,
                                  K // 32, fmt, fmt, fmt, fmt, 1.0, b1, bias1, act, None, 0, 0.0, T, F, K, 0, 0,
                                  ws, need)
                mx.mxfp8_gemm_act(out, K, None, 0, None, 0, None, 0, None, 0, h, F, w2, F, sh, F // 32, s2,
                                  F // 32, fmt, fmt, fmt, fmt, 1.0, *back)
    return (out, kept) if keep else out


def dense_block_backward(dout, kept, w1t, s1t, w2t, s2t, fmt_grad=mx.MXFP8_E4M3, stream=None) -> DenseGrads:
    """Gradients of ``dense_block(..., keep=True)``.

    dout bf16 [T, K] of 16-byte aligned rows; w1t uint8 [K, F], s1t [K, F / 32], w2t
    [F, K], s2t [F, K / 32]: the weights' transposed forms (qt, st of mxfp8_forms), in
    the forward pass's format.  Gradients are products' operands in `fmt_grad`.  The
    gradients are those of the arithmetic that ran: from z as it was kept, with every
    rounding's slope taken as one.  dh and the gradient behind the norm pass through
    bf16; dz and h are rounded to their forms from fp32.
    """
    import torch
    where = "dense_block_backward"
    _check_rows(where, "kept.x", kept.x, None)
    T, K = kept.x.shape
    if kept.z.dim() != 2:
        mx._refuse(f"{where}: kept.z of two dimensions")
    F = kept.z.shape[1]
    if K % 32 or F % 32 or not K or not F:
        mx._refuse(f"{where}: K and F multiples of 32")
    if K > _MAX_NORM:
        mx._refuse(f"{where}: K of at most {_MAX_NORM}")
    T32 = _up32(T)
    _check_codes(where, kept.act, kept.fmt, fmt_grad)
    codes = _CODES[kept.fmt]
    for name, shape, means in (("yt", (K, T32), codes), ("syt", (K, T32 // 32), _SCALES), ("z", (T, F), codes),
                               ("sz", (T, F // 32), _SCALES)):
        _check_bytes(where, "kept." + name, getattr(kept, name), shape, means)
    for name in ("mean", "rstd"):
        t = getattr(kept, name)
        if t.dtype != torch.float32:
            mx._refuse(f"{where}: kept.{name} of type torch.float32", TypeError)
        if tuple(t.shape) != (T,) or not t.is_contiguous():
            mx._refuse(f"{where}: kept.{name} contiguous, of shape ({T},)")
    _check_rows(where, "dout", dout, (T, K), aligned=True)
    for name, t, shape, means in (("w1t", w1t, (K, F), codes), ("w2t", w2t, (F, K), codes), ("s1t", s1t, (K, F // 32), _SCALES),
                                  ("s2t", s2t, (F, K // 32), _SCALES)):
        _check_bytes(where, name, t, shape, means)
    x, norm_w, mean, rstd, yt, syt, z, sz, act, fmt = kept
    norm = _check_params(where, [("kept.norm_w", norm_w, K)])
    inputs = [dout, w1t, s1t, w2t, s2t, *kept[:8]]
    _check_place(where, stream, *inputs)
    made = []
    with mx._on_stream(stream, inputs, made):
        u8 = lambda *shape: torch.empty(shape, dtype=torch.uint8, device=x.device)
        # (no tokens: the sums are nothing)
        make = torch.empty if T else torch.zeros
        bf16 = lambda *shape: make(shape, dtype=torch.bfloat16, device=x.device)
        f32 = lambda n: make(n, dtype=torch.float32, device=x.device)
        g = DenseGrads(bf16(T, K), bf16(F, K), bf16(K, F), f32(F), f32(K), f32(K), f32(K))
        made += g
        if T:
            size = mx.mxfp8_gemm_workspace_size
            need = max(size(T, F, K, 0), size(T, K, F, 0), size(K, F, T32, 0), size(F, K, T32, 0),
                       mx.mxfp8_checkpoint_workspace_size(T, K), mx.mxfp8_checkpoint_workspace_size(T, F),
                       mx.mxfp4_layer_norm_workspace_size(T, K))
            ws = u8(max(need, 256))

            def product(D, A, sa, B, sb, fmt_a, fmt_b, M, N, depth):
                mx.mxfp8_gemm(D, N, None, 0, A, depth, B, depth, sa, depth // 32, sb, depth // 32, fmt_a, fmt_b,
                              1.0, 0.0, M, N, depth, 0, ws, need)

            # dout, dz and h in the orientations of the products that read them.
            o, so, ot, sot = u8(T, K), u8(T, K // 32), u8(K, T32), u8(K, T32 // 32)
            mx.mxfp8_checkpoint(o, K, so, K // 32, ot, T32, sot, T32 // 32, g.db2, dout, _ld(dout), T, K, fmt_grad,
                                ws, need)
            dh = torch.empty((T, F), dtype=torch.bfloat16, device=x.device)
            product(dh, o, so, w2t, s2t, fmt_grad, fmt, T, F, K)
            dz, sdz, dzt, sdzt = u8(T, F), u8(T, F // 32), u8(F, T32), u8(F, T32 // 32)
            ht, sht = u8(F, T32), u8(F, T32 // 32)
            mx.mxfp8_act_backward(None, 0, dz, F, sdz, F // 32, dzt, T32, sdzt, T32 // 32, ht, T32, sht, T32 // 32,
                                  g.db1, dh, F, z, F, sz, F // 32, fmt, act, T, F, fmt_grad, fmt, ws, need)
            product(g.dw2, ot, sot, ht, sht, fmt_grad, fmt, K, F, T32)
            product(g.dw1, dzt, sdzt, yt, syt, fmt_grad, fmt, F, K, T32)
            product(g.dx, dz, sdz, w1t, s1t, fmt_grad, fmt, T, K, F)
            mx.mxfp4_layer_norm_backward(g.dx, K, g.dnorm_w, g.dnorm_b, g.dx, K, x, _ld(x), mean, rstd, norm_w,
                                         norm, dout, _ld(dout), T, K, ws, need)
    return g
