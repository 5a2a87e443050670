"""The decoding operators of libfg.so (include/fg.h) on torch tensors: residual
RMS norm with 8-bit output, router choice, products with 4-bit weights, and the
expert layer for few tokens.

Every function checks its tensors' types, shapes, strides and device, launches on
the current stream (or on `stream`) without synchronising, and raises
fg.FgError (code fg.EINVAL) for arguments it does not take. Outputs are allocated
unless given. All of them may be captured into a graph; nothing is kept between
calls. The formulas and limits stand at the entry points in include/fg.h."""
from __future__ import annotations

import ctypes as C
from typing import NamedTuple, Optional, Union

import torch

from . import fg

BF16, I8, E4M3, F32 = 0, 1, 2, 3
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
NORM_MAX_N = 65536
W4_MAX_ROWS = 1048576
MOE_FEW_TOKENS, MOE_FEW_TOPK, MOE_FEW_EXPERTS = 64, 16, 1024

_bf16, _f32, _i32, _u8, _i8, _e4m3 = (torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.int8,
                                      torch.float8_e4m3fn)
_ROWS = {_bf16: BF16, _i8: I8, _e4m3: E4M3}
_OUT8 = {"i8": (I8, _i8), "e4m3": (E4M3, _e4m3)}
_SCORES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}


class NormResult(NamedTuple):
    sum: Optional[torch.Tensor]      # bf16 [rows, n]: x + residual (None without a residual and without a buffer)
    y: Optional[torch.Tensor]        # bf16 [rows, n]
    q: Optional[torch.Tensor]        # int8 or float8_e4m3fn [rows, n]
    scale: Optional[torch.Tensor]    # fp32 [rows, 1 or n / 128]


class W4Weight(NamedTuple):
    """4-bit weights [.., n, k]: `q` uint8 [.., n, k // 2], the low nibble first;
    `scale` bf16 [.., n, k // group]; `zero` uint8 like scale, or None (8)."""
    q: torch.Tensor
    scale: torch.Tensor
    zero: Optional[torch.Tensor] = None


def _refuse(what: str) -> None:
    raise fg.FgError(fg.EINVAL, what)


def _rows2d(t: torch.Tensor, what: str) -> None:
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        _refuse(f"{what} must be [rows, columns] with consecutive columns and rows that do not overlap")


def _ld(t: torch.Tensor) -> int:
    """Row distance in elements; that of a single row does not matter."""
    return t.stride(0) if t.shape[0] > 1 else -(-t.shape[1] // 8) * 8


def _same_device(dev: torch.device, *ts) -> None:
    if dev.type != "cuda":
        _refuse("tensors must be on the GPU")
    for t in ts:
        if t is not None and t.device != dev:
            _refuse("tensors are on different devices")


def _out(t, shape, dtype, dev, what):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != dev:
        _refuse(f"{what} must be {dtype} {tuple(shape)} on {dev}")
    return t


def _p(t):
    return None if t is None else t.data_ptr()


_lib = None


def _library():
    global _lib
    if _lib is None:
        _lib = fg.load_library()
    return _lib


def _run(name: str, dev: torch.device, stream, tensors, args) -> None:
    """Launch on dev's current stream, or on `stream`: then the allocator is told
    that the tensors are used there."""
    fn = getattr(_library(), name)
    if stream is None:
        handle = torch.cuda.current_stream(dev).cuda_stream
    else:
        if stream.device != dev:
            _refuse("stream and tensors are on different devices")
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        handle = stream.cuda_stream
    if torch.cuda.current_device() == dev.index:
        code = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            code = fn(*args, handle)
    if code != fg.OK:
        raise fg.FgError(code, name)


def _activations(x, x_scale, k, what):
    """(type, scale group) of product activations [rows, k]."""
    _rows2d(x, what)
    kind = _ROWS.get(x.dtype)
    if kind is None or x.shape[1] != k:
        _refuse(f"{what} must be bf16, int8 or float8_e4m3fn with {k} columns")
    if kind == BF16:
        if x_scale is not None:
            _refuse("bf16 activations take no x_scale")
        return kind, 0
    if x_scale is None or x_scale.dtype != _f32 or not x_scale.is_contiguous():
        _refuse("8-bit activations need a contiguous float32 x_scale")
    rows = x.shape[0]
    if tuple(x_scale.shape) in ((rows,), (rows, 1)):
        return kind, 0
    if k % 128 == 0 and tuple(x_scale.shape) == (rows, k // 128):
        return kind, 128
    _refuse(f"x_scale must be [{rows}], [{rows}, 1] or [{rows}, {k}/128]")


def _w4(w: W4Weight, lead, n, k, what) -> int:
    """Group size of 4-bit weights of the given shape."""
    if w.q.dtype != _u8 or tuple(w.q.shape) != (*lead, n, k // 2) or k % 2 or not w.q.is_contiguous():
        _refuse(f"{what}.q must be contiguous uint8 {(*lead, n, k // 2)}")
    groups = w.scale.shape[-1] if w.scale.dim() else 0
    if w.scale.dtype != _bf16 or groups < 1 or k % groups or tuple(w.scale.shape) != (*lead, n, groups) or not w.scale.is_contiguous():
        _refuse(f"{what}.scale must be contiguous bf16 {(*lead, n)} + (k // group,)")
    if w.zero is not None and (w.zero.dtype != _u8 or w.zero.shape != w.scale.shape or not w.zero.is_contiguous()):
        _refuse(f"{what}.zero must be contiguous uint8 like scale")
    return k // groups


def add_rmsnorm(x: torch.Tensor, gamma: torch.Tensor, *, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
                out: str = "bf16", group: int = 0, keep_bf16: bool = False, sum: Optional[torch.Tensor] = None,
                y: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                stream=None) -> NormResult:
    """h = x (+ residual), y = h / rms(h) * gamma, as bf16 (`out` "bf16"), or as
    "i8" / "e4m3" codes with fp32 scales per row (`group` 0) or per 128 columns
    (128); keep_bf16 gives the bf16 y beside the codes. sum, y, q and scale are
    optional output buffers; sum and y may be x or residual."""
    _rows2d(x, "x")
    rows, n = x.shape
    if x.dtype != _bf16 or gamma.dtype != _bf16 or tuple(gamma.shape) != (n,) or (n > 1 and gamma.stride(0) != 1):
        _refuse("x must be bf16 [rows, n] and gamma bf16 [n]")
    if residual is not None:
        _rows2d(residual, "residual")
        if residual.dtype != _bf16 or residual.shape != x.shape:
            _refuse("residual must be bf16 like x")
    if out != "bf16" and out not in _OUT8:
        _refuse("out must be 'bf16', 'i8' or 'e4m3'")
    if group not in (0, 128) or (group and (n % 128 or out == "bf16")):
        _refuse("group must be 0, or 128 for 8-bit outputs of a multiple of 128 columns")
    dev = x.device
    if residual is not None or sum is not None:
        sum = _out(sum, x.shape, _bf16, dev, "sum")
        _rows2d(sum, "sum")
    if out == "bf16" or keep_bf16 or y is not None:
        y = _out(y, x.shape, _bf16, dev, "y")
        _rows2d(y, "y")
    kind = 0
    if out != "bf16":
        kind, dtype = _OUT8[out]
        q = _out(q, x.shape, dtype, dev, "q")
        _rows2d(q, "q")
        scale = _out(scale, (rows, n // group if group else 1), _f32, dev, "scale")
        if not scale.is_contiguous():
            _refuse("scale must be contiguous")
    elif q is not None or scale is not None:
        _refuse("q and scale need an 8-bit out")
    _same_device(dev, residual, gamma, sum, y, q, scale)
    _run("fg_add_rmsnorm", dev, stream, (x, residual, gamma, sum, y, q, scale),
         (x.data_ptr(), _ld(x), _p(residual), _ld(residual) if residual is not None else 0, gamma.data_ptr(), eps,
          _p(sum), _ld(sum) if sum is not None else 0, _p(y), _ld(y) if y is not None else 0,
          _p(q), _ld(q) if q is not None else 0, kind, group, _p(scale), rows, n))
    return NormResult(sum, y, q, scale)


def moe_route(logits: torch.Tensor, k: int, *, score: str = "softmax", renorm: bool = True, scale: float = 1.0,
              topk: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None, stream=None):
    """(topk int32 [rows, k], weights fp32 [rows, k]) of fp32 or bf16 logits
    [rows, experts]: the k largest, largest first, ties by lowest index, with
    softmax or sigmoid scores, divided by their sum if renorm, times scale."""
    _rows2d(logits, "logits")
    if logits.dtype not in (_f32, _bf16) or score not in _SCORES:
        _refuse("logits must be float32 or bf16, score 'softmax' or 'sigmoid'")
    rows, experts = logits.shape
    dev = logits.device
    if not 1 <= k <= min(experts, 64):
        _refuse("k must be in 1..min(experts, 64)")
    topk = _out(topk, (rows, k), _i32, dev, "topk")
    weights = _out(weights, (rows, k), _f32, dev, "weights")
    if not topk.is_contiguous() or not weights.is_contiguous():
        _refuse("topk and weights must be contiguous")
    _same_device(dev)
    _run("fg_moe_route", dev, stream, (logits, topk, weights),
         (logits.data_ptr(), _ld(logits), F32 if logits.dtype == _f32 else BF16, rows, experts, k, _SCORES[score],
          1 if renorm else 0, scale, topk.data_ptr(), weights.data_ptr()))
    return topk, weights


def w4_linear(x: torch.Tensor, w: W4Weight, *, x_scale: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x [rows, k] (bf16, or int8 / float8_e4m3fn with x_scale) times 4-bit weights
    w [n, k], plus a bf16 bias [n]: bf16 [rows, n]."""
    if w.q.dim() != 2:
        _refuse("w.q must be [n, k // 2]")
    n, k = w.q.shape[0], 2 * w.q.shape[1]
    kind, x_group = _activations(x, x_scale, k, "x")
    group = _w4(w, (), n, k, "w")
    if bias is not None and (bias.dtype != _bf16 or tuple(bias.shape) != (n,) or (n > 1 and bias.stride(0) != 1)):
        _refuse("bias must be bf16 [n]")
    dev, rows = x.device, x.shape[0]
    out = _out(out, (rows, n), _bf16, dev, "out")
    _rows2d(out, "out")
    _same_device(dev, x_scale, w.q, w.scale, w.zero, bias)
    _run("fg_w4_linear", dev, stream, (x, x_scale, w.q, w.scale, w.zero, bias, out),
         (x.data_ptr(), _ld(x), kind, _p(x_scale), x_group, w.q.data_ptr(), w.scale.data_ptr(), _p(w.zero), group, _p(bias),
          out.data_ptr(), _ld(out), rows, n, k))
    return out


def moe_few_bytes(tokens: int, k: int, width: int) -> int:
    """Workspace bytes of moe_few."""
    v = C.c_int64(0)
    code = _library().fg_moe_few_bytes(tokens, k, width, C.byref(v))
    if code != fg.OK:
        raise fg.FgError(code, "fg_moe_few_bytes")
    return v.value


def moe_few(x: torch.Tensor, w1: Union[torch.Tensor, W4Weight], w2: Union[torch.Tensor, W4Weight], topk: torch.Tensor,
            weights: torch.Tensor, *, expert_base: int = 0, x_scale: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The expert layer of up to 64 tokens x [tokens, K] on this GPU's experts
    expert_base..: w1 [n_local, 2F, K] (gate rows, then up rows) and w2
    [n_local, K, F], both bf16 or both W4Weight; topk int32 [tokens, k] and weights
    fp32 [tokens, k] as moe_route gives them. bf16 [tokens, K]."""
    quant = isinstance(w1, W4Weight)
    if quant != isinstance(w2, W4Weight):
        _refuse("w1 and w2 must be of the same kind")
    a, b = (w1.q, w2.q) if quant else (w1, w2)
    if a.dim() != 3 or b.dim() != 3 or x.dim() != 2:
        _refuse("w1 and w2 must be [experts, rows, columns]")
    tokens, K = x.shape
    n_local, F = a.shape[0], a.shape[1] // 2
    if quant:
        group = _w4(w1, (n_local,), 2 * F, K, "w1")
        if _w4(w2, (n_local,), K, F, "w2") != group:
            _refuse("w1 and w2 must have the same group size")
    else:
        group = 0
        if w1.dtype != _bf16 or w2.dtype != _bf16 or tuple(w1.shape) != (n_local, 2 * F, K) or tuple(w2.shape) != (n_local, K, F):
            _refuse(f"w1 must be bf16 [n_local, 2F, {K}] and w2 bf16 [n_local, {K}, F]")
        if not w1.is_contiguous() or not w2.is_contiguous():
            _refuse("w1 and w2 must be contiguous")
    kind, x_group = _activations(x, x_scale, K, "x")
    if topk.dtype != _i32 or weights.dtype != _f32 or topk.dim() != 2 or topk.shape[0] != tokens or weights.shape != topk.shape:
        _refuse("topk must be int32 [tokens, k] and weights float32 like it")
    if not topk.is_contiguous() or not weights.is_contiguous():
        _refuse("topk and weights must be contiguous")
    k = topk.shape[1]
    if tokens > MOE_FEW_TOKENS or not 1 <= k <= MOE_FEW_TOPK:
        _refuse(f"moe_few takes up to {MOE_FEW_TOKENS} tokens with 1..{MOE_FEW_TOPK} picks each")
    dev = x.device
    out = _out(out, (tokens, K), _bf16, dev, "out")
    _rows2d(out, "out")
    need = 4 * tokens * k * F
    if workspace is None:
        workspace = torch.empty(need, dtype=_u8, device=dev)
    elif not workspace.is_contiguous():
        _refuse("workspace must be contiguous")
    _same_device(dev, x_scale, a, b, topk, weights, workspace, *(() if not quant else (w1.scale, w1.zero, w2.scale, w2.zero)))
    s1, z1, s2, z2 = (w1.scale, w1.zero, w2.scale, w2.zero) if quant else (None, None, None, None)
    _run("fg_moe_few", dev, stream, (x, x_scale, a, s1, z1, b, s2, z2, topk, weights, workspace, out),
         (x.data_ptr(), _ld(x), kind, _p(x_scale), x_group, a.data_ptr(), _p(s1), _p(z1), b.data_ptr(), _p(s2), _p(z2), group,
          topk.data_ptr(), weights.data_ptr(), tokens, k, expert_base, n_local, K, F, workspace.data_ptr(),
          workspace.numel() * workspace.element_size(), out.data_ptr(), _ld(out)))
    return out
