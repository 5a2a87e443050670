"""The decoding operators of libfg.so (include/fg.h) on torch tensors: residual
RMS norm with 8-bit output, router choice, products with 4-bit weights, and the
expert layer for few tokens.

Every function checks its tensors' types, shapes, strides and device, launches on
the current stream (or on `stream`) without synchronising, and raises
fg.FgError (code fg.EINVAL) for arguments it does not take. Outputs are allocated
unless given. All of them may be captured into a graph; nothing is kept between
calls. The formulas and limits stand at the entry points in include/fg.h.

There is no backward pass: tensors that require gradients are refused unless
gradients are off (torch.no_grad()). Given buffers count as written in place.

With `stream`, the caller orders that stream after whatever makes the inputs (and
last used given outputs), and the use of the outputs after that stream. What a call
allocates comes from that stream's memory, so it needs no further order; tensors of
either stream may be dropped right after the call.

The work of a call is done by the extension fg_torch (csrc/fg_torch.cpp)."""
from __future__ import annotations

import ctypes as C
import importlib.machinery
import importlib.util
import os
from typing import NamedTuple, Optional, Union

import torch

from . import fg

BF16, I8, E4M3, F32 = 0, 1, 2, 3
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
NORM_MAX_N = 65536
W4_MAX_ROWS = 1048576
FEW_MAX_SIZE, FEW_MAX_ROW_BYTES = 16777216, 67108864
MOE_FEW_TOKENS, MOE_FEW_TOPK, MOE_FEW_EXPERTS = 64, 16, 1024


class NormResult(NamedTuple):
    sum: Optional[torch.Tensor]      # bf16 [rows, n]: x + residual (None without a residual and without a buffer)
    y: Optional[torch.Tensor]        # bf16 [rows, n]
    q: Optional[torch.Tensor]        # int8 or float8_e4m3fn [rows, n]
    scale: Optional[torch.Tensor]    # fp32 [rows, 1 or n / 128]


class W4Weight(NamedTuple):
    """4-bit weights [.., n, k]: `q` uint8 [.., n, k // 2], the low nibble first;
    `scale` bf16 [.., n, k // group]; `zero` uint8 like scale, or None (8). With int8
    activations a zero point above 128 makes its row's results NaN."""
    q: torch.Tensor
    scale: torch.Tensor
    zero: Optional[torch.Tensor] = None


EXTENSION = os.path.join(os.path.dirname(fg.LIB_PATH), "fg_torch.so")
_native = None


def load_extension():
    """Load fg_torch.so; raises if it has not been built (no fallback exists)."""
    global _native
    if _native is None:
        fg.load_library()
        if not os.path.exists(EXTENSION):
            raise FileNotFoundError(f"{EXTENSION} is missing: build it with `python -m sync_protocols_amd.build`")
        loader = importlib.machinery.ExtensionFileLoader("fg_torch", EXTENSION)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("fg_torch", loader))
        loader.exec_module(module)
        module.setup(fg.FgError)
        _native = module
    return _native


def add_rmsnorm(x: torch.Tensor, gamma: torch.Tensor, *, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
                out: str = "bf16", group: int = 0, keep_bf16: bool = False, sum: Optional[torch.Tensor] = None,
                y: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                stream=None) -> NormResult:
    """h = x (+ residual), y = h / rms(h) * gamma, as bf16 (`out` "bf16"), or as
    "i8" / "e4m3" codes with fp32 scales per row (`group` 0) or per 128 columns
    (128); keep_bf16 gives the bf16 y beside the codes. sum, y, q and scale are
    optional output buffers; sum and y may be x or residual."""
    return NormResult(*(_native or load_extension()).add_rmsnorm(x, gamma, residual, eps, out, group, keep_bf16, sum, y, q, scale,
                                                                 stream))


def moe_route(logits: torch.Tensor, k: int, *, score: str = "softmax", renorm: bool = True, scale: float = 1.0,
              topk: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None, stream=None):
    """(topk int32 [rows, k], weights fp32 [rows, k]) of fp32 or bf16 logits
    [rows, experts]: the k largest, largest first, ties by lowest index, with
    softmax or sigmoid scores, divided by their sum if renorm, times scale."""
    return (_native or load_extension()).moe_route(logits, k, score, renorm, scale, topk, weights, stream)


def w4_linear(x: torch.Tensor, w: W4Weight, *, x_scale: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x [rows, k] (bf16, or int8 / float8_e4m3fn with x_scale) times 4-bit weights
    w [n, k], plus a bf16 bias [n]: bf16 [rows, n]."""
    return (_native or load_extension()).w4_linear(x, x_scale, w.q, w.scale, w.zero, bias, out, stream)


def moe_few_bytes(tokens: int, k: int, width: int) -> int:
    """Workspace bytes of moe_few."""
    v = C.c_int64(0)
    code = fg.load_library().fg_moe_few_bytes(tokens, k, width, C.byref(v))
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
    a = w1 if isinstance(w1, W4Weight) else (w1, None, None)
    b = w2 if isinstance(w2, W4Weight) else (w2, None, None)
    return (_native or load_extension()).moe_few(x, x_scale, *a, *b, topk, weights, expert_base, out, workspace, stream)
