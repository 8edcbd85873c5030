"""Torch-facing wrappers of the operators that serve the layer in 8 and 4
bits: block norms with E4M3 output, the sort of such tokens by expert, weights
rounded to E2M1 and the routed experts of a few tokens on them.  As in
block_ops, they check their tensors, allocate with torch and pass pointers and
the current stream; a plan's buffers serve one call at a time."""
import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import PREC, call, moe_weights_mxfp4
from .block_ops import Block, BlockNormPlan, _check, _device, _launch, _need
from .ops import Dims, Weights

_U8, _I32, _F32, _BF16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16


def _given(name, t, dtype, shape, device):
    """_check of a tensor that may not be missing."""
    if t is None:
        raise ValueError("%s is missing" % name)
    return _check(name, t, dtype, shape, device)


# ---- norms whose output is in 8 bits ---------------------------------------
class BlockNormMxfp8Plan(BlockNormPlan):
    """Outputs of moe_block_norm_mxfp8 for one configuration: x_out [T][d]
    (None with output=False), a_q [T][d] and a_scale [T][d/32] uint8, a [T][d]
    bf16 (None with keep_a=False), r_post and r_pre [T] for the backward."""

    def __init__(self, block: Block, device="cuda", keep_a=True, output=True):
        if block.prec != "bf16":
            raise ValueError("the block's prec must be 'bf16', not %r" % (block.prec,))
        if block.d % 32:
            raise ValueError("d must be a multiple of 32, not %d" % block.d)
        super().__init__(block, device, pre_norm=keep_a, output=output)
        if self.r_pre is None:
            self.r_pre = torch.empty(block.T, dtype=_F32, device=self.device)
        self.a_q = torch.empty(block.T, block.d, dtype=_U8, device=self.device)
        self.a_scale = torch.empty(block.T, block.d // 32, dtype=_U8, device=self.device)

    def run(self, x, y=None, w_pre=None, w_post=None, gate=None):
        """(x_out, a_q, a_scale); x_out is x itself where there is no block
        output y.  With keep_a the bf16 a is in self.a."""
        dev = self.device
        px, py = _given("x", x, self._res, self._rows, dev), _check("y", y, self._act, self._rows, dev)
        _launch(dev, "moe_block_norm_mxfp8", self.cblock, px, py, *self._vectors(w_pre, w_post, gate),
                None if y is None or self.x_out is None else self.x_out.data_ptr(),
                None if self.a is None else self.a.data_ptr(), self.a_q.data_ptr(), self.a_scale.data_ptr(),
                None if self.r_post is None else self.r_post.data_ptr(), self.r_pre.data_ptr())
        return (x if y is None else self.x_out), self.a_q, self.a_scale


def block_norm_mxfp8(block: Block, x, y=None, w_pre=None, w_post=None, gate=None, keep_a=True):
    """moe_block_norm_mxfp8 into fresh tensors: (x_out, a_q, a_scale, plan); the
    plan keeps a, and r_pre and r_post for block_norm_backward."""
    plan = BlockNormMxfp8Plan(block, _need("x", x), keep_a, y is not None)
    return plan.run(x, y, w_pre, w_post, gate) + (plan,)


# ---- tokens in 8 bits sorted by expert -------------------------------------
class SortMxfp8Plan:
    """Outputs and workspace of moe_sort_tokens_mxfp8 for one configuration.
    x_perm, x_perm_scale and row_token may be the caller's; their entries from
    row offsets[E] on are never written."""

    def __init__(self, dims: Dims, device="cuda", x_perm=None, x_perm_scale=None, row_token=None):
        if dims.d % 32:
            raise ValueError("d must be a multiple of 32, not %d" % dims.d)
        n = ctypes.c_size_t(0)
        self.dims, self.cdims = dims, dims.c()
        call("moe_workspace_bytes", ctypes.byref(self.cdims), PREC["bf16"], 5, ctypes.byref(n))
        given = [t for t in (x_perm, x_perm_scale, row_token) if t is not None]
        self.device = dev = _device(given[0].device if given else device)
        self.counts = torch.empty(dims.E, dtype=_I32, device=dev)
        self.offsets = torch.empty(dims.E + 1, dtype=_I32, device=dev)
        self.token_row = torch.empty(dims.T, dims.k, dtype=_I32, device=dev)
        new = lambda t, shape, dtype: torch.empty(shape, dtype=dtype, device=dev) if t is None else t  # noqa: E731
        rows, scales = (dims.R, dims.d), (dims.R, dims.d // 32)
        self.row_token = new(row_token, (dims.R,), _I32)
        self.x_perm, self.x_perm_scale = new(x_perm, rows, _U8), new(x_perm_scale, scales, _U8)
        _check("row_token", self.row_token, _I32, (dims.R,), dev)
        _check("x_perm", self.x_perm, _U8, rows, dev)
        _check("x_perm_scale", self.x_perm_scale, _U8, scales, dev)
        self._ids, self._rows, self._scales = (dims.T, dims.k), (dims.T, dims.d), (dims.T, dims.d // 32)
        self.ws_bytes = n.value
        self.ws = torch.empty(max(n.value, 16), dtype=_U8, device=dev)

    def run(self, topk_idx, x, x_scale):
        """(counts, offsets, row_token, token_row, x_perm, x_perm_scale) of the
        ids topk_idx [T][k] int32 and the tokens x [T][d], x_scale [T][d/32]."""
        dev = self.device
        args = (_given("topk_idx", topk_idx, _I32, self._ids, dev), _given("x", x, _U8, self._rows, dev),
                _given("x_scale", x_scale, _U8, self._scales, dev))
        _launch(dev, "moe_sort_tokens_mxfp8", self.cdims, *args, self.counts.data_ptr(), self.offsets.data_ptr(),
                self.row_token.data_ptr(), self.token_row.data_ptr(), self.x_perm.data_ptr(),
                self.x_perm_scale.data_ptr(), self.ws.data_ptr(), self.ws_bytes)
        return self.counts, self.offsets, self.row_token, self.token_row, self.x_perm, self.x_perm_scale


def sort_tokens_mxfp8(topk_idx, x, x_scale, dims: Dims):
    """moe_sort_tokens_mxfp8 into fresh tensors: (counts, offsets, row_token,
    token_row, x_perm, x_perm_scale), the last two as expert_ffn takes them in
    'mxfp8'.  Nothing of use from row offsets[E] on; token_row is -1 for an
    absent route, which unsort_tokens takes and combine must not be given."""
    return SortMxfp8Plan(dims, _need("topk_idx", topk_idx)).run(topk_idx, x, x_scale)


# ---- weights in 4 bits -----------------------------------------------------
def quantize_mxfp4(src):
    """moe_quantize_mxfp4 of a bf16 matrix [rows][cols]: (codes [rows][cols/2],
    scale [cols/128][rows][4]), uint8."""
    dev = _need("src", src)
    if src.dim() != 2 or src.shape[1] % 128:
        raise ValueError("src must be a matrix with a multiple of 128 columns, not of shape %s" % (tuple(src.shape),))
    rows, cols = src.shape
    p = _check("src", src, _BF16, (rows, cols), dev)
    codes = torch.empty(rows, cols // 2, dtype=_U8, device=dev)
    scale = torch.empty(cols // 128, rows, 4, dtype=_U8, device=dev)
    _launch(dev, "moe_quantize_mxfp4", p, rows, cols, codes.data_ptr(), scale.data_ptr())
    return codes, scale


def dequantize_mxfp4(codes, scale):
    """moe_dequantize_mxfp4: the bf16 matrix [rows][cols] of codes
    [rows][cols/2] and scale [cols/128][rows][4]."""
    dev = _need("codes", codes)
    if codes.dim() != 2 or codes.shape[1] % 64:
        raise ValueError("codes must be a matrix with a multiple of 64 bytes a row, not of shape %s" % (
            tuple(codes.shape),))
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    args = (_check("codes", codes, _U8, (rows, cols // 2), dev),
            _given("scale", scale, _U8, (cols // 128, rows, 4), dev))
    dst = torch.empty(rows, cols, dtype=_BF16, device=dev)
    _launch(dev, "moe_dequantize_mxfp4", *args, rows, cols, dst.data_ptr())
    return dst


@dataclass
class WeightsMxfp4:
    """Routed experts in 4 bits (moe_weights_mxfp4): codes [E][rows][cols/2]
    and scales [cols/128][E*rows][4] of the stacked matrices."""
    q_gate: torch.Tensor
    q_gate_scale: torch.Tensor
    q_up: torch.Tensor
    q_up_scale: torch.Tensor
    q_down: torch.Tensor
    q_down_scale: torch.Tensor


def prepare_mxfp4(weights: Weights, dims: Dims) -> WeightsMxfp4:
    """The routed experts' bf16 weights in 4 bits (blocks along each product's
    K: d for gate and up, I for down), made once per weight update."""
    out = {}
    for name, rows, cols in (("gate", dims.I, dims.d), ("up", dims.I, dims.d), ("down", dims.d, dims.I)):
        w = getattr(weights, "w_" + name)
        dev = _need("w_" + name, w)
        _check("w_" + name, w, _BF16, (dims.E, rows, cols), dev)
        codes, out["q_%s_scale" % name] = quantize_mxfp4(w.view(dims.E * rows, cols))
        out["q_" + name] = codes.view(dims.E, rows, cols // 2)
    return WeightsMxfp4(**out)


# ---- the routed experts of a few tokens ------------------------------------
class RoutedFfnPlan:
    """Output and workspace of moe_routed_ffn_mxfp4 for one configuration: y
    [T][d] bf16."""

    def __init__(self, dims: Dims, device="cuda"):
        n = ctypes.c_size_t(0)
        self.dims, self.cdims = dims, dims.c()
        call("moe_workspace_bytes", ctypes.byref(self.cdims), PREC["mxfp8"], 6, ctypes.byref(n))
        self.device = dev = _device(device)
        T, d, E, k, I = dims.T, dims.d, dims.E, dims.k, dims.I
        self.y = torch.empty(T, d, dtype=_BF16, device=dev)
        self._x, self._scale, self._ids = (T, d), (T, d // 32), (T, k)
        self._shapes = [(f, s) for name, rows, cols in (("gate", I, d), ("up", I, d), ("down", d, I))
                        for f, s in (("q_" + name, (E, rows, cols // 2)),
                                     ("q_%s_scale" % name, (cols // 128, E * rows, 4)))]
        self.ws_bytes = n.value
        self.ws = torch.empty(max(n.value, 16), dtype=_U8, device=dev)

    def run(self, x, x_scale, topk_idx, topk_w, weights: WeightsMxfp4, y_add=None):
        """y [T][d] of the tokens x [T][d], x_scale [T][d/32], their ids and
        weights [T][k]; y_add [T][d] bf16 or None is added."""
        dev = self.device
        args = (_given("x", x, _U8, self._x, dev), _given("x_scale", x_scale, _U8, self._scale, dev),
                _given("topk_idx", topk_idx, _I32, self._ids, dev), _given("topk_w", topk_w, _F32, self._ids, dev))
        w = moe_weights_mxfp4(*[_given(name, getattr(weights, name), _U8, shape, dev) for name, shape in self._shapes])
        add = _check("y_add", y_add, _BF16, self._x, dev)
        _launch(dev, "moe_routed_ffn_mxfp4", self.cdims, *args, w, add, self.y.data_ptr(), self.ws.data_ptr(),
                self.ws_bytes)
        return self.y


def routed_ffn_mxfp4(x, x_scale, topk_idx, topk_w, weights: WeightsMxfp4, dims: Dims, y_add=None):
    """moe_routed_ffn_mxfp4 into a fresh tensor: y [T][d] bf16."""
    return RoutedFfnPlan(dims, _need("x", x)).run(x, x_scale, topk_idx, topk_w, weights, y_add)
