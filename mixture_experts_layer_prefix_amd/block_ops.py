"""Torch-facing wrappers of the operators around the layer: routed tokens
sorted by expert and back, the norms before and after a residual block, and
gradient clipping.  They check their tensors, allocate outputs and workspaces
with torch and pass pointers and the stream that is current on the tensors'
device; no arithmetic happens here.  A plan's buffers serve one call at a
time: calls that may overlap (on two streams, in two graphs replayed at once)
need plans of their own."""
import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import PREC, call, moe_block
from .ops import Dims

_ACT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _act(prec):
    if prec not in _ACT:
        raise ValueError("prec must be 'f32' or 'bf16', not %r" % (prec,))
    return _ACT[prec]


def _address(*args):
    """_tensors.address, found at the first call."""
    global _address
    _address = _lib.tensors().address
    return _address(*args)


def _check(name, t, dtype, shape, device):
    """t as a device pointer; raises unless it is a contiguous tensor of this
    type and shape on this device.  None: a null pointer."""
    if t is None:
        return None
    p = _address(t, dtype, shape, device.index)
    if p < 0:
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s, not %s of shape %s on %s%s" % (
            name, dtype, shape, device, t.dtype, tuple(t.shape), t.device,
            "" if t.is_contiguous() else " (not contiguous)"))
    return p


def _need(name, t):
    if t is None:
        raise ValueError("%s is missing" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be on a GPU, not on %s" % (name, t.device))
    return t.device


def _launch(device, name, *args):
    """Calls an entry point on the stream that is current on `device`, with
    that device current.  The stream is what torch.cuda.current_stream(device)
    gives, read without making a Stream object (1 us) for each call."""
    index = device.index
    if torch.cuda.current_device() == index:
        call(name, *args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            call(name, *args, torch._C._cuda_getCurrentRawStream(index))


def _device(device):
    d = torch.device(device)
    return torch.device(d.type, torch.cuda.current_device()) if d.type == "cuda" and d.index is None else d


# ---- routed tokens sorted by expert and back -------------------------------
class SortPlan:
    """Outputs and workspace of moe_sort_tokens for one configuration, so that
    repeated calls allocate nothing.  x_perm and row_token may be the
    caller's; their entries from row offsets[E] on are never written.
    gather=False: the schedule alone, no x_perm."""

    def __init__(self, dims: Dims, prec: str, device="cuda", x_perm=None, row_token=None, gather=True):
        act = _act(prec)
        n = ctypes.c_size_t(0)
        self.dims, self.prec = dims, prec
        self.cdims = dims.c()
        call("moe_workspace_bytes", ctypes.byref(self.cdims), PREC[prec], 5, ctypes.byref(n))
        self.device = dev = _device(x_perm.device if x_perm is not None else
                                    row_token.device if row_token is not None else device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.counts = torch.empty(dims.E, **i32)
        self.offsets = torch.empty(dims.E + 1, **i32)
        self.token_row = torch.empty(dims.T, dims.k, **i32)
        self.row_token = torch.empty(dims.R, **i32) if row_token is None else row_token
        self.x_perm = torch.empty(dims.R, dims.d, dtype=act, device=dev) if x_perm is None and gather else x_perm
        _check("row_token", self.row_token, torch.int32, (dims.R,), dev)
        _check("x_perm", self.x_perm, act, (dims.R, dims.d), dev)
        self._prec, self._act, self._ids, self._rows = PREC[prec], act, (dims.T, dims.k), (dims.T, dims.d)
        self.ws_bytes = n.value
        self.ws = torch.empty(max(n.value, 16), dtype=torch.uint8, device=dev)

    def run(self, topk_idx, x=None):
        """(counts, offsets, row_token, token_row, x_perm) of the ids topk_idx
        [T][k] int32 and the tokens x [T][d]."""
        dev = self.device
        if self.x_perm is not None:
            _need("x", x)
        _need("topk_idx", topk_idx)
        idx = _check("topk_idx", topk_idx, torch.int32, self._ids, dev)
        xp = _check("x", x, self._act, self._rows, dev)
        _launch(dev, "moe_sort_tokens", self.cdims, self._prec, idx, xp, self.counts.data_ptr(),
                self.offsets.data_ptr(), self.row_token.data_ptr(), self.token_row.data_ptr(),
                None if self.x_perm is None else self.x_perm.data_ptr(), self.ws.data_ptr(), self.ws_bytes)
        return self.counts, self.offsets, self.row_token, self.token_row, self.x_perm


def sort_tokens(topk_idx, x, dims: Dims, prec: str, gather=True):
    """moe_sort_tokens into fresh tensors: (counts, offsets, row_token,
    token_row, x_perm).  row_token and x_perm hold nothing of use from row
    offsets[E] on.  token_row is -1 for an absent route, which unsort_tokens
    and the gradients here take and combine and layer_backward must not be
    given."""
    return SortPlan(dims, prec, _need("topk_idx", topk_idx), gather=gather).run(topk_idx, x)


def sort_tokens_backward(dx_perm, token_row, dx_add, dims: Dims, prec: str, dx=None):
    """moe_sort_tokens_backward: dx [T][d] from dx_perm [T*k][d]; dx_add [T][d]
    or None is added.  dx: the output tensor, which may be dx_add."""
    act, dev = _act(prec), _need("dx_perm", dx_perm)
    if dx is None:
        dx = torch.empty(dims.T, dims.d, dtype=act, device=dev)
    args = (_check("dx_perm", dx_perm, act, (dims.R, dims.d), dev),
            _check("token_row", token_row, torch.int32, (dims.T, dims.k), dev),
            _check("dx_add", dx_add, act, (dims.T, dims.d), dev), _check("dx", dx, act, (dims.T, dims.d), dev))
    _launch(dev, "moe_sort_tokens_backward", dims.c(), PREC[prec], *args)
    return dx


def unsort_tokens(o_perm, token_row, topk_w, y_add, dims: Dims, prec: str, y=None):
    """moe_unsort_tokens: the weighted sum y [T][d] of o_perm's rows, y_add
    [T][d] or None added.  y: the output tensor, which may be y_add."""
    act, dev = _act(prec), _need("o_perm", o_perm)
    if y is None:
        y = torch.empty(dims.T, dims.d, dtype=act, device=dev)
    args = (_check("o_perm", o_perm, act, (dims.R, dims.d), dev),
            _check("token_row", token_row, torch.int32, (dims.T, dims.k), dev),
            _check("topk_w", topk_w, torch.float32, (dims.T, dims.k), dev),
            _check("y_add", y_add, act, (dims.T, dims.d), dev), _check("y", y, act, (dims.T, dims.d), dev))
    _launch(dev, "moe_unsort_tokens", dims.c(), PREC[prec], *args)
    return y


def unsort_tokens_backward(dy, o_perm, token_row, topk_w, dims: Dims, prec: str, do_perm=None, need_do=True,
                           need_dw=True):
    """moe_unsort_tokens_backward: (do_perm [T*k][d], dtopk_w [T][k] fp32), None
    for one that is not needed.  do_perm: the output tensor; rows of no route
    are left as they were (a fresh tensor holds nothing of use there)."""
    act, dev = _act(prec), _need("dy", dy)
    if do_perm is None and need_do:
        do_perm = torch.empty(dims.R, dims.d, dtype=act, device=dev)
    if not need_do:
        do_perm = None
    dw = torch.empty(dims.T, dims.k, dtype=torch.float32, device=dev) if need_dw else None
    args = (_check("dy", dy, act, (dims.T, dims.d), dev), _check("o_perm", o_perm, act, (dims.R, dims.d), dev),
            _check("token_row", token_row, torch.int32, (dims.T, dims.k), dev),
            _check("topk_w", topk_w, torch.float32, (dims.T, dims.k), dev),
            _check("do_perm", do_perm, act, (dims.R, dims.d), dev), None if dw is None else dw.data_ptr())
    _launch(dev, "moe_unsort_tokens_backward", dims.c(), PREC[prec], *args)
    return do_perm, dw


# ---- norms before and after a residual block -------------------------------
@dataclass(frozen=True)
class Block:
    """The step between two blocks (moe_block): T tokens of d channels, prec of
    the activations, res_f32 an fp32 residual, post_norm a norm of the block's
    output, alpha and beta the scales of residual and output, gate_every the
    tokens per gate row (0: one row for all)."""
    T: int
    d: int
    prec: str = "bf16"
    res_f32: bool = False
    post_norm: bool = False
    alpha: float = 1.0
    beta: float = 1.0
    eps: float = 1e-6
    gate_every: int = 0

    def __post_init__(self):
        _lib.check_sizes(self.T, self.d)
        _lib.check_sizes(self.gate_every)

    @property
    def every(self):
        return self.gate_every or max(self.T, 1)

    @property
    def gates(self):
        """Rows of the gate."""
        return (self.T + self.every - 1) // self.every if self.gate_every else 1

    @property
    def act(self):
        return _act(self.prec)

    @property
    def res(self):
        return torch.float32 if self.res_f32 else self.act

    def c(self):
        return moe_block(self.T, self.every, self.d, self.res_f32, self.post_norm, self.alpha, self.beta, self.eps)


class _BlockPlan:
    """What both directions' plans check their tensors against."""

    def __init__(self, block: Block, device):
        self.block, self.device, self.cblock = block, _device(device), block.c()
        self._prec, self._act, self._res = PREC[block.prec], block.act, block.res
        self._rows, self._vec, self._gates = (block.T, block.d), (block.d,), (block.gates, block.d)

    def _vectors(self, w_pre, w_post, gate):
        f32, dev = torch.float32, self.device
        return (_check("w_post", w_post, f32, self._vec, dev), _check("gate", gate, f32, self._gates, dev),
                _check("w_pre", w_pre, f32, self._vec, dev))


class BlockNormPlan(_BlockPlan):
    """Outputs of moe_block_norm for one configuration: x_out [T][d] (None
    without a block output), a [T][d] (None with pre_norm=False), r_post and
    r_pre [T] for the backward."""

    def __init__(self, block: Block, device="cuda", pre_norm=True, output=True):
        """output=False: a step without a block output (no x_out)."""
        super().__init__(block, device)
        T, d, dev = block.T, block.d, self.device
        self.x_out = torch.empty(T, d, dtype=block.res, device=dev) if output else None
        self.a = torch.empty(T, d, dtype=block.act, device=dev) if pre_norm else None
        self.r_pre = torch.empty(T, dtype=torch.float32, device=dev) if pre_norm else None
        self.r_post = torch.empty(T, dtype=torch.float32, device=dev) if block.post_norm else None

    def run(self, x, y=None, w_pre=None, w_post=None, gate=None):
        """(x_out, a); x_out is x itself where there is no block output y."""
        dev = self.device
        _need("x", x)
        px, py = _check("x", x, self._res, self._rows, dev), _check("y", y, self._act, self._rows, dev)
        _launch(dev, "moe_block_norm", self.cblock, self._prec, px, py, *self._vectors(w_pre, w_post, gate),
                None if y is None or self.x_out is None else self.x_out.data_ptr(),
                None if self.a is None else self.a.data_ptr(),
                None if self.r_post is None else self.r_post.data_ptr(),
                None if self.r_pre is None else self.r_pre.data_ptr())
        return (x if y is None else self.x_out), self.a


def block_norm(block: Block, x, y=None, w_pre=None, w_post=None, gate=None, pre_norm=True):
    """moe_block_norm into fresh tensors: (x_out, a, plan); the plan keeps
    r_pre and r_post for block_norm_backward."""
    plan = BlockNormPlan(block, _need("x", x), pre_norm, y is not None)
    return plan.run(x, y, w_pre, w_post, gate) + (plan,)


class BlockNormBackwardPlan(_BlockPlan):
    """Gradients and workspace of moe_block_norm_backward for one
    configuration: dx and dy [T][d], grads of the weights that are given (fp32
    dw_pre, dw_post [d], dgate [gates][d])."""

    def __init__(self, block: Block, device="cuda", w_pre=True, w_post=True, gate=False, output=True):
        """output=False: a step without a block output (no dy)."""
        super().__init__(block, device)
        T, d, dev = block.T, block.d, self.device
        self.dx = torch.empty(T, d, dtype=block.res, device=dev)
        self.dy = torch.empty(T, d, dtype=block.act, device=dev) if output else None
        self.grads = {}
        if w_pre:
            self.grads["dw_pre"] = torch.empty(d, dtype=torch.float32, device=dev)
        if w_post and block.post_norm:
            self.grads["dw_post"] = torch.empty(d, dtype=torch.float32, device=dev)
        if gate:
            self.grads["dgate"] = (torch.empty if T else torch.zeros)(block.gates, d, dtype=torch.float32, device=dev)
        self.ws_bytes = _lib.lib().moe_block_norm_scratch_bytes(T, d)
        self.ws = torch.empty(max(self.ws_bytes, 16), dtype=torch.uint8, device=dev)

    def run(self, dx_out, da, x_out, y, r_pre, r_post, w_pre=None, w_post=None, gate=None):
        """(dx, dy, grads) from the gradients of x_out and a (None: no
        gradient), the forward's x_out, y and row statistics (without da, r_pre
        and w_pre are None)."""
        dev, rows, tokens, f32 = self.device, self._rows, (self.block.T,), torch.float32
        _need("dx_out or da", da if dx_out is None else dx_out)
        args = (_check("dx_out", dx_out, self._res, rows, dev), _check("da", da, self._act, rows, dev),
                _check("x_out", x_out, self._res, rows, dev), _check("y", y, self._act, rows, dev),
                _check("r_post", r_post, f32, tokens, dev), _check("r_pre", r_pre, f32, tokens, dev))
        vec = self._vectors(w_pre, w_post, gate)
        g = {n: t.data_ptr() for n, t in self.grads.items()}
        _launch(dev, "moe_block_norm_backward", self.cblock, self._prec, *args, *vec, self.dx.data_ptr(),
                None if self.dy is None else self.dy.data_ptr(), g.get("dw_post"), g.get("dgate"), g.get("dw_pre"),
                self.ws.data_ptr(), self.ws_bytes)
        return self.dx, self.dy, self.grads


def block_norm_backward(block: Block, dx_out, da, x_out, y, r_pre, r_post, w_pre=None, w_post=None, gate=None):
    """moe_block_norm_backward into fresh tensors: (dx, dy, grads), grads of
    every weight that is given."""
    plan = BlockNormBackwardPlan(block, _need("dx_out or da", da if dx_out is None else dx_out), w_pre is not None,
                                 w_post is not None, gate is not None, y is not None)
    return plan.run(dx_out, da, x_out, y, r_pre, r_post, w_pre, w_post, gate)


# ---- gradient norm and clipping --------------------------------------------
def _tensors(name, tensors):
    """Host arrays (addresses, element counts, types) of a list of tensors,
    and their device."""
    got = _lib.tensors().describe(tensors)
    if isinstance(got, int):
        raise ValueError("%s[%d] must be a contiguous bf16 or fp32 tensor on the GPU of the others" % (name, got))
    if got[3] < 0:
        raise ValueError("%s holds no tensor" % name)
    return got[0], got[1], got[2], torch.device("cuda", got[3])


def _scratch(numel, n, device):
    size = _lib.lib().moe_grad_norm_scratch_bytes(numel, n)
    return torch.empty(max(size, 16), dtype=torch.uint8, device=device), size


def grad_norm(grads):
    """moe_grad_norm: the norm over all tensors, fp32 [1] on their device."""
    ptrs, numel, types, dev = _tensors("grads", grads)
    norm = torch.empty(1, dtype=torch.float32, device=dev)
    ws, size = _scratch(numel, len(grads), dev)
    _launch(dev, "moe_grad_norm", ptrs, numel, types, len(grads), norm.data_ptr(), ws.data_ptr(), size)
    return norm


def clip_grads(grads, max_norm, norm=None, out=None):
    """moe_clip_grads: scales the gradients to a global norm of at most
    max_norm, in place or into the tensors `out`; returns (out, norm).  norm
    (fp32 [1]): the norm to clip by, for instance one joined over ranks; None:
    that of these tensors.  A tensor that is written may overlap no other one
    of either list and not norm."""
    ptrs, numel, types, dev = _tensors("grads", grads)
    optrs = ptrs
    if out is not None:
        optrs, onumel, otypes, odev = _tensors("out", out)
        if onumel != numel or otypes != types or odev != dev:
            raise ValueError("out must match grads in number, size, type and device")
    given = _check("norm", norm, torch.float32, (1,), dev)
    if not _lib.tensors().distinct(optrs, numel, types, ptrs, given or 0):
        raise ValueError("%s overlap each other%s or norm" % (("grads", "") if out is None else
                                                              ("tensors of out", ", another's gradient")))
    ws, size = None, 0
    if norm is None:
        norm = torch.empty(1, dtype=torch.float32, device=dev)
        ws, size = _scratch(numel, len(grads), dev)
    _launch(dev, "moe_clip_grads", ptrs, optrs, numel, types, len(grads), max_norm, given, norm.data_ptr(),
            None if ws is None else ws.data_ptr(), size)
    return (grads if out is None else out), norm
