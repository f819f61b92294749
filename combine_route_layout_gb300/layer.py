"""What a mixture-of-experts layer has around dispatch and combine, on torch
tensors: the router with its balance loss (EpRouterOp) and the experts'
products (EpLinearOp). Argument checks and marshalling only; the work is the
CUDA kernels behind ep_router_* and ep_linear_* of include/ep.h, on torch's
current stream. An operator owns its workspace; calls on one operator are
ordered by the caller (same stream, or events).
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import ep
from .ep import EP_ERR_INVALID_ARG, EpError, _ptr

_SCORE_OF = {"softmax": ep.EP_SCORE_SOFTMAX, "sigmoid": ep.EP_SCORE_SIGMOID}
_ACT_OF = {"none": ep.EP_ACT_NONE, "relu": ep.EP_ACT_RELU, "silu": ep.EP_ACT_SILU,
           "gelu": ep.EP_ACT_GELU, "swiglu": ep.EP_ACT_SWIGLU}
_FLOAT_OF = {torch.float32: ep.EP_DTYPE_FP32, torch.bfloat16: ep.EP_DTYPE_BF16}


def _refuse(msg: str):
    raise EpError(EP_ERR_INVALID_ARG, msg)


def _code(table: dict, value, what: str) -> int:
    if value not in table:
        _refuse(f"{what} {value!r} is not one of {sorted(map(str, table))}")
    return table[value]


class _Op:
    """A handle and the workspace it works in."""

    def __init__(self, nbytes: int, create, destroy, device):
        if nbytes == 0:
            raise EpError(EP_ERR_INVALID_ARG, ep.ep_last_error())
        raw = torch.empty(nbytes + 255, dtype=torch.uint8, device=device)
        skip = -raw.data_ptr() % 256
        self.workspace = raw[skip:skip + nbytes]
        self.device = self.workspace.device
        self._destroy = destroy
        self._handle = create(self.workspace.data_ptr(), nbytes)

    def __del__(self):
        h = getattr(self, "_handle", None)
        if h:
            self._destroy(h)
            self._handle = None

    def _stream(self):
        return torch.cuda.current_stream(self.device).cuda_stream

    def _need(self, t, what: str, shape, dtype, optional: bool = False) -> None:
        if t is None:
            if not optional:
                _refuse(f"{what} must be given")
            return
        if t.dtype != dtype or t.device != self.device or not t.is_contiguous() or \
                tuple(t.shape) != tuple(shape):
            _refuse(f"{what} must be a contiguous {dtype} {tuple(shape)} tensor on {self.device}, "
                    f"got {t.dtype} {tuple(t.shape)} on {t.device}"
                    f"{'' if t.is_contiguous() else ' (strided)'}")


# --------------------------------------------------------------------- router

@dataclass
class EpRouterConfig:
    """ep_router_config; the logits of all source ranks come as [R, Tmax, E]."""
    world_size: int
    max_num_inp_token_per_rank: int
    num_experts: int
    num_experts_per_token: int
    logits_dtype: torch.dtype = torch.float32   # float32 or bfloat16
    score_func: str = "softmax"                 # "softmax" | "sigmoid"
    num_groups: int = 1
    topk_groups: int = 1
    normalize_weights: bool = True
    route_scale: float = 1.0
    seq_len: int = 0            # balance loss: tokens per segment; 0: all of them are one
    balance_coef: float = 1.0

    def to_c(self) -> ep.ep_router_config:
        c = ep.ep_router_config()
        for n in ("world_size", "max_num_inp_token_per_rank", "num_experts",
                  "num_experts_per_token", "num_groups", "topk_groups", "seq_len"):
            setattr(c, n, int(getattr(self, n)))
        c.logits_dtype = _code(_FLOAT_OF, self.logits_dtype, "logits_dtype")
        c.score_func = _code(_SCORE_OF, self.score_func, "score_func")
        c.normalize_weights = int(bool(self.normalize_weights))
        c.route_scale = float(self.route_scale)
        c.balance_coef = float(self.balance_coef)
        return c


class EpRouterOp(_Op):
    """Router over one workspace. `num_tokens` gives each source rank's token
    count (default Tmax); rows past it get index -1, weight 0, gradient 0."""

    def __init__(self, config: EpRouterConfig, device: torch.device | str = "cuda"):
        self.config = config
        c = config.to_c()
        super().__init__(ep.ep_router_workspace_size(c),
                         lambda ws, n: ep.ep_router_create(c, ws, n), ep.ep_router_destroy,
                         device)
        R, T = config.world_size, config.max_num_inp_token_per_rank
        self.num_segments = R * -(-T // config.seq_len) if config.seq_len > 0 else 1
        self._slots = (R, T, config.num_experts_per_token)
        self._rows = (R, T, config.num_experts)
        self._counts = (self.num_segments, config.num_experts)

    def _tokens(self, num_tokens):
        if num_tokens is not None and len(num_tokens) != self.config.world_size:
            _refuse("num_tokens must give one count per source rank")
        return num_tokens

    def _new(self, shape, dtype):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def forward(self, logits, bias=None, num_tokens=None, balance=False):
        """(weights, indices), and with balance (weights, indices, counts, loss):
        weights [R, Tmax, k] f32 and indices [R, Tmax, k] int32 are dispatch's inputs;
        counts [segments, E] int32; loss an f32 scalar."""
        self._need(logits, "logits", self._rows, self.config.logits_dtype)
        self._need(bias, "bias", (self.config.num_experts,), torch.float32, optional=True)
        indices = self._new(self._slots, torch.int32)
        weights = self._new(self._slots, torch.float32)
        counts = self._new(self._counts, torch.int32) if balance else None
        loss = self._new((), torch.float32) if balance else None
        ep.ep_router_forward(self._handle, _ptr(logits), _ptr(bias), self._tokens(num_tokens),
                             _ptr(indices), _ptr(weights), _ptr(counts), _ptr(loss),
                             self._stream())
        return (weights, indices, counts, loss) if balance else (weights, indices)

    def balance_loss(self, logits, indices, num_tokens=None):
        """(counts, loss) of indices decided elsewhere."""
        self._need(logits, "logits", self._rows, self.config.logits_dtype)
        self._need(indices, "indices", self._slots, torch.int32)
        counts, loss = self._new(self._counts, torch.int32), self._new((), torch.float32)
        ep.ep_router_balance_loss(self._handle, _ptr(logits), _ptr(indices),
                                  self._tokens(num_tokens), _ptr(counts), _ptr(loss),
                                  self._stream())
        return counts, loss

    def backward(self, logits, indices=None, d_weights=None, counts=None, d_loss=None,
                 num_tokens=None, out=None):
        """d_logits from d_weights (with the forward's indices), from d_loss (with the
        loss's counts), or from both."""
        self._need(logits, "logits", self._rows, self.config.logits_dtype)
        self._need(indices, "indices", self._slots, torch.int32, optional=d_weights is None)
        self._need(d_weights, "d_weights", self._slots, torch.float32, optional=True)
        self._need(counts, "counts", self._counts, torch.int32, optional=d_loss is None)
        self._need(d_loss, "d_loss", (), torch.float32, optional=counts is None)
        self._need(out, "out", self._rows, self.config.logits_dtype, optional=True)
        if out is None:
            out = self._new(self._rows, self.config.logits_dtype)
        ep.ep_router_backward(self._handle, _ptr(logits), _ptr(indices),
                              self._tokens(num_tokens), _ptr(d_weights), _ptr(counts),
                              _ptr(d_loss), _ptr(out), self._stream())
        return out

    def sync(self):
        ep.ep_router_sync(self._handle, self._stream())


# ---------------------------------------------------------- experts' products

@dataclass
class EpLinearConfig:
    """ep_linear_config: y = act(x W_g^T + b_g) + residual over the segments of a pool
    of max_rows rows (num_groups 1 and no segments: one dense product)."""
    num_groups: int
    in_features: int
    out_features: int
    max_rows: int
    out_dtype: torch.dtype = torch.bfloat16           # of y, residual and dy
    weight_grad_dtype: torch.dtype = torch.bfloat16   # of dweight
    activation: str = "none"    # "none" | "relu" | "silu" | "gelu" | "swiglu"
    groups_per_base: int = 0    # with row_base: segments that share an entry of it

    @property
    def weight_rows(self) -> int:
        return self.out_features * (2 if self.activation == "swiglu" else 1)

    def to_c(self, backward: bool) -> ep.ep_linear_config:
        c = ep.ep_linear_config()
        for n in ("num_groups", "groups_per_base", "in_features", "out_features", "max_rows"):
            setattr(c, n, int(getattr(self, n)))
        c.out_dtype = _code(_FLOAT_OF, self.out_dtype, "out_dtype")
        c.weight_grad_dtype = _code(_FLOAT_OF, self.weight_grad_dtype, "weight_grad_dtype")
        c.activation = _code(_ACT_OF, self.activation, "activation")
        c.backward = int(bool(backward))
        return c


class EpLinearOp(_Op):
    """The product over one workspace (backward: reserve its scratch too).

    Segments: row_begin and row_count [G] int32, plus row_base (one entry per
    groups_per_base segments) where given; the packed layout's expert_offset,
    packed_recv_count and rank_base fit as they are. Without them, num_rows
    rows (default: all of x's)."""

    def __init__(self, config: EpLinearConfig, device: torch.device | str = "cuda",
                 backward: bool = False):
        self.config = config
        c = config.to_c(backward)
        super().__init__(ep.ep_linear_workspace_size(c),
                         lambda ws, n: ep.ep_linear_create(c, ws, n), ep.ep_linear_destroy,
                         device)

    def _rows(self, x, row_begin, row_count, row_base, num_rows):
        """Check x and the segments; the rows that pool tensors have."""
        cfg = self.config
        if x is None or x.dim() != 2 or x.shape[0] > cfg.max_rows:
            _refuse("x must be [rows, in_features] with at most max_rows rows")
        rows = x.shape[0]
        if (row_begin is None) != (row_count is None) or \
                (row_begin is None and (cfg.num_groups != 1 or row_base is not None)):
            _refuse("give row_begin and row_count together; only one group may go without")
        if row_begin is not None and rows != cfg.max_rows:
            _refuse("with segments, x must hold all max_rows rows of the pool")
        self._need(x, "x", (rows, cfg.in_features), torch.bfloat16)
        for name, t in (("row_begin", row_begin), ("row_count", row_count)):
            if t is not None:
                self._need(t.reshape(-1), name, (cfg.num_groups,), torch.int32)
                if not t.is_contiguous():
                    _refuse(f"{name} must be contiguous")
        if row_base is not None:
            per = cfg.groups_per_base
            if per < 1:
                _refuse("row_base needs groups_per_base")
            self._need(row_base, "row_base", (-(-cfg.num_groups // per),), torch.int32)
        n = rows if num_rows is None else int(num_rows)
        if not 0 <= n <= rows:
            _refuse("num_rows outside [0, rows of x]")
        return rows, n

    def _weight_shape(self):
        cfg = self.config
        return (cfg.num_groups, cfg.weight_rows, cfg.in_features)

    def forward(self, x, weight, bias=None, residual=None, row_begin=None, row_count=None,
                row_base=None, num_rows=None, out=None, preact=None):
        """y [rows, N] (in `out` if given). `preact`: a [rows, Nw] bf16 tensor that
        receives z for the backward pass. Rows outside the segments stay as they are."""
        cfg = self.config
        rows, n = self._rows(x, row_begin, row_count, row_base, num_rows)
        self._need(weight, "weight", self._weight_shape(), torch.bfloat16)
        self._need(bias, "bias", self._weight_shape()[:2], torch.float32, optional=True)
        self._need(residual, "residual", (rows, cfg.out_features), cfg.out_dtype, optional=True)
        self._need(out, "out", (rows, cfg.out_features), cfg.out_dtype, optional=True)
        self._need(preact, "preact", (rows, cfg.weight_rows), torch.bfloat16, optional=True)
        if out is None:
            out = torch.empty((rows, cfg.out_features), dtype=cfg.out_dtype, device=self.device)
        if rows == 0:
            return out
        ep.ep_linear_forward(self._handle, _ptr(x), _ptr(weight), _ptr(bias), _ptr(residual),
                             _ptr(row_begin), _ptr(row_count), _ptr(row_base), n, _ptr(out),
                             _ptr(preact), self._stream())
        return out

    def backward(self, dy, x, weight, preact=None, row_begin=None, row_count=None, row_base=None,
                 num_rows=None, want_dx=True, want_dweight=True, want_dbias=False, dx=None,
                 dweight=None):
        """(dx, dweight, dbias), None where not wanted. dx's rows outside the segments
        stay as they are (`dx`, `dweight`: tensors to write to)."""
        cfg = self.config
        rows, n = self._rows(x, row_begin, row_count, row_base, num_rows)
        self._need(dy, "dy", (rows, cfg.out_features), cfg.out_dtype)
        self._need(weight, "weight", self._weight_shape(), torch.bfloat16)
        self._need(preact, "preact", (rows, cfg.weight_rows), torch.bfloat16,
                   optional=cfg.activation == "none")
        self._need(dx, "dx", (rows, cfg.in_features), torch.bfloat16, optional=True)
        self._need(dweight, "dweight", self._weight_shape(), cfg.weight_grad_dtype, optional=True)
        dev = self.device
        if want_dx and dx is None:
            dx = torch.empty((rows, cfg.in_features), dtype=torch.bfloat16, device=dev)
        if want_dweight and dweight is None:
            dweight = torch.empty(self._weight_shape(), dtype=cfg.weight_grad_dtype, device=dev)
        dbias = torch.empty(self._weight_shape()[:2], dtype=torch.float32, device=dev) \
            if want_dbias else None
        dx, dweight = dx if want_dx else None, dweight if want_dweight else None
        if rows == 0:
            for t in (dweight, dbias):
                if t is not None:
                    t.zero_()
            return dx, dweight, dbias
        if dx is not None or dweight is not None or dbias is not None:
            ep.ep_linear_backward(self._handle, _ptr(dy), _ptr(x), _ptr(weight), _ptr(preact),
                                  _ptr(row_begin), _ptr(row_count), _ptr(row_base), n, _ptr(dx),
                                  _ptr(dweight), _ptr(dbias), self._stream())
        return dx, dweight, dbias

    def sync(self):
        ep.ep_linear_sync(self._handle, self._stream())
