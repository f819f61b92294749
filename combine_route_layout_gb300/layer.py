"""What a mixture-of-experts layer has around dispatch and combine, on torch
tensors: the router with its balance loss (EpRouterOp) and the experts'
products (EpLinearOp). Argument checks and marshalling only; the work is the
CUDA kernels behind ep_router_* and ep_linear_* of include/ep.h, on torch's
current stream. An operator owns its workspace; calls on one operator are
ordered by the caller (same stream, or events), with the operator's device the
current one. Results carry no autograd graph, as dispatch's and combine's do not:
gradients come from the operators' own backward().
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import ep
from .ep import EP_ERR_INVALID_ARG, EpError, _check, _lib

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
        self._raw = torch.empty(nbytes + 255, dtype=torch.uint8, device=device)
        skip = -self._raw.data_ptr() % 256
        self.workspace = self._raw[skip:skip + nbytes]
        self.device = self.workspace.device
        self._device_index = self.device.index or 0
        # the stream that the allocator knows the workspace by, and others it was told of
        self._streams = {_raw_stream(self._device_index)} if self.device.type == "cuda" else {0}
        self._destroy = destroy
        self._handle = create(self.workspace.data_ptr(), nbytes)

    def __del__(self):
        h = getattr(self, "_handle", None)
        if h:
            self._destroy(h)
            self._handle = None

    def _stream(self):
        """torch's current stream of the workspace's device, as a pointer. That device has to
        be the current one, which is where the library launches. The allocator is told of a
        stream other than the workspace's own, so that freeing the operator waits for the
        work on it."""
        if torch.cuda.current_device() != self._device_index:
            _refuse(f"the operator is on {self.device}, which is not the current device "
                    f"({torch.cuda.current_device()})")
        s = _raw_stream(self._device_index)
        if s not in self._streams:
            self._raw.record_stream(torch.cuda.current_stream(self.device))
            self._streams.add(s)
        return s

    def _need(self, t, what: str, shape, dtype) -> int:
        """The address of a contiguous tensor of this shape and type on this device."""
        if t is None:
            _refuse(f"{what} must be given")
        if t.dtype is not dtype or t.shape != shape or t.device != self.device or \
                not t.is_contiguous():
            _refuse(f"{what} must be a contiguous {dtype} {tuple(shape)} tensor on {self.device}, "
                    f"got {t.dtype} {tuple(t.shape)} on {t.device}"
                    f"{'' if t.is_contiguous() else ' (strided)'}")
        return t.data_ptr()

    def _form(self, shape, dtype):
        """A tensor that results are made like: a third of the cost of making them from a shape."""
        return torch.empty(shape, dtype=dtype, device=self.device)


_new = torch.empty_like


def _raw_stream(device_index: int) -> int:
    return torch._C._cuda_getCurrentRawStream(device_index)


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
        R, T, E = config.world_size, config.max_num_inp_token_per_rank, config.num_experts
        self.num_segments = R * -(-T // config.seq_len) if config.seq_len > 0 else 1
        self._slots = torch.Size((R, T, config.num_experts_per_token))
        self._rows = torch.Size((R, T, E))
        self._counts = torch.Size((self.num_segments, E))
        self._scalar, self._bias = torch.Size(()), torch.Size((E,))
        self._indices_form = self._form(self._slots, torch.int32)
        self._weights_form = self._form(self._slots, torch.float32)
        self._counts_form = self._form(self._counts, torch.int32)
        self._loss_form = self._form((), torch.float32)
        self._last = (None, None)       # token counts and the C array that they became

    def _tokens(self, num_tokens):
        """The counts as a C array; the same counts as last time are not converted again."""
        if num_tokens is None:
            return None
        last, array = self._last
        if type(num_tokens) is list and num_tokens == last:
            return array
        if len(num_tokens) != self.config.world_size:
            _refuse("num_tokens must give one count per source rank")
        counts = [int(n) for n in num_tokens]
        array = ep._i32_array(counts)
        self._last = (counts, array)    # in one step: host threads may ask meanwhile
        return array

    def forward(self, logits, bias=None, num_tokens=None, balance=False):
        """(weights, indices), and with balance (weights, indices, counts, loss):
        weights [R, Tmax, k] f32 and indices [R, Tmax, k] int32 are dispatch's inputs;
        counts [segments, E] int32; loss an f32 scalar."""
        x = self._need(logits, "logits", self._rows, self.config.logits_dtype)
        b = None if bias is None else self._need(bias, "bias", self._bias, torch.float32)
        tokens = self._tokens(num_tokens)
        indices, weights = _new(self._indices_form), _new(self._weights_form)
        if not balance:
            _check(_lib.ep_router_forward(self._handle, x, b, tokens, indices.data_ptr(),
                                          weights.data_ptr(), None, None, self._stream()))
            return weights, indices
        counts, loss = _new(self._counts_form), _new(self._loss_form)
        _check(_lib.ep_router_forward(self._handle, x, b, tokens, indices.data_ptr(),
                                      weights.data_ptr(), counts.data_ptr(), loss.data_ptr(),
                                      self._stream()))
        return weights, indices, counts, loss

    def balance_loss(self, logits, indices, num_tokens=None):
        """(counts, loss) of indices decided elsewhere."""
        x = self._need(logits, "logits", self._rows, self.config.logits_dtype)
        i = self._need(indices, "indices", self._slots, torch.int32)
        counts, loss = _new(self._counts_form), _new(self._loss_form)
        _check(_lib.ep_router_balance_loss(self._handle, x, i, self._tokens(num_tokens),
                                           counts.data_ptr(), loss.data_ptr(), self._stream()))
        return counts, loss

    def backward(self, logits, indices=None, d_weights=None, counts=None, d_loss=None,
                 num_tokens=None, out=None):
        """d_logits from d_weights (with the forward's indices), from d_loss (with the
        loss's counts), or from both."""
        dt = self.config.logits_dtype
        x = self._need(logits, "logits", self._rows, dt)
        i = w = c = d = None
        if d_weights is not None:
            w = self._need(d_weights, "d_weights", self._slots, torch.float32)
        if indices is not None or w is not None:
            i = self._need(indices, "indices", self._slots, torch.int32)
        if counts is not None or d_loss is not None:
            c = self._need(counts, "counts", self._counts, torch.int32)
            d = self._need(d_loss, "d_loss", self._scalar, torch.float32)
        if out is None:
            out = torch.empty_like(logits)
            o = out.data_ptr()
        else:
            o = self._need(out, "out", self._rows, dt)
        _check(_lib.ep_router_backward(self._handle, x, i, self._tokens(num_tokens), w, c, d, o,
                                       self._stream()))
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

        G, Nw = config.num_groups, config.weight_rows
        self._weight = torch.Size((G, Nw, config.in_features))
        self._bias = torch.Size((G, Nw))
        self._act_none = config.activation == "none"

    def _per_group(self, t, what: str, n: int) -> int:
        if t.dtype is not torch.int32 or t.numel() != n or t.device != self.device or \
                not t.is_contiguous():
            _refuse(f"{what} must hold {n} contiguous int32 on {self.device}")
        return t.data_ptr()

    def _segments(self, x, row_begin, row_count, row_base, num_rows):
        """Check x and the segments: (rows of pool tensors, row_begin, row_count, row_base,
        num_rows) as the C calls take them."""
        cfg = self.config
        if x is None or x.dim() != 2 or x.shape[0] > cfg.max_rows:
            _refuse("x must be [rows, in_features] with at most max_rows rows")
        rows = x.shape[0]
        if row_begin is None or row_count is None:
            if row_begin is not row_count or cfg.num_groups != 1 or row_base is not None:
                _refuse("give row_begin and row_count together; only one group may go without")
            n = rows if num_rows is None else int(num_rows)
            if not 0 <= n <= rows:
                _refuse("num_rows outside [0, rows of x]")
            return rows, None, None, None, n
        if rows != cfg.max_rows:
            _refuse("with segments, x must hold all max_rows rows of the pool")
        base = None
        if row_base is not None:
            per = cfg.groups_per_base
            if per < 1:
                _refuse("row_base needs groups_per_base")
            base = self._per_group(row_base, "row_base", -(-cfg.num_groups // per))
        return (rows, self._per_group(row_begin, "row_begin", cfg.num_groups),
                self._per_group(row_count, "row_count", cfg.num_groups), base, 0)

    def forward(self, x, weight, bias=None, residual=None, row_begin=None, row_count=None,
                row_base=None, num_rows=None, out=None, preact=None):
        """y [rows, N] (in `out` if given). `preact`: a [rows, Nw] bf16 tensor that
        receives z for the backward pass. Rows outside the segments stay as they are."""
        cfg = self.config
        rows, begin, count, base, n = self._segments(x, row_begin, row_count, row_base, num_rows)
        xp = self._need(x, "x", (rows, cfg.in_features), torch.bfloat16)
        w = self._need(weight, "weight", self._weight, torch.bfloat16)
        b = r = z = None
        if bias is not None:
            b = self._need(bias, "bias", self._bias, torch.float32)
        if residual is not None:
            r = self._need(residual, "residual", (rows, cfg.out_features), cfg.out_dtype)
        if preact is not None:
            z = self._need(preact, "preact", (rows, cfg.weight_rows), torch.bfloat16)
        if out is None:
            out = torch.empty((rows, cfg.out_features), dtype=cfg.out_dtype, device=self.device)
            y = out.data_ptr()
        else:
            y = self._need(out, "out", (rows, cfg.out_features), cfg.out_dtype)
        if rows:
            _check(_lib.ep_linear_forward(self._handle, xp, w, b, r, begin, count, base, n, y, z,
                                          self._stream()))
        return out

    def backward(self, dy, x, weight, preact=None, row_begin=None, row_count=None, row_base=None,
                 num_rows=None, want_dx=True, want_dweight=True, want_dbias=False, dx=None,
                 dweight=None):
        """(dx, dweight, dbias), None where not wanted. dx's rows outside the segments
        stay as they are (`dx`, `dweight`: tensors to write to)."""
        cfg, bf16 = self.config, torch.bfloat16
        rows, begin, count, base, n = self._segments(x, row_begin, row_count, row_base, num_rows)
        xp = self._need(x, "x", (rows, cfg.in_features), bf16)
        w = self._need(weight, "weight", self._weight, bf16)
        dyp = self._need(dy, "dy", (rows, cfg.out_features), cfg.out_dtype)
        z = dxp = dwp = dbp = dbias = None
        if preact is not None or not self._act_none:
            z = self._need(preact, "preact", (rows, cfg.weight_rows), bf16)
        if not want_dx:
            dx = None
        elif dx is None:
            dx = torch.empty_like(x)
            dxp = dx.data_ptr()
        else:
            dxp = self._need(dx, "dx", x.shape, bf16)
        if not want_dweight:
            dweight = None
        elif dweight is None:
            dweight = torch.empty(self._weight, dtype=cfg.weight_grad_dtype, device=self.device)
            dwp = dweight.data_ptr()
        else:
            dwp = self._need(dweight, "dweight", self._weight, cfg.weight_grad_dtype)
        if want_dbias:
            dbias = torch.empty(self._bias, dtype=torch.float32, device=self.device)
            dbp = dbias.data_ptr()
        if rows == 0:
            for t in (dweight, dbias):
                if t is not None:
                    t.zero_()
        elif dxp or dwp or dbp:
            _check(_lib.ep_linear_backward(self._handle, dyp, xp, w, z, begin, count, base, n,
                                           dxp, dwp, dbp, self._stream()))
        return dx, dweight, dbias

    def sync(self):
        ep.ep_linear_sync(self._handle, self._stream())
