"""What a mixture-of-experts layer has around dispatch and combine, on torch
tensors: the router with its balance loss (EpRouterOp), the experts' products
(EpLinearOp) and their form for the E4M3 rows of FP8 dispatch (EpQuantLinearOp),
the quantiser (EpQuantOp), and the norms around the layer (EpNormOp). Argument
checks and marshalling only; the work is the CUDA kernels behind ep_router_*,
ep_linear_*, ep_qlinear_*, ep_quant* and ep_norm_* of include/ep.h, on torch's
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
_GATE_OF = {"none": ep.EP_GATE_NONE, "token": ep.EP_GATE_TOKEN, "feature": ep.EP_GATE_FEATURE}
_QUANT_OF = {"none": ep.EP_QUANT_NONE, "fp8_e4m3_block128": ep.EP_QUANT_FP8_E4M3_BLOCK128}
_E4M3 = torch.float8_e4m3fn


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


class _PoolOp(_Op):
    """An operator over the segments of a pool of max_rows rows, as its config has them."""

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
            _refuse("x must be [rows, features] with at most max_rows rows")
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


_new = torch.empty_like


def _empty(rows: int, cols: int, dtype, device):
    """torch.empty of a matrix, whose strides given take half of its time."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


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


class EpLinearOp(_PoolOp):
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


# -------------------------------------------------------- block quantisation

def _blocks(n: int) -> int:
    return -(-n // ep.EP_QUANT_BLOCK)


@dataclass
class EpQuantConfig:
    """ep_quant_config: E4M3 codes with an f32 scale for each 128 elements of a row
    (block_rows 1) or for each 128 x 128 of num_groups matrices of max_rows rows
    (block_rows 128)."""
    num_groups: int
    features: int
    max_rows: int
    block_rows: int = 1
    dtype: torch.dtype = torch.bfloat16   # of what is quantised: bfloat16 or float32
    groups_per_base: int = 0    # with row_base: segments that share an entry of it

    def to_c(self) -> ep.ep_quant_config:
        c = ep.ep_quant_config()
        for n in ("num_groups", "groups_per_base", "features", "block_rows", "max_rows"):
            setattr(c, n, int(getattr(self, n)))
        c.dtype = _code(_FLOAT_OF, self.dtype, "dtype")
        return c


class EpQuantOp(_PoolOp):
    """The quantiser over one workspace. Rows: [rows, K] tensors and EpLinearOp's
    segments. Matrices: [G, max_rows, K] tensors, scales [G, ceil(max_rows / 128),
    ceil(K / 128)]; SWIGLU's [G, 2 N, K] weights are 2 G matrices of N rows."""

    def __init__(self, config: EpQuantConfig, device: torch.device | str = "cuda"):
        self.config = config
        c = config.to_c()
        super().__init__(ep.ep_quant_workspace_size(c), lambda ws, n: ep.ep_quant_create(c, ws, n),
                         ep.ep_quant_destroy, device)
        self._kb = _blocks(config.features)
        G, M = config.num_groups, config.max_rows
        self._matrices = torch.Size((G, M, config.features))
        self._matrix_scales = torch.Size((G, _blocks(M), self._kb))

    def _places(self, t, row_begin, row_count, row_base, num_rows):
        """(shape of t, shape of its scales, segments as the C calls take them)."""
        cfg = self.config
        if cfg.block_rows == 1:
            rows, *at = self._segments(t, row_begin, row_count, row_base, num_rows)
            return (rows, cfg.features), (rows, self._kb), at
        if any(v is not None for v in (row_begin, row_count, row_base, num_rows)):
            _refuse("blocks of 128 rows take whole matrices: no segments")
        return self._matrices, self._matrix_scales, (None, None, None, cfg.max_rows)

    def quantize(self, x, row_begin=None, row_count=None, row_base=None, num_rows=None, codes=None,
                 scales=None):
        """(codes, scales) of x (in `codes` and `scales` if given). Rows outside the
        segments stay as they are."""
        shape, scale_shape, at = self._places(x, row_begin, row_count, row_base, num_rows)
        xp = self._need(x, "x", shape, self.config.dtype)
        if codes is None:
            codes = torch.empty(shape, dtype=_E4M3, device=self.device)
            cp = codes.data_ptr()
        else:
            cp = self._need(codes, "codes", shape, _E4M3)
        if scales is None:
            scales = torch.empty(scale_shape, dtype=torch.float32, device=self.device)
            sp = scales.data_ptr()
        else:
            sp = self._need(scales, "scales", scale_shape, torch.float32)
        if shape[0]:
            _check(_lib.ep_quantize(self._handle, xp, *at, cp, sp, self._stream()))
        return codes, scales

    def dequantize(self, codes, scales, row_begin=None, row_count=None, row_base=None, num_rows=None,
                   out=None):
        """What codes and scales stand for, rounded to the config's dtype."""
        shape, scale_shape, at = self._places(codes, row_begin, row_count, row_base, num_rows)
        cp = self._need(codes, "codes", shape, _E4M3)
        sp = self._need(scales, "scales", scale_shape, torch.float32)
        if out is None:
            out = torch.empty(shape, dtype=self.config.dtype, device=self.device)
            xp = out.data_ptr()
        else:
            xp = self._need(out, "out", shape, self.config.dtype)
        if shape[0]:
            _check(_lib.ep_dequantize(self._handle, cp, sp, *at, xp, self._stream()))
        return out

    def sync(self):
        ep.ep_quant_sync(self._handle, self._stream())


# ----------------------------------- experts' products of quantised operands

class EpQuantLinearOp(_PoolOp):
    """EpLinearOp's product of E4M3 operands: x [rows, K] with x_scale [rows, ceil(K / 128)],
    as FP8 dispatch or EpQuantOp gives them, and weight [G, Nw, K] with weight_scale
    [G, Nw / N ceil(N / 128), ceil(K / 128)]. The rest is EpLinearOp's, except that
    in_features is a multiple of 16."""

    def __init__(self, config: EpLinearConfig, device: torch.device | str = "cuda",
                 backward: bool = False):
        self.config = config
        c = config.to_c(backward)
        super().__init__(ep.ep_qlinear_workspace_size(c),
                         lambda ws, n: ep.ep_qlinear_create(c, ws, n), ep.ep_qlinear_destroy,
                         device)
        G, N, Nw = config.num_groups, config.out_features, config.weight_rows
        self._kb = _blocks(config.in_features)
        self._weight = torch.Size((G, Nw, config.in_features))
        self._weight_scale = torch.Size((G, Nw // N * _blocks(N), self._kb))
        self._bias = torch.Size((G, Nw))
        self._act_none = config.activation == "none"

    def _operands(self, rows, x, x_scale, weight, weight_scale):
        return (self._need(x, "x", (rows, self.config.in_features), _E4M3),
                self._need(x_scale, "x_scale", (rows, self._kb), torch.float32),
                self._need(weight, "weight", self._weight, _E4M3),
                self._need(weight_scale, "weight_scale", self._weight_scale, torch.float32))

    def forward(self, x, x_scale, weight, weight_scale, bias=None, residual=None, row_begin=None,
                row_count=None, row_base=None, num_rows=None, out=None, preact=None):
        """y [rows, N] (in `out` if given). `preact`: a [rows, Nw] bf16 tensor that
        receives z for the backward pass. Rows outside the segments stay as they are."""
        cfg = self.config
        rows, *at = self._segments(x, row_begin, row_count, row_base, num_rows)
        operands = self._operands(rows, x, x_scale, weight, weight_scale)
        b = r = z = None
        if bias is not None:
            b = self._need(bias, "bias", self._bias, torch.float32)
        if residual is not None:
            r = self._need(residual, "residual", (rows, cfg.out_features), cfg.out_dtype)
        if preact is not None:
            z = self._need(preact, "preact", (rows, cfg.weight_rows), torch.bfloat16)
        if out is None:
            out = _empty(rows, cfg.out_features, cfg.out_dtype, self.device)
            y = out.data_ptr()
        else:
            y = self._need(out, "out", (rows, cfg.out_features), cfg.out_dtype)
        if rows:
            _check(_lib.ep_qlinear_forward(self._handle, *operands, b, r, *at, y, z,
                                           self._stream()))
        return out

    def backward(self, dy, x, x_scale, weight, weight_scale, preact=None, row_begin=None,
                 row_count=None, row_base=None, num_rows=None, want_dx=True, want_dweight=True,
                 want_dbias=False, dx=None, dweight=None):
        """(dx, dweight, dbias), None where not wanted: dx bf16, dweight [G, Nw, K] of
        weight_grad_dtype. dx's rows outside the segments stay as they are (`dx`,
        `dweight`: tensors to write to)."""
        cfg, bf16 = self.config, torch.bfloat16
        rows, *at = self._segments(x, row_begin, row_count, row_base, num_rows)
        operands = self._operands(rows, x, x_scale, weight, weight_scale)
        dyp = self._need(dy, "dy", (rows, cfg.out_features), cfg.out_dtype)
        z = dxp = dwp = dbp = dbias = None
        if preact is not None or not self._act_none:
            z = self._need(preact, "preact", (rows, cfg.weight_rows), bf16)
        if not want_dx:
            dx = None
        elif dx is None:
            dx = _empty(rows, cfg.in_features, bf16, self.device)
            dxp = dx.data_ptr()
        else:
            dxp = self._need(dx, "dx", (rows, cfg.in_features), bf16)
        if not want_dweight:
            dweight = None
        elif dweight is None:
            dweight = torch.empty(self._weight, dtype=cfg.weight_grad_dtype, device=self.device)
            dwp = dweight.data_ptr()
        else:
            dwp = self._need(dweight, "dweight", self._weight, cfg.weight_grad_dtype)
        if want_dbias:
            dbias = _empty(*self._bias, torch.float32, self.device)
            dbp = dbias.data_ptr()
        if rows == 0:
            for t in (dweight, dbias):
                if t is not None:
                    t.zero_()
        elif dxp or dwp or dbp:
            _check(_lib.ep_qlinear_backward(self._handle, dyp, *operands, z, *at, dxp, dwp, dbp,
                                            self._stream()))
        return dx, dweight, dbias

    def sync(self):
        ep.ep_qlinear_sync(self._handle, self._stream())


# ---------------------------------------------------------------------- norms

@dataclass
class EpNormConfig:
    """ep_norm_config: stream = residual + residual_scale gate u, with u the block's
    output or (post_norm) its norm, and out = norm(stream)."""
    hidden_dim: int
    max_rows: int
    eps: float = 1e-6
    post_norm: bool = False
    gate: str = "none"          # "none" | "token" | "feature"
    residual_scale: float = 1.0
    stream_dtype: torch.dtype = torch.bfloat16   # of residual and stream: bfloat16 or float32
    block_dtype: torch.dtype = torch.bfloat16    # of the block's output: combine's type
    quant_type: str = "none"    # "none": out is bf16 | "fp8_e4m3_block128": codes with scales

    def to_c(self, backward: bool) -> ep.ep_norm_config:
        c = ep.ep_norm_config()
        c.hidden_dim, c.max_rows = int(self.hidden_dim), int(self.max_rows)
        c.eps, c.residual_scale = float(self.eps), float(self.residual_scale)
        c.post_norm = int(bool(self.post_norm))
        c.gate = _code(_GATE_OF, self.gate, "gate")
        c.quant_type = _code(_QUANT_OF, self.quant_type, "quant_type")
        c.stream_dtype = _code(_FLOAT_OF, self.stream_dtype, "stream_dtype")
        c.block_dtype = _code(_FLOAT_OF, self.block_dtype, "block_dtype")
        c.backward = int(bool(backward))
        return c


class EpNormOp(_Op):
    """The norms around a block over one workspace (backward: reserve its scratch too).
    Tensors are [rows, hidden_dim] with at most max_rows rows; weight, weight_post and a
    gate of features are f32 [hidden_dim], a gate of tokens is f32 [rows]."""

    def __init__(self, config: EpNormConfig, device: torch.device | str = "cuda",
                 backward: bool = False):
        self.config = config
        c = config.to_c(backward)
        super().__init__(ep.ep_norm_workspace_size(c), lambda ws, n: ep.ep_norm_create(c, ws, n),
                         ep.ep_norm_destroy, device)
        self._features = torch.Size((config.hidden_dim,))
        self._hb = _blocks(config.hidden_dim)
        self._quant = config.quant_type != "none"

    def _shared(self, t, weight, block, weight_post, gate):
        """(shape, block, gate, weight_post, weight) of a call, the last four as addresses."""
        cfg = self.config
        if t is None or t.dim() != 2 or t.shape[0] > cfg.max_rows:
            _refuse("tensors must be [rows, hidden_dim] with at most max_rows rows")
        shape = t.shape
        f32, b, p, g = torch.float32, None, None, None
        if block is not None:
            b = self._need(block, "block", shape, cfg.block_dtype)
            if cfg.post_norm:
                p = self._need(weight_post, "weight_post", self._features, f32)
            if cfg.gate != "none":
                g = self._need(gate, "gate", self._features if cfg.gate == "feature" else shape[:1], f32)
        if (weight_post is not None) != (p is not None) or (gate is not None) != (g is not None):
            _refuse("weight_post and gate go with a block and the config's post_norm and gate")
        return shape, b, g, p, self._need(weight, "weight", self._features, f32)

    def forward(self, residual, weight, block=None, weight_post=None, gate=None, stream=None,
                out=None, scales=None, stats=None):
        """(stream, out, scales, stats): stream is `residual` itself without a block; out is
        bf16, scales None, or E4M3 codes with f32 scales [rows, ceil(hidden_dim / 128)];
        stats [rows, 2] f32 are for the backward pass. `stream` (which may be
        `residual`), `out`, `scales`, `stats`: tensors to write to."""
        cfg, dev, f32 = self.config, self.device, torch.float32
        shape, b, g, p, w = self._shared(residual, weight, block, weight_post, gate)
        rows = shape[0]
        r = self._need(residual, "residual", (rows, cfg.hidden_dim), cfg.stream_dtype)
        s = sc = None
        if b is None:
            if stream is not None and stream is not residual:
                _refuse("without a block, stream is the residual")
            stream = residual
        elif stream is None:
            stream = _new(residual)
            s = stream.data_ptr()
        else:
            s = self._need(stream, "stream", shape, cfg.stream_dtype)
        dt = _E4M3 if self._quant else torch.bfloat16
        if out is None:
            out = _empty(rows, cfg.hidden_dim, dt, dev)
            o = out.data_ptr()
        else:
            o = self._need(out, "out", shape, dt)
        if not self._quant:
            if scales is not None:
                _refuse("scales go with quantisation")
        elif scales is None:
            scales = _empty(rows, self._hb, f32, dev)
            sc = scales.data_ptr()
        else:
            sc = self._need(scales, "scales", (rows, self._hb), f32)
        if stats is None:
            stats = _empty(rows, 2, f32, dev)
            st = stats.data_ptr()
        else:
            st = self._need(stats, "stats", (rows, 2), f32)
        if rows:
            _check(_lib.ep_norm_forward(self._handle, r, b, g, p, w, rows, s, o, sc, st,
                                        self._stream()))
        return stream, out, scales, stats

    def backward(self, d_out, stream, weight, stats, d_stream=None, block=None, weight_post=None,
                 gate=None, d_residual=None):
        """(d_residual, d_block, d_weight, d_weight_post, d_gate), None for what the forward
        pass did not take, from d_out [rows, hidden_dim] bf16, the stream's own gradient and
        what forward took and gave. `d_residual` (a tensor to write to) may be `d_stream`."""
        cfg, dev, f32 = self.config, self.device, torch.float32
        shape, b, g, p, w = self._shared(stream, weight, block, weight_post, gate)
        rows = shape[0]
        s = self._need(stream, "stream", (rows, cfg.hidden_dim), cfg.stream_dtype)
        do = self._need(d_out, "d_out", shape, torch.bfloat16)
        ds = None if d_stream is None else self._need(d_stream, "d_stream", shape, cfg.stream_dtype)
        st = self._need(stats, "stats", (rows, 2), f32)
        if d_residual is None:
            d_residual = _new(stream)
            dr = d_residual.data_ptr()
        else:
            dr = self._need(d_residual, "d_residual", shape, cfg.stream_dtype)
        d_weight = _new(weight)
        d_block = d_post = d_gate = None
        db = dp = dg = None
        if b is not None:
            d_block = _new(block)
            db = d_block.data_ptr()
            if p is not None:
                d_post = _new(weight_post)
                dp = d_post.data_ptr()
            if g is not None:
                d_gate = _new(gate)
                dg = d_gate.data_ptr()
        if rows:
            _check(_lib.ep_norm_backward(self._handle, do, ds, s, b, g, p, w, st, rows, dr, db,
                                         d_weight.data_ptr(), dp, dg, self._stream()))
        else:
            for t in (d_weight, d_post, d_gate):
                if t is not None:
                    t.zero_()
        return d_residual, d_block, d_weight, d_post, d_gate

    def sync(self):
        ep.ep_norm_sync(self._handle, self._stream())
