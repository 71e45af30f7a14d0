"""The selective state space scan and the short causal convolution before it, as libmoe calls: forward and
backward over packed prompts, and the one-token steps of decoding. A sequence mixer beside linear attention
(linattn.py).

    convolution  p_t = bias + sum_j weight[:, j] x_{t - (W-1) + j};  y = silu(p)
    scan         dt = softplus(delta + dt_bias);  h_t = exp(dt A) h_{t-1} + dt u_t B_t;  y = (C_t . h_t + skip u_t) silu(z_t)

States, sums and gradients of weights are fp32. Bounds and slots that only the device can check set bits of `err`
(MOE_FLAG_*). One instance holds outputs, workspaces and gradients for a fixed number of packed tokens T, so a call
allocates nothing.
"""
from __future__ import annotations

import torch

from . import _lib as M
from .linattn import on_stream

BF16 = torch.bfloat16


def _vector(name, x, n):
    if x is not None and (x.dtype != torch.float32 or x.shape != (n,) or not x.is_contiguous()):
        raise ValueError(f"{name} is fp32 [{n}], contiguous")


# (a small call's time is the host's: each check asks a tensor as little as it can)
def _rows(name, x, T, width):
    """Checks a bf16 [T, width] operand; returns the elements between tokens."""
    if x.shape != (T, width) or x.dtype is not BF16:
        raise ValueError(f"{name} is bf16 {[T, width]}, got {x.dtype} {list(x.shape)}")
    token, value = x.stride()
    if value != 1 and width > 1 and x.numel():
        raise ValueError(f"{name}: the values of a token have to be contiguous")
    if T < 2:
        return width  # (the stride of a single token means nothing)
    if token > 0x7FFFFFFF:
        raise ValueError(f"{name}: tokens lie less than 2^31 values apart")
    return token


def _group_rows(name, x, T, groups, width):
    """Checks a bf16 [T, groups, width] operand; returns the elements between tokens."""
    if x.shape != (T, groups, width) or x.dtype is not BF16:
        raise ValueError(f"{name} is bf16 {[T, groups, width]}, got {x.dtype} {list(x.shape)}")
    token, group, value = x.stride()
    if ((value != 1 and width > 1) or (group != width and groups > 1)) and x.numel():
        raise ValueError(f"{name}: the values of a token have to be contiguous")
    if T < 2:
        return groups * width
    if token > 0x7FFFFFFF:
        raise ValueError(f"{name}: tokens lie less than 2^31 values apart")
    return token


def _bounds(cu_seqlens, N):
    if cu_seqlens is not None and (cu_seqlens.dtype is not torch.int32 or cu_seqlens.shape != (N + 1,)
                                   or not cu_seqlens.is_contiguous()):
        raise ValueError(f"cu_seqlens is int32 [{N + 1}], contiguous")


def _like(name, x, shape, dtype):
    if x is not None and (x.shape != shape or x.dtype is not dtype or not x.is_contiguous()):
        raise ValueError(f"{name} is {dtype} {list(shape)}, contiguous")


def _cache(state, state_idx, T, shape, dtype):
    slots = state.shape[0] if state.dim() else 0
    _like("state", state, (slots, *shape), dtype)
    if state_idx is not None and (state_idx.dtype is not torch.int32 or state_idx.shape != (T,) or not state_idx.is_contiguous()):
        raise ValueError(f"state_idx is int32 [{T}], contiguous")
    return slots


class CausalConv:
    def __init__(self, weight, bias, T: int, N: int = 1, silu: bool = True, backward: bool = True):
        """weight: fp32 [D, W] (D a multiple of 8, W = 2 .. 4 taps, the last one the token's own); bias: fp32 [D] or None. T packed tokens
        of N sequences."""
        if weight.dtype != torch.float32 or weight.dim() != 2 or not weight.is_contiguous():
            raise ValueError("weight is fp32 [D, W], contiguous")
        self.D, self.W = weight.shape
        _vector("bias", bias, self.D)
        self.weight, self.bias, self.T, self.N, self.silu, self.trains = weight, bias, T, N, silu, backward
        self.dev = weight.device
        self.y = self._new(T, self.D)
        self.err = torch.zeros(1, dtype=torch.int32, device=self.dev)
        self._state_out = self._d_state_in = self._state_first = None
        self.saved = None
        if backward:
            self.dx = self._new(T, self.D)
            self.dw = self._new(self.D, self.W, dt=torch.float32)
            self.db = self._new(self.D, dt=torch.float32)
            self.ws_bytes = M.moe_workspace_size(M.MOE_OP_CONV_BWD, T=T, d=self.D, l=self.W, S=N)
            self.ws = self._new(max(self.ws_bytes, 256), dt=torch.uint8)

    def _new(self, *shape, dt=BF16):
        return torch.empty(shape, dtype=dt, device=self.dev)

    # buffers that only some callers want are made when first asked for
    @property
    def state_out(self):
        if self._state_out is None:
            self._state_out = self._new(self.N, self.W - 1, self.D)
        return self._state_out

    @property
    def d_state_in(self):
        if self._d_state_in is None:
            self._d_state_in = self._new(self.N, self.W - 1, self.D)
        return self._d_state_in

    def forward(self, x, cu_seqlens=None, state_in=None, want_state: bool = False, stream=None):
        """y [T, D] (bf16, this instance's buffer) for x [T, D], which may be a slice of wider rows. cu_seqlens (int32 [N + 1]): sequence n
        is the tokens cu_seqlens[n] .. cu_seqlens[n + 1] - 1; without it all have T / N. state_in [N, W - 1, D]: the inputs before each
        sequence; with want_state, state_out holds the last ones, and state_in may be state_out. What was given has to stay as it
        is until backward."""
        ldx = _rows("x", x, self.T, self.D)
        _bounds(cu_seqlens, self.N)
        _like("state_in", state_in, (self.N, self.W - 1, self.D), BF16)
        if want_state and state_in is not None and state_in.data_ptr() == self.state_out.data_ptr():
            # (the kernel needs the first states and the last ones apart, and so does a backward)
            with on_stream(stream, self.dev):
                if self._state_first is None:
                    self._state_first = torch.empty_like(state_in)
                state_in = self._state_first.copy_(state_in)
        if self.trains:
            self.saved = (x, cu_seqlens, state_in)
        M.moe_conv_fwd(x, self.weight, self.bias, cu_seqlens, state_in, self.N, self.T, self.D, self.W, ldx, self.D,
                       self.silu, self.y, self.state_out if want_state else None, self.err, stream)
        return self.y

    def backward(self, dy, d_state_out=None, stream=None):
        """dx [T, D] of the last forward for dy = d loss / d y and d_state_out = d loss / d state_out; dw and db hold the weights'
        gradients, and where the forward was given a state or d_state_out is given, d_state_in the state's."""
        if not self.trains:
            raise ValueError("this instance was made without a backward")
        if self.saved is None:
            raise ValueError("backward needs a forward before it")
        x, cu_seqlens, state_in = self.saved
        ld = _rows("dy", dy, self.T, self.D), _rows("x", x, self.T, self.D)
        _like("d_state_out", d_state_out, (self.N, self.W - 1, self.D), BF16)
        want = state_in is not None or d_state_out is not None
        M.moe_conv_bwd(dy, x, self.weight, self.bias, cu_seqlens, state_in, d_state_out, self.N, self.T, self.D, self.W, *ld,
                       self.D, self.silu, self.dx, self.dw, self.db, self.d_state_in if want else None, self.ws,
                       self.ws_bytes, self.err, stream)
        return self.dx

    def step(self, x, state, state_idx=None, stream=None):
        """One token for each of T rows: y from x and the inputs kept in the cache [slots, W - 1, D] (bf16) at slot state_idx[row]
        (int32, negative for an empty row; default: the row), which moves on by x."""
        ldx = _rows("x", x, self.T, self.D)
        slots = _cache(state, state_idx, self.T, (self.W - 1, self.D), BF16)
        M.moe_conv_step(x, self.weight, self.bias, state, state_idx, slots, self.T, self.D, self.W, ldx, self.D, self.silu,
                        self.y, self.err, stream)
        return self.y


class SelectiveScan:
    def __init__(self, A, T: int, skip=None, dt_bias=None, groups: int = 1, N: int = 1, max_seqlen: int | None = None,
                 softplus: bool = True, backward: bool = True):
        """A: fp32 [D, S] (D a multiple of 8, S = 4, 8, 12 or 16 states a channel); skip, dt_bias: fp32 [D] or None. B and C have one row for each
        of `groups` equal runs of channels. T packed tokens of N sequences, none longer than max_seqlen (default: T / N); a
        longer one is skipped and flagged. An instance with a backward keeps the states before every 32nd token."""
        if A.dtype != torch.float32 or A.dim() != 2 or not A.is_contiguous():
            raise ValueError("A is fp32 [D, S], contiguous")
        self.D, self.S = A.shape
        if groups < 1 or self.D % groups:
            raise ValueError("groups divides D")
        _vector("skip", skip, self.D)
        _vector("dt_bias", dt_bias, self.D)
        self.A, self.skip, self.dt_bias, self.G = A, skip, dt_bias, groups
        self.T, self.N, self.softplus, self.trains = T, N, softplus, backward
        self.max_seqlen = (T // N if N else 0) if max_seqlen is None else min(max_seqlen, 0x7FFFFFFF)
        self.dev = A.device
        f32 = torch.float32
        self.y = self._new(T, self.D)
        self.err = torch.zeros(1, dtype=torch.int32, device=self.dev)
        self._state_out = self._d_state_in = self._dz = self.tile_states = None
        self.saved = None
        dims = dict(T=self.max_seqlen, d=self.D, l=self.S, E=groups, f=T, S=N)
        self.ws_bytes = M.moe_workspace_size(M.MOE_OP_SCAN_FWD, **dims)
        if backward:
            self.ws_bytes = max(self.ws_bytes, M.moe_workspace_size(M.MOE_OP_SCAN_BWD, **dims))
            self.tile_states = self._new(max(M.moe_workspace_size(M.MOE_OP_SCAN_TILE_STATES, **dims), 256), dt=torch.uint8)
            self.du, self.ddelta = self._new(T, self.D), self._new(T, self.D)
            self.dB, self.dC = self._new(T, groups, self.S), self._new(T, groups, self.S)
            self.dA, self.dskip, self.d_dt_bias = self._new(self.D, self.S, dt=f32), self._new(self.D, dt=f32), self._new(self.D, dt=f32)
        self.ws = self._new(max(self.ws_bytes, 256), dt=torch.uint8)

    def _new(self, *shape, dt=BF16):
        return torch.empty(shape, dtype=dt, device=self.dev)

    # buffers that only some callers want are made when first asked for
    @property
    def state_out(self):
        if self._state_out is None:
            self._state_out = self._new(self.N, self.D, self.S, dt=torch.float32)
        return self._state_out

    @property
    def d_state_in(self):
        if self._d_state_in is None:
            self._d_state_in = self._new(self.N, self.D, self.S, dt=torch.float32)
        return self._d_state_in

    @property
    def dz(self):
        if self._dz is None:
            self._dz = self._new(self.T, self.D)
        return self._dz

    def _operands(self, u, delta, B, C, z):
        T, D, G, S = self.T, self.D, self.G, self.S
        return (_rows("u", u, T, D), _rows("delta", delta, T, D), _group_rows("B", B, T, G, S), _group_rows("C", C, T, G, S),
                0 if z is None else _rows("z", z, T, D))

    def forward(self, u, delta, B, C, z=None, cu_seqlens=None, state_in=None, want_state: bool = False, stream=None):
        """y [T, D] (bf16, this instance's buffer) for u, delta and the gate z [T, D], B and C [T, groups, S]: slices of wider rows will
        do. cu_seqlens as in CausalConv.forward. state_in (fp32 [N, D, S]) is each sequence's state before its first
        token; with want_state, state_out holds those after the last, and state_in may be state_out. What else was given has to
        stay as it is until backward."""
        ld = self._operands(u, delta, B, C, z)
        _bounds(cu_seqlens, self.N)
        _like("state_in", state_in, (self.N, self.D, self.S), torch.float32)
        if self.trains:
            self.saved = (u, delta, B, C, z, cu_seqlens, state_in is not None)
        M.moe_scan_fwd(u, delta, self.A, B, C, self.skip, z, self.dt_bias, cu_seqlens, state_in, self.N, self.T,
                       self.max_seqlen, self.D, self.S, self.G, *ld, self.D, self.softplus, self.y,
                       self.state_out if want_state else None, self.tile_states, self.ws, self.ws_bytes, self.err, stream)
        return self.y

    def backward(self, dy, d_state_out=None, stream=None):
        """(du, ddelta, dB, dC, dz) of the last forward (dz None without a gate) for dy = d loss / d y and d_state_out = d loss /
        d state_out; dA, dskip and d_dt_bias hold the weights' gradients, and where the forward was given a state or
        d_state_out is given, d_state_in the state's."""
        if not self.trains:
            raise ValueError("this instance was made without a backward")
        if self.saved is None:
            raise ValueError("backward needs a forward before it")
        u, delta, B, C, z, cu_seqlens, had_state = self.saved
        ld = [_rows("dy", dy, self.T, self.D), *self._operands(u, delta, B, C, z)]
        _like("d_state_out", d_state_out, (self.N, self.D, self.S), torch.float32)
        want = had_state or d_state_out is not None
        dz = self.dz if z is not None else None
        M.moe_scan_bwd(dy, u, delta, self.A, B, C, self.skip, z, self.dt_bias, cu_seqlens, self.tile_states, d_state_out,
                       self.N, self.T, self.max_seqlen, self.D, self.S, self.G, *ld, self.softplus, self.du, self.ddelta,
                       self.dB, self.dC, dz, self.D, self.D, self.D, self.dA, self.dskip, self.d_dt_bias,
                       self.d_state_in if want else None, self.ws, self.ws_bytes, self.err, stream)
        return self.du, self.ddelta, self.dB, self.dC, dz

    def step(self, u, delta, B, C, z, state, state_idx=None, stream=None):
        """One token for each of T rows: updates the state cache [slots, D, S] (fp32) in place at slot state_idx[row]
        (int32, negative for an empty row; default: the row) and returns y. z may be None."""
        ld = self._operands(u, delta, B, C, z)
        slots = _cache(state, state_idx, self.T, (self.D, self.S), torch.float32)
        M.moe_scan_step(u, delta, self.A, B, C, self.skip, z, self.dt_bias, state, state_idx, slots, self.T, self.D, self.S,
                        self.G, *ld, self.D, self.softplus, self.y, self.err, stream)
        return self.y
