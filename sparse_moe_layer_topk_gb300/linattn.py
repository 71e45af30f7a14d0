"""Linear attention with a decay for each state head, the sequence mixer of a
block, as libmoe calls: chunked forward over packed prompts, its backward, and
the one-token step of decoding.

    S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T;   o_t = scale S_t^T q_t

Hs state heads, each read by r query heads. The chunked passes hold and sum states in fp32 from
products of bf16 terms: states are 3e-6 off (rms), outputs and gradients up to 2.4e-3, of which
1.7e-3 is their own rounding to bf16; the step is fp32 throughout. Bounds, slots and decays that only
the device can check set bits of `err` (MOE_FLAG_*). PyTorch only provides the device
buffers and the stream. One instance holds the outputs, workspaces and gradients
for a fixed number of packed tokens T, so a call allocates nothing.
"""
from __future__ import annotations

import torch

from . import _lib as M

BF16 = torch.bfloat16


class LinearAttention:
    def __init__(self, log_decay, T: int, Dk: int, Dv: int, r: int = 1, N: int = 1,
                 max_seqlen: int | None = None, scale: float | None = None, backward: bool = True):
        """log_decay: fp32 [Hs] on the device, <= 0. T packed tokens of N sequences, none
        longer than max_seqlen (default: T / N where the sequences are of one length, else T
        has to be given); a longer one is skipped and flagged. scale: Dk ** -0.5 if not given."""
        if log_decay.dtype != torch.float32 or log_decay.dim() != 1:
            raise ValueError("log_decay is an fp32 vector with one entry for each state head")
        self.log_decay = log_decay.contiguous()
        self.Hs, self.r, self.Dk, self.Dv, self.T, self.N = log_decay.numel(), r, Dk, Dv, T, N
        self.max_seqlen = (T // N if N else 0) if max_seqlen is None else min(max_seqlen, 0x7FFFFFFF)
        self.scale = Dk ** -0.5 if scale is None else scale
        dev = log_decay.device
        e = lambda *shape, dt=BF16: torch.empty(shape, dtype=dt, device=dev)  # noqa: E731
        Hq = self.Hs * r
        self.o = e(T, Hq, Dv)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self._state_out = None
        self.trains = backward
        if backward:
            self.dq, self.dk, self.dv = e(T, Hq, Dk), e(T, self.Hs, Dk), e(T, self.Hs, Dv)
        self._d_state_in = None
        dims = dict(T=self.max_seqlen, d=Dk, l=Dv, E=self.Hs, k=r, f=T, S=N)
        self.ws_bytes = max(M.moe_workspace_size(M.MOE_OP_LINATTN_FWD, **dims),
                            M.moe_workspace_size(M.MOE_OP_LINATTN_BWD, **dims) if backward else 0)
        self.ws = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=dev)
        self._state_first = None
        self.saved = None

    # buffers that only some callers want are made when first asked for
    @property
    def state_out(self):
        if self._state_out is None:
            self._state_out = torch.empty(self.N, self.Hs, self.Dk, self.Dv, device=self.o.device)
        return self._state_out

    @property
    def d_state_in(self):
        if self._d_state_in is None:
            self._d_state_in = torch.empty(self.N, self.Hs, self.Dk, self.Dv, device=self.o.device)
        return self._d_state_in

    def _rows(self, name, x, heads, width):
        """Checks a [T][heads][width] bf16 operand; returns the elements between tokens."""
        if x.shape != (self.T, heads, width) or x.dtype != BF16:
            raise ValueError(f"{name} is bf16 [{self.T}, {heads}, {width}], got {x.dtype} "
                             f"{list(x.shape)}")
        token, head, value = x.stride()
        if (value != 1 or (head != width and heads > 1)) and x.numel():
            raise ValueError(f"{name}: the heads of a token have to be contiguous")
        if token > 0x7FFFFFFF and self.T > 1:
            raise ValueError(f"{name}: tokens lie less than 2^31 values apart")
        return token if self.T > 1 else heads * width  # (the stride of a single token means nothing)

    def _operands(self, q, k, v):
        return (self._rows("q", q, self.Hs * self.r, self.Dk), self._rows("k", k, self.Hs, self.Dk),
                self._rows("v", v, self.Hs, self.Dv))

    def _state(self, name, x):
        if x is not None and (x.shape != (self.N, self.Hs, self.Dk, self.Dv)
                              or x.dtype != torch.float32 or not x.is_contiguous()):
            raise ValueError(f"{name} is fp32 {[self.N, self.Hs, self.Dk, self.Dv]}, contiguous")

    def _keep_first(self, state, stream):
        """A copy, made on the call's stream, of states that the call is about to overwrite."""
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            # (ExternalStream takes a handle of 0, the default stream, for none and makes a new one)
            stream = (torch.cuda.ExternalStream(int(stream), device=state.device) if int(stream) else
                      torch.cuda.default_stream(state.device))
        with torch.cuda.stream(stream):  # (None: the current one)
            if self._state_first is None:
                self._state_first = torch.empty_like(state)
            return self._state_first.copy_(state)

    def forward(self, q, k, v, cu_seqlens=None, state_in=None, want_state: bool = False,
                stream=None):
        """o [T, Hs * r, Dv] (bf16, this instance's buffer) for q [T, Hs * r, Dk],
        k [T, Hs, Dk], v [T, Hs, Dv]: slices of one projection's rows will do. cu_seqlens (int32
        [N + 1]): sequence n is the tokens cu_seqlens[n] .. cu_seqlens[n + 1] - 1; without it all
        have T / N tokens. With
        want_state, state_out holds each sequence's state after its last token. state_in may be
        state_out: the states are then updated in place, and backward still starts from those that
        were there before (this instance keeps a copy). What else was given to this call has to
        stay as it is until backward."""
        Hq = self.Hs * self.r
        ld = self._operands(q, k, v)
        if cu_seqlens is not None and (cu_seqlens.dtype != torch.int32 or cu_seqlens.shape != (self.N + 1,)
                                       or not cu_seqlens.is_contiguous()):
            raise ValueError(f"cu_seqlens is int32 [{self.N + 1}], contiguous")
        self._state("state_in", state_in)
        first = state_in
        if self.trains and want_state and state_in is not None and state_in.data_ptr() == self.state_out.data_ptr():
            first = self._keep_first(state_in, stream)
        if self.trains:
            self.saved = (q, k, v, cu_seqlens, first)
        M.moe_linattn_fwd(q, k, v, self.log_decay, cu_seqlens, state_in, self.N, self.T,
                          self.max_seqlen, self.Hs, self.r, self.Dk, self.Dv, *ld, Hq * self.Dv,
                          self.scale, self.o, self.state_out if want_state else None, self.ws,
                          self.ws_bytes, self.err, stream)
        return self.o

    def backward(self, dout, d_state_out=None, stream=None):
        """(dq, dk, dv) of the last forward call for dout = d loss / d o and d_state_out = d
        loss / d state_out; where the forward was given a state or d_state_out is given,
        d_state_in holds d loss / d state_in."""
        if not self.trains:
            raise ValueError("this instance was made without a backward")
        if self.saved is None:
            raise ValueError("backward needs a forward before it")
        q, k, v, cu_seqlens, state_in = self.saved
        Hs, Hq, Dk, Dv = self.Hs, self.Hs * self.r, self.Dk, self.Dv
        ld = [self._rows("dout", dout, Hq, Dv), *self._operands(q, k, v)]
        self._state("d_state_out", d_state_out)
        want = state_in is not None or d_state_out is not None
        M.moe_linattn_bwd(dout, q, k, v, self.log_decay, cu_seqlens, state_in, d_state_out, self.N,
                          self.T, self.max_seqlen, Hs, self.r, Dk, Dv, *ld, self.scale, self.dq,
                          self.dk, self.dv, Hq * Dk, Hs * Dk, Hs * Dv,
                          self.d_state_in if want else None, self.ws, self.ws_bytes, self.err,
                          stream)
        return self.dq, self.dk, self.dv

    def step(self, q, k, v, state, state_idx=None, stream=None):
        """One token for each of T rows: updates the state cache [slots, Hs, Dk, Dv] (fp32) in
        place at slot state_idx[row] (int32, negative for an empty row; default: the row) and
        returns o."""
        Hq = self.Hs * self.r
        ld = self._operands(q, k, v)
        slots = state.shape[0] if state.dim() else 0
        if (state.shape != (slots, self.Hs, self.Dk, self.Dv) or state.dtype != torch.float32
                or not state.is_contiguous()):
            raise ValueError(f"state is fp32 [slots, {self.Hs}, {self.Dk}, {self.Dv}], contiguous")
        if state_idx is not None and (state_idx.dtype != torch.int32 or state_idx.shape != (self.T,)
                                      or not state_idx.is_contiguous()):
            raise ValueError(f"state_idx is int32 [{self.T}], contiguous")
        M.moe_linattn_step(q, k, v, self.log_decay, state, state_idx, slots, self.T, self.Hs,
                           self.r, self.Dk, self.Dv, *ld, Hq * self.Dv, self.scale, self.o, self.err,
                           stream)
        return self.o
