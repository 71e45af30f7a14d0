"""AdamW over many tensors in one launch (libmoe), states in 32 or 8 bits, with
the global gradient norm clipped on the device.

The tensors' addresses go into a plan when the optimizer is made: the gradients
are read from the same buffers at every step, as LatentMoELayer.grads and
LinearAttention's gradient buffers are. A step allocates nothing, waits for
nothing and counts itself on the device, so it can be captured in a CUDA graph.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib as M

BLOCK = 256  # values that share a scale in the 8-bit states
_DTYPES = {torch.float32: M.MOE_DTYPE_F32, torch.bfloat16: M.MOE_DTYPE_BF16}


class AdamW:
    def __init__(self, params, grads, lr: float, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay=0.0, max_norm: float = 0.0, state_bits: int = 32,
                 master: bool = False, seed: int = 0):
        """params, grads: lists of contiguous tensors (fp32 or bf16), one gradient for each.
        weight_decay: one number, or one for each tensor. max_norm > 0 clips the norm
        over all gradients. state_bits 8 holds m and sqrt(v) as E4M3 with one scale for 256
        values. master keeps an fp32 copy of each bf16 weight; without it bf16 weights are
        rounded stochastically (from seed, the step and the value's place)."""
        params, grads = list(params), list(grads)
        if len(params) != len(grads) or not params:
            raise ValueError("one gradient for each of at least one tensor")
        if state_bits not in (8, 32):
            raise ValueError("state_bits is 8 or 32")
        decays = list(weight_decay) if hasattr(weight_decay, "__len__") else [weight_decay] * len(params)
        if len(decays) != len(params):
            raise ValueError("one weight_decay for each tensor, or one number")
        for p, g in zip(params, grads):
            if p.dtype not in _DTYPES or g.dtype not in _DTYPES:
                raise ValueError("weights and gradients are fp32 or bf16")
            if p.numel() != g.numel() or p.device != g.device or not p.is_cuda:
                raise ValueError("a weight and its gradient have the same size and GPU")
            if p.device != params[0].device:
                raise ValueError("all tensors of an optimizer are on one GPU")
            if not (p.is_contiguous() and g.is_contiguous()):
                raise ValueError("weights and gradients are contiguous")
        held = sorted((p.data_ptr(), p.numel() * p.element_size()) for p in params if p.numel())
        if any(a + size > b for (a, size), (b, _) in zip(held, held[1:])):
            raise ValueError("two weights share memory: a step would update it twice")
        self.params, self.grads, self.state_bits = params, grads, state_bits
        self.lr, self.betas, self.eps, self.max_norm, self.seed = lr, betas, eps, max_norm, seed
        dev = params[0].device
        e8 = torch.float8_e4m3fn
        blocks = lambda p: -(-p.numel() // BLOCK)  # noqa: E731
        # (flat, like the values' order in memory; zeros in the 8-bit format are zero bytes)
        state = lambda p: (torch.zeros(p.numel(), device=dev) if state_bits == 32 else  # noqa: E731
                           torch.zeros(p.numel(), dtype=torch.uint8, device=dev).view(e8))
        self.m, self.v = [state(p) for p in params], [state(p) for p in params]
        scales = lambda: [torch.zeros(blocks(p), device=dev) for p in params]  # noqa: E731
        self.m_scale = scales() if state_bits == 8 else None
        self.v_scale = scales() if state_bits == 8 else None
        wide = lambda p: p.dtype == torch.bfloat16  # noqa: E731
        self.master = [p.detach().float().flatten() if wide(p) else None for p in params] if master else None
        self.ctl = torch.zeros(M.MOE_ADAMW_CTL_BYTES // 8, dtype=torch.int64, device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.lr_dev = None
        n = len(params)
        rows = (M.AdamWTensor * n)()
        ptr = lambda xs, i: None if xs is None or xs[i] is None or not xs[i].numel() else xs[i].data_ptr()  # noqa: E731
        for i in range(n):
            rows[i] = M.AdamWTensor(ptr(params, i), ptr(grads, i), ptr(self.m, i), ptr(self.v, i),
                                    ptr(self.m_scale, i), ptr(self.v_scale, i), ptr(self.master, i),
                                    params[i].numel(), decays[i], _DTYPES[params[i].dtype],
                                    _DTYPES[grads[i].dtype])
        plan = torch.empty(M.moe_workspace_size(M.MOE_OP_ADAMW_PLAN, T=n), dtype=torch.uint8)
        chunks = ctypes.c_longlong()
        M.moe_adamw_plan(rows, n, state_bits, plan.data_ptr(), plan.numel(), chunks)
        self.plan, self.chunks = plan.to(dev), chunks.value
        self.ws_bytes = M.moe_workspace_size(M.MOE_OP_ADAMW_STEP)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)

    def step(self, stream=None):
        M.moe_adamw_step(self.plan, len(self.params), self.chunks, self.state_bits, self.lr,
                         self.lr_dev, 1.0 - self.betas[0], 1.0 - self.betas[1], self.eps, self.max_norm,
                         self.seed, self.ctl, self.ws, self.ws_bytes, self.err, stream)

    def schedule_on_device(self, lr_dev):
        """From now on the learning rate is read from lr_dev (device fp32 [1]) at each step:
        a captured step follows it."""
        if lr_dev is not None and (lr_dev.dtype != torch.float32 or not lr_dev.is_cuda or lr_dev.numel() != 1):
            raise ValueError("lr_dev is a device fp32 tensor of one value")
        self.lr_dev = lr_dev

    @property
    def step_count(self):
        """Steps taken (int64, device)."""
        return self.ctl[0]

    @property
    def grad_norm(self):
        """The gradient norm of the last clipped step (fp32, device)."""
        return self.ctl.view(torch.float32)[2]

    def state_dict(self):
        copy = lambda xs: None if xs is None else [None if x is None else x.clone() for x in xs]  # noqa: E731
        return dict(step=int(self.step_count), m=copy(self.m), v=copy(self.v), m_scale=copy(self.m_scale),
                    v_scale=copy(self.v_scale), master=copy(self.master), seed=self.seed)

    def load_state(self, step, m, v, m_scale=None, v_scale=None, master=None, seed=None):
        """Takes over a state_dict's values (`load_state(**d)`); without a master copy given, it is
        made from the weights. Nothing is taken over where an entry is missing or does not fit.
        Without a seed the rounding goes on with this optimizer's own."""
        pairs = []
        for name, given in dict(m=m, v=v, m_scale=m_scale, v_scale=v_scale, master=master).items():
            mine = getattr(self, name)
            if mine is None:
                continue
            if given is None:
                if name != "master":
                    raise ValueError("8-bit states come with their scales")
                given = [None if x is None else p.detach().float().flatten() for x, p in zip(mine, self.params)]
            if len(given) != len(mine):
                raise ValueError(f"{name}: one entry for each of {len(mine)} tensors, got {len(given)}")
            for dst, src in zip(mine, given):
                if dst is None:
                    continue
                if src is None or dst.dtype != src.dtype or dst.numel() != src.numel():
                    raise ValueError(f"{name}: the state has another type or size")
                pairs.append((dst, src))
        self.ctl.zero_()
        self.ctl[0] = step
        if seed is not None:
            self.seed = seed
        for dst, src in pairs:
            dst.copy_(src.flatten())
