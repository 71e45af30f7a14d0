"""Root-mean-square norm of x + residual, as libmoe calls: output in bf16 or in 8 bits with scales, and its
gradients.

    u = x + residual;  y = u * weight / sqrt(mean(u^2) + eps)

One instance holds its outputs for a fixed number of rows T, so a call allocates nothing.
"""
from __future__ import annotations

import torch

from . import _lib as M

BF16 = torch.bfloat16
_DTYPES = {torch.float32: M.MOE_DTYPE_F32, BF16: M.MOE_DTYPE_BF16}


class RMSNorm:
    def __init__(self, weight, T: int, eps: float = 1e-6, residual_dtype=None, out: str = "bf16", block: int = 0,
                 backward: bool = True):
        """weight: fp32 [d] (d a multiple of 8 up to 16384). residual_dtype: type of the residual stream (float32 or bfloat16), None
        where there is none. out "fp8": y is E4M3 with one scale (largest magnitude / 448) for each `block` = 64, 128 or
        d columns (default 128) of a row."""
        if weight.dtype != torch.float32 or weight.dim() != 1 or not weight.is_contiguous():
            raise ValueError("weight is an fp32 vector, contiguous")
        if residual_dtype is not None and residual_dtype not in _DTYPES:
            raise ValueError("residual_dtype is float32, bfloat16 or None")
        if out not in ("bf16", "fp8"):
            raise ValueError("out is 'bf16' or 'fp8'")
        if not eps > 0:
            raise ValueError("eps is above 0")
        self.weight, self.T, self.d, self.eps = weight, T, weight.numel(), eps
        self.residual_dtype, self.fp8, self.trains = residual_dtype, out == "fp8", backward
        self.block = block or 128
        dev = weight.device
        d = self.d
        e = lambda dt, *shape: torch.empty(shape, dtype=dt, device=dev)  # noqa: E731
        self.sum = e(residual_dtype, T, d) if residual_dtype is not None else None
        if self.fp8:
            if self.block not in (64, 128, d):
                raise ValueError("block is 64, 128 or d")
            self.y = e(torch.float8_e4m3fn, T, d)
            self.scale = e(torch.float32, T, -(-d // self.block))
        else:
            self.y, self.scale = e(BF16, T, d), None
        self.saved = None
        if backward:
            self.dx, self.dw = e(BF16, T, d), e(torch.float32, d)
            self._d_residual = e(torch.float32, T, d) if residual_dtype == torch.float32 else None
            self.ws_bytes = M.moe_workspace_size(M.MOE_OP_RMSNORM_BWD, T=T, d=d)
            self.ws = e(torch.uint8, max(self.ws_bytes, 256))

    @property
    def d_residual(self):
        """The residual's gradient, in its type (with a bf16 residual the same as dx)."""
        return self.dx if self._d_residual is None else self._d_residual

    def _rows(self, name, x, dtype, strided=False):
        if x.shape != (self.T, self.d) or x.dtype is not dtype:
            raise ValueError(f"{name} is {dtype} [{self.T}, {self.d}], got {x.dtype} {list(x.shape)}")
        if not strided:
            if not x.is_contiguous():
                raise ValueError(f"{name} is contiguous")
            return self.d
        if x.stride(1) != 1 and x.numel():
            raise ValueError(f"{name}: the columns of a row have to be contiguous")
        if x.stride(0) > 0x7FFFFFFF and self.T > 1:
            raise ValueError(f"{name}: rows lie less than 2^31 values apart")
        return x.stride(0) if self.T > 1 else self.d  # (the stride of a single row means nothing)

    def forward(self, x, residual=None, in_place: bool = False, stream=None):
        """y [T, d] (this instance's buffer; in 8 bits with `scale` beside it) for bf16 x [T, d], whose rows may be slices of wider
        ones. residual [T, d]: `sum` receives x + residual, or residual itself does with in_place. What backward reads (the sum,
        or x without a residual) has to stay as it is until then."""
        ldx = self._rows("x", x, BF16, strided=True)
        if (residual is None) != (self.residual_dtype is None):
            raise ValueError("a residual is given exactly where residual_dtype is")
        total = None
        if residual is not None:
            self._rows("residual", residual, self.residual_dtype)
            total = residual if in_place else self.sum
        M.moe_rmsnorm_fwd(x, residual, self.weight, self.T, self.d, ldx, _DTYPES[self.residual_dtype or BF16], self.eps,
                          total, self.y, M.MOE_DTYPE_E4M3 if self.fp8 else M.MOE_DTYPE_BF16, self.scale, self.block,
                          stream)
        self.saved = (x, ldx) if total is None else (total, self.d)
        return self.y

    def backward(self, dy, d_sum=None, stream=None):
        """dx [T, d] (bf16) of the last forward for dy = d loss / d y (bf16) and d_sum = d loss / d sum (the residual's type); dw holds
        the weight's gradient, d_residual the residual's."""
        if not self.trains:
            raise ValueError("this instance was made without a backward")
        if self.saved is None:
            raise ValueError("backward needs a forward before it")
        self._rows("dy", dy, BF16)
        if d_sum is not None:
            if self.residual_dtype is None:
                raise ValueError("without a residual there is no sum")
            self._rows("d_sum", d_sum, self.residual_dtype)
        u, ldu = self.saved
        M.moe_rmsnorm_bwd(dy, u, self.weight, d_sum, self.T, self.d, ldu, _DTYPES[self.residual_dtype or BF16], self.eps,
                          self.dx, self._d_residual, self.dw, self.ws, self.ws_bytes, stream)
        return self.dx
