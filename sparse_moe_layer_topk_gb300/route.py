"""Routing of tokens to experts from given logits, as libmoe calls: sigmoid or softmax scores, a bias for
balance that chooses only, groups of experts, top-k, renormalised weights; and the logits' gradient.

One instance holds its outputs for a fixed number of tokens T, so a call allocates nothing. What only the device
can see (a logit that is not a number, a bad id) sets bits of `err` (MOE_FLAG_*).
"""
from __future__ import annotations

import torch

from . import _lib as M

SCORES = {"sigmoid": M.MOE_SCORE_SIGMOID, "softmax": M.MOE_SCORE_SOFTMAX}
_DTYPES = {torch.float32: M.MOE_DTYPE_F32, torch.bfloat16: M.MOE_DTYPE_BF16}


class Router:
    def __init__(self, T: int, E: int, k: int, score: str = "sigmoid", groups: int = 1, group_k: int | None = None,
                 group_top: int = 2, renorm: bool = True, scale: float = 1.0, grad_dtype=torch.float32,
                 device="cuda"):
        """k of E experts (k <= 32, E <= 1024) for each of T tokens; of `groups` equal runs of experts only the
        group_k best stay (by the sum of their group_top = 1 or 2 largest values). grad_dtype: of d_logits."""
        if score not in SCORES:
            raise ValueError("score is 'sigmoid' or 'softmax'")
        if grad_dtype not in _DTYPES:
            raise ValueError("grad_dtype is float32 or bfloat16")
        group_k = groups if group_k is None else group_k
        if groups < 1 or E % groups or not 1 <= group_k <= groups or groups > 32:
            raise ValueError("groups divides E and is at most 32; group_k is 1 .. groups")
        if not 1 <= k <= min(32, group_k * (E // groups)):
            raise ValueError("k is at most 32 and at most the experts of the groups that stay")
        if group_top not in (1, 2):
            raise ValueError("group_top is 1 or 2")
        if not scale:
            raise ValueError("scale is not 0")
        self.T, self.E, self.k, self.score, self.renorm, self.scale = T, E, k, SCORES[score], bool(renorm), float(scale)
        self.groups, self.group_k, self.group_top = groups, group_k, group_top
        self.grad_dtype, self.device = grad_dtype, torch.device(device)
        e = lambda dt: torch.empty(T, k, dtype=dt, device=self.device)  # noqa: E731
        self.topk_idx, self.topk_w, self.topk_s = e(torch.int32), e(torch.float32), e(torch.float32)
        self.err = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._d_logits = None
        self.saved = None

    @property
    def d_logits(self):
        if self._d_logits is None:
            self._d_logits = torch.empty(self.T, self.E, dtype=self.grad_dtype, device=self.device)
        return self._d_logits

    def _check(self, name, x, shape, dtype=torch.float32):
        if tuple(x.shape) != shape or x.dtype != dtype or not x.is_contiguous():
            raise ValueError(f"{name} is {dtype} {list(shape)}, contiguous, got {x.dtype} {list(x.shape)}")

    def forward(self, logits, bias=None, stream=None):
        """(topk_idx, topk_w), this instance's buffers [T, k], for fp32 logits [T, E] and bias [E]; topk_s holds the scores.
        The logits have to stay as they are until backward where its scores are softmax and not renormalised (and to lie on 16
        bytes there, if E is a multiple of 4)."""
        self._check("logits", logits, (self.T, self.E))
        if bias is not None:
            self._check("bias", bias, (self.E,))
        self.saved = logits
        M.moe_route_scores(logits, bias, self.T, self.E, self.k, self.score, self.groups, self.group_k, self.group_top,
                           self.renorm, self.scale, self.topk_idx, self.topk_w, self.topk_s, self.err, stream)
        return self.topk_idx, self.topk_w

    def backward(self, d_w, slot_of=None, d_topk_w=None, stream=None, logits=None):
        """d_logits [T, E] of the last forward for d_w = d loss / d topk_w (fp32 [T, k]); with slot_of (int32 [T, k] of
        moe_permute) d_w is that of the permuted rows, and d_topk_w (fp32 [T, k]), if given, receives it in the tokens' order.
        logits: the forward's, if they are still as they were. Sigmoid scores next to one then keep their gradient: from the
        fp32 score alone 1 - s is off by 2^-23, and 0 for logits above 17."""
        if self.saved is None:
            raise ValueError("backward needs a forward before it")
        if slot_of is None:
            self._check("d_w", d_w, (self.T, self.k))
        else:
            self._check("slot_of", slot_of, (self.T, self.k), torch.int32)
            self._check("d_w", d_w, (self.T * self.k,))
        if d_topk_w is not None:
            self._check("d_topk_w", d_topk_w, (self.T, self.k))
        if logits is not None:
            self._check("logits", logits, (self.T, self.E))
        elif self.score == M.MOE_SCORE_SOFTMAX and not self.renorm:
            logits = self.saved
        M.moe_route_scores_bwd(d_w, slot_of, logits, self.topk_idx, self.topk_w, self.topk_s, self.T, self.E, self.k,
                               self.score, self.renorm, self.scale, self.d_logits, _DTYPES[self.grad_dtype], d_topk_w,
                               self.err, stream)
        return self.d_logits
