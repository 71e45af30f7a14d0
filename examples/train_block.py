"""A block's training step and its decoding through libmoe: the sequence mixer
(linear attention with a decay for each head), the LatentMoE layer after it, and AdamW
over all weights.

    u   = x + LinearAttention(x W_qkv) W_o
    out = u + LatentMoE(u)

    python examples/train_block.py [--steps 20] [--tokens 256]

The data is synthetic: packed sequences of random tokens, each to be answered with the
token before it, which only the mixer can carry over. PyTorch provides memory, streams,
the residual sums and the loss.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from sparse_moe_layer_topk_gb300 import _lib as M  # noqa: E402
from sparse_moe_layer_topk_gb300 import inputs as I  # noqa: E402
from sparse_moe_layer_topk_gb300.layer import LatentMoELayer, weights_to_device  # noqa: E402
from sparse_moe_layer_topk_gb300.linattn import LinearAttention  # noqa: E402
from sparse_moe_layer_topk_gb300.optim import AdamW  # noqa: E402

BF16 = torch.bfloat16
HS, R, DK, DV = 2, 2, 64, 128  # state heads, query heads for each, widths


class Weights:
    """A block's weights on the device: the mixer's two projections and the layer's."""

    def __init__(self, seed=0):
        inp = I.make_layer_inputs(seed)
        self.cfg = inp["cfg"]
        d = self.cfg.d
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: (torch.randn(*s, generator=g) * s[0] ** -0.5).to(BF16).cuda()  # noqa: E731
        self.W_qkv = n(d, HS * (R * DK + DK + DV))
        self.W_o = n(HS * R * DV, d)
        self.log_decay = torch.tensor([-0.5 * 4.0 ** -h for h in range(HS)], device="cuda")
        self.moe = weights_to_device(inp)


class Block:
    """Forward and backward over T packed tokens of N sequences."""

    def __init__(self, w: Weights, T: int, N: int, max_seqlen: int, backward=True):
        self.w, self.T, self.d = w, T, w.cfg.d
        self.mixer = LinearAttention(w.log_decay, T, DK, DV, r=R, N=N, max_seqlen=max_seqlen, backward=backward)
        self.moe = LatentMoELayer(w.moe, T, w.cfg.k)
        e = lambda *s: torch.empty(s, dtype=BF16, device="cuda")  # noqa: E731
        self.qkv, self.att = e(T, w.W_qkv.shape[1]), e(T, self.d)
        if backward:
            self.do, self.dx = e(T, HS * R, DV), e(T, self.d)
            self.grads = {"W_qkv": torch.empty(w.W_qkv.shape, device="cuda"),
                          "W_o": torch.empty(w.W_o.shape, device="cuda")}

    def _heads(self, x):
        """q, k and v: slices of the projection's rows."""
        M.moe_latent_proj(x, self.w.W_qkv, self.T, self.d, self.qkv.shape[1], self.qkv)
        q, k, v = self.qkv.split([HS * R * DK, HS * DK, HS * DV], dim=1)
        return q.unflatten(1, (HS * R, DK)), k.unflatten(1, (HS, DK)), v.unflatten(1, (HS, DV))

    def _rest(self, x, o):
        M.moe_latent_proj(o, self.w.W_o, self.T, HS * R * DV, self.d, self.att)
        self.u = x + self.att
        return self.u + self.moe.forward(self.u)

    def forward(self, x, cu_seqlens, want_state=False):
        self.x = x
        return self._rest(x, self.mixer.forward(*self._heads(x), cu_seqlens, want_state=want_state))

    def decode(self, x, state, state_idx):
        """One token for each of T rows; the states at state_idx are updated in place."""
        return self._rest(x, self.mixer.step(*self._heads(x), state, state_idx))

    def backward(self, dout):
        w, wd = self.w, M.MOE_DTYPE_F32
        du = dout + self.moe.backward(dout)
        M.moe_latent_proj_bwd(du, self.mixer.o, w.W_o, self.T, HS * R * DV, self.d, self.do, self.grads["W_o"], wd)
        dqkv = torch.cat([g.flatten(1) for g in self.mixer.backward(self.do)], dim=1)
        M.moe_latent_proj_bwd(dqkv, self.x, w.W_qkv, self.T, self.d, dqkv.shape[1], self.dx, self.grads["W_qkv"], wd)
        return du + self.dx

    def parameters(self):
        """(weights, gradients), matched by name."""
        names = list(self.moe.grads)
        return ([self.w.W_qkv, self.w.W_o] + [self.w.moe[n] for n in names],
                [self.grads["W_qkv"], self.grads["W_o"]] + [self.moe.grads[n] for n in names])


def train(lens, steps, lr=2e-3, seed=0, state_bits=8):
    """Loss of each step, and the block."""
    T, cu = sum(lens), torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    block = Block(Weights(seed), T, len(lens), max(lens))
    params, grads = block.parameters()
    opt = AdamW(params, grads, lr, max_norm=1.0, weight_decay=0.01, state_bits=state_bits, master=True)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, block.d, generator=g).to(BF16).cuda()
    target = torch.cat([torch.cat([torch.zeros_like(s[:1]), s[:-1]]) for s in x.split(lens)]).float()
    losses = []
    for _ in range(steps):
        diff = block.forward(x, cu).float() - target
        losses.append(diff.square().mean())
        block.backward((diff * (2.0 / diff.numel())).to(BF16))
        opt.step()
    torch.cuda.synchronize()
    if int(block.mixer.err) | int(block.moe.err) | int(opt.err):
        raise RuntimeError("a call met an index or a value out of its range")
    return [float(v) for v in losses], block


def decode(w, prompts, slots=None):
    """The answers to each prompt's last token: the prompt before it in one pass, then one
    step from the states that it left in a cache of `slots` rows."""
    lens = [p.shape[0] - 1 for p in prompts]
    N = len(prompts)
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    first = Block(w, sum(lens), N, max(lens), backward=False)
    first.forward(torch.cat([p[:-1] for p in prompts]), cu, want_state=True)
    cache = torch.zeros(slots or N, HS, DK, DV, device="cuda")
    idx = torch.arange(N - 1, -1, -1, dtype=torch.int32, device="cuda")  # (any free slots)
    cache[idx.long()] = first.mixer.state_out
    one = Block(w, N, N, 1, backward=False)
    return one.decode(torch.stack([p[-1] for p in prompts]), cache, idx), one


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=256)
    args = ap.parse_args()
    a = max(args.tokens * 2 // 5, 1)
    losses, block = train([a, max(args.tokens - a, 1)], args.steps)
    print("loss " + " ".join(f"{v:.4f}" for v in losses))
    out, _ = decode(block.w, [block.x[:a], block.x[a:]])
    print(f"decoded {out.shape[0]} tokens of width {out.shape[1]}")


if __name__ == "__main__":
    main()
