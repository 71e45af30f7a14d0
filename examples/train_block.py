"""A block's training step and its decoding through libmoe: a sequence mixer, the LatentMoE
layer after it, and AdamW over all weights. The mixer is linear attention with a decay for each head,

    u   = x + LinearAttention(x W_qkv) W_o
    out = u + LatentMoE(u)

or, with --mixer scan, a short convolution and the selective scan, with norms before both halves and experts
chosen in groups:

    v, z = norm(x) W_in;  w = conv(v);  dt, B, C = w W_x;  u = x + scan(w, dt W_dt, B, C, z) W_out
    out  = u + LatentMoE(norm(u))

    python examples/train_block.py [--steps 20] [--tokens 256] [--mixer attention]

The data is synthetic: packed sequences of random tokens, each to be answered with the
token before it, which only the mixer can carry over. PyTorch provides memory, streams,
the residual sums and the loss.
"""
import argparse
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from sparse_moe_layer_topk_gb300 import _lib as M  # noqa: E402
from sparse_moe_layer_topk_gb300 import inputs as I  # noqa: E402
from sparse_moe_layer_topk_gb300.layer import LatentMoELayer, weights_to_device  # noqa: E402
from sparse_moe_layer_topk_gb300.linattn import LinearAttention  # noqa: E402
from sparse_moe_layer_topk_gb300.norm import RMSNorm  # noqa: E402
from sparse_moe_layer_topk_gb300.optim import AdamW  # noqa: E402
from sparse_moe_layer_topk_gb300.scan import CausalConv, SelectiveScan  # noqa: E402

BF16 = torch.bfloat16
HS, R, DK, DV = 2, 2, 64, 128  # state heads, query heads for each, widths


def _layer_inputs(seed):
    return I.make_layer_inputs(dataclasses.replace(I.CONFIGS[0], seed=seed))


class Weights:
    """A block's weights on the device: the mixer's two projections and the layer's."""

    def __init__(self, seed=0):
        inp = _layer_inputs(seed)
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


class ScanWeights:
    """A block's weights on the device, its mixer the convolution and the scan of INNER channels."""
    INNER, STATES, RANK, TAPS = 512, 16, 64, 4

    def __init__(self, seed=0):
        inp = _layer_inputs(seed)
        self.cfg = inp["cfg"]
        d, D, S, R = self.cfg.d, self.INNER, self.STATES, self.RANK
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: (torch.randn(*s, generator=g) * s[0] ** -0.5).to(BF16).cuda()  # noqa: E731
        self.W_in, self.W_x, self.W_dt, self.W_out = n(d, 2 * D), n(D, 2 * R), n(R, D), n(D, d)  # (W_x: R + 2 S columns used)
        self.norm = torch.ones(d, device="cuda")
        self.conv_w, self.conv_b = (torch.randn(D, self.TAPS, generator=g) * 0.5).cuda(), torch.zeros(D, device="cuda")
        self.log_A = torch.log(torch.arange(1.0, S + 1)).repeat(D, 1).cuda()
        dt = torch.exp(torch.rand(D, generator=g) * 4.6 - 6.9)  # time steps from 0.001 to 0.1
        self.dt_bias, self.skip = (dt + torch.log(-torch.expm1(-dt))).cuda(), torch.ones(D, device="cuda")
        self.moe = weights_to_device({**inp, "norm": torch.ones(d)})


class ScanBlock:
    """Forward and backward over T packed tokens of N sequences."""
    MIXER = ("W_in", "W_x", "W_dt", "W_out", "norm", "conv_w", "conv_b", "log_A", "dt_bias", "skip")

    def __init__(self, w: ScanWeights, T: int, N: int, max_seqlen: int, backward=True):
        self.w, self.T, self.d, D, S, R = w, T, w.cfg.d, w.INNER, w.STATES, w.RANK
        self.A = -torch.exp(w.log_A)
        self.norm = RMSNorm(w.norm, T, backward=backward)
        self.conv = CausalConv(w.conv_w, w.conv_b, T, N=N, backward=backward)
        self.mixer = SelectiveScan(self.A, T, w.skip, w.dt_bias, N=N, max_seqlen=max_seqlen, backward=backward)
        self.moe = LatentMoELayer(w.moe, T, w.cfg.k, residual_dtype=BF16, router=dict(groups=4, group_k=2))
        e = lambda *s: torch.empty(s, dtype=BF16, device="cuda")  # noqa: E731
        self.vz, self.bc, self.delta, self.att = e(T, 2 * D), e(T, 2 * R), e(T, D), e(T, self.d)
        if backward:
            self.d_scan, self.d_rank, self.d_bc, self.d_w, self.d_norm = e(T, D), e(T, R), torch.zeros(T, 2 * R, dtype=BF16, device="cuda"), e(T, D), e(T, self.d)
            f = lambda x: torch.empty(x.shape, device="cuda")  # noqa: E731
            self.grads = {n: f(getattr(w, n)) for n in ("W_in", "W_x", "W_dt", "W_out", "log_A")}
            self.grads |= dict(norm=self.norm.dw, conv_w=self.conv.dw, conv_b=self.conv.db, dt_bias=self.mixer.d_dt_bias, skip=self.mixer.dskip)

    def _inner(self, x):
        """The two halves of the projection: what the convolution reads, and the gate."""
        w, D = self.w, self.w.INNER
        torch.exp(w.log_A, out=self.A).neg_()
        M.moe_latent_proj(self.norm.forward(x), w.W_in, self.T, self.d, 2 * D, self.vz)
        return self.vz[:, :D], self.vz[:, D:]

    def _operands(self, v):
        """What the scan takes of the convolution's output."""
        w, D, R, S = self.w, self.w.INNER, self.w.RANK, self.w.STATES
        M.moe_latent_proj(v, w.W_x, self.T, D, 2 * R, self.bc)
        self.rank = self.bc[:, :R].contiguous()
        M.moe_latent_proj(self.rank, w.W_dt, self.T, R, D, self.delta)
        return v, self.delta, self.bc[:, R:R + S].unflatten(1, (1, S)), self.bc[:, R + S:R + 2 * S].unflatten(1, (1, S))

    def _rest(self, x, y):
        M.moe_latent_proj(y, self.w.W_out, self.T, self.w.INNER, self.d, self.att)
        out = self.moe.forward(self.att, residual=x)
        return self.moe.norm.sum + out

    def forward(self, x, cu_seqlens, want_state=False):
        v, z = self._inner(x)
        self.x = x
        return self._rest(x, self.mixer.forward(*self._operands(self.conv.forward(v, cu_seqlens, want_state=want_state)), z, cu_seqlens,
                                                want_state=want_state))

    def decode(self, x, conv_state, scan_state, state_idx):
        """One token for each of T rows; both caches are updated in place at state_idx."""
        v, z = self._inner(x)
        return self._rest(x, self.mixer.step(*self._operands(self.conv.step(v, conv_state, state_idx)), z, scan_state, state_idx))

    def backward(self, dout):
        w, wd, g, T, d, D, R, S = self.w, M.MOE_DTYPE_F32, self.grads, self.T, self.d, self.w.INNER, self.w.RANK, self.w.STATES
        d_att = self.moe.backward(dout, d_sum=dout)  # (also the residual's gradient)
        M.moe_latent_proj_bwd(d_att, self.mixer.y, w.W_out, T, D, d, self.d_scan, g["W_out"], wd)
        du, ddelta, dB, dC, dz = self.mixer.backward(self.d_scan)
        M.moe_latent_proj_bwd(ddelta, self.rank, w.W_dt, T, R, D, self.d_rank, g["W_dt"], wd)
        self.d_bc[:, :R], self.d_bc[:, R:R + S], self.d_bc[:, R + S:R + 2 * S] = self.d_rank, dB.flatten(1), dC.flatten(1)
        M.moe_latent_proj_bwd(self.d_bc, self.conv.y, w.W_x, T, D, 2 * R, self.d_w, g["W_x"], wd)
        dvz = torch.cat([self.conv.backward(du + self.d_w), dz], 1)
        M.moe_latent_proj_bwd(dvz, self.norm.y, w.W_in, T, d, 2 * D, self.d_norm, g["W_in"], wd)
        torch.mul(self.mixer.dA, self.A, out=g["log_A"])
        return d_att + self.norm.backward(self.d_norm)

    def parameters(self):
        """(weights, gradients), matched by name."""
        names = list(self.moe.grads)
        return ([getattr(self.w, n) for n in self.MIXER] + [self.w.moe[n] for n in names],
                [self.grads[n] for n in self.MIXER] + [self.moe.grads[n] for n in names])


def train(lens, steps, lr=2e-3, seed=0, state_bits=8, mixer="attention"):
    """Loss of each step, and the block."""
    T, cu = sum(lens), torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    block = (Block(Weights(seed), T, len(lens), max(lens)) if mixer == "attention" else
             ScanBlock(ScanWeights(seed), T, len(lens), max(lens)))
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


def decode_scan(w, prompts, slots=None):
    """decode() for the block with the scan."""
    lens = [p.shape[0] - 1 for p in prompts]
    N = len(prompts)
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    first = ScanBlock(w, sum(lens), N, max(lens), backward=False)
    first.forward(torch.cat([p[:-1] for p in prompts]), cu, want_state=True)
    idx = torch.arange(N - 1, -1, -1, dtype=torch.int32, device="cuda")
    caches = []
    for state in (first.conv.state_out, first.mixer.state_out):
        caches.append(torch.zeros(slots or N, *state.shape[1:], dtype=state.dtype, device="cuda"))
        caches[-1][idx.long()] = state
    one = ScanBlock(w, N, N, 1, backward=False)
    return one.decode(torch.stack([p[-1] for p in prompts]), *caches, idx), one


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--mixer", choices=["attention", "scan"], default="attention")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=256)
    args = ap.parse_args()
    a = max(args.tokens * 2 // 5, 1)
    losses, block = train([a, max(args.tokens - a, 1)], args.steps, mixer=args.mixer)
    print("loss " + " ".join(f"{v:.4f}" for v in losses))
    out, _ = (decode if args.mixer == "attention" else decode_scan)(block.w, [block.x[:a], block.x[a:]])
    print(f"decoded {out.shape[0]} tokens of width {out.shape[1]}")


if __name__ == "__main__":
    main()
