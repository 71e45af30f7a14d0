"""Norm, convolution, scan, routing in groups and the experts together, as the layer and the example block run them: against
PyTorch's autograd in 64 bits of the same formulas.

bf16 activations and gradients are rounded once between two operators (2^-9 rms each, a dozen of them one behind the other): relative
norms within the layer's own bound, 1e-2, twice that for gradients that pass the whole block."""
import importlib.util
import pathlib

import numpy as np
import pytest
import torch
import torch.nn.functional as F

from sparse_moe_layer_topk_gb300 import inputs as I
from gpu_util import REL_FRO, f64, need_gpu

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.fixture(scope="module")
def example():
    path = pathlib.Path(__file__).resolve().parent.parent / "examples" / "train_block.py"
    spec = importlib.util.spec_from_file_location("train_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _off(got, want, tol, name=""):
    got, want = f64(got), f64(want)
    rel = np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-300)
    assert np.isfinite(got).all() and rel <= tol, f"{name}: {rel:.2e}"


def _leaf(w):
    return {n: t.detach().cuda().double().requires_grad_() for n, t in w.items() if t is not None}


def _norm(u, w, eps=1e-6):
    return u * torch.rsqrt(u.square().mean(-1, keepdim=True) + eps) * w


def _experts(n, w, idx, score="sigmoid", renorm=True, scale=1.0):
    """The layer behind its norm, for the ids that were chosen."""
    l = n @ w["Wr"]
    s = (torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, -1)).gather(1, idx)
    rw = scale * (s / s.sum(1, keepdim=True) if renorm else s)
    z = n @ w["W_dn"]

    def swiglu(z, W13, W2):
        g, u = (z @ W13).chunk(2, -1)
        return (F.silu(g) * u) @ W2
    y = sum(swiglu(z, w["W13_sh"][i], w["W2_sh"][i]) for i in range(w["W13_sh"].shape[0]))
    every = torch.stack([swiglu(z, w["W13"][e], w["W2"][e]) for e in range(w["W13"].shape[0])], 1)
    y = y + (rw[..., None] * every.gather(1, idx[..., None].expand(-1, -1, z.shape[1]))).sum(1)
    return y @ w["W_up"]


ROUTERS = [None, {}, dict(groups=4, group_k=2, scale=2.5), dict(score="softmax", renorm=False, scale=3.0), dict(score="softmax", groups=2, group_k=1)]


@pytest.mark.parametrize("router", ROUTERS, ids=str)
@pytest.mark.parametrize("res", [None, BF, F32])
def test_layer(router, res):
    from sparse_moe_layer_topk_gb300.layer import LatentMoELayer, weights_to_device
    inp = I.make_layer_inputs(0)
    cfg = inp["cfg"]
    g = torch.Generator().manual_seed(4)
    inp["norm"] = 1 + 0.2 * torch.randn(cfg.d, generator=g)
    w = weights_to_device(inp)
    layer = LatentMoELayer(w, cfg.T, cfg.k, residual_dtype=res, router=router)
    r = None if res is None else torch.randn(cfg.T, cfg.d, generator=g).to(res)
    ds = None if res is None else torch.randn(cfg.T, cfg.d, generator=g).to(res)
    out = layer.forward(inp["x"].cuda(), residual=None if r is None else r.cuda())
    dx = layer.backward(inp["g"].cuda(), d_sum=None if ds is None else ds.cuda())
    assert int(layer.err) == 0
    ref = _leaf(w)
    ref.pop("bias", None)
    x = inp["x"].cuda().double().requires_grad_()
    u = x + (0 if r is None else r.cuda().double())
    kw = {k: v for k, v in (router or {}).items() if k in ("score", "renorm", "scale")}
    want = _experts(_norm(u, ref["norm"]), ref, layer.topk_idx.long(), **kw)
    loss = (want * inp["g"].cuda().double()).sum() + (0 if ds is None else (u * ds.cuda().double()).sum())
    loss.backward()
    _off(out, want.detach(), REL_FRO, "out")
    _off(dx, x.grad, 2 * REL_FRO, "dx")
    if res is not None:
        _off(layer.norm.d_residual, x.grad, 2 * REL_FRO, "d_residual")
    for n in layer.grads:
        _off(layer.grads[n], ref[n].grad, 2 * REL_FRO, n)


def test_the_plain_router_and_the_sigmoid_one_agree():
    from sparse_moe_layer_topk_gb300.layer import LatentMoELayer, weights_to_device
    inp = I.make_layer_inputs(0)
    cfg, w = inp["cfg"], weights_to_device(inp)
    a, b = LatentMoELayer(w, cfg.T, cfg.k), LatentMoELayer(w, cfg.T, cfg.k, router={})
    oa, ob = a.forward(inp["x"].cuda()), b.forward(inp["x"].cuda())
    assert torch.equal(a.topk_idx, b.topk_idx)
    np.testing.assert_allclose(f64(a.topk_w), f64(b.topk_w), rtol=1e-6)
    _off(ob, oa, 1e-3)
    _off(b.backward(inp["g"].cuda()), a.backward(inp["g"].cuda()), 1e-3)


def test_layer_in_a_graph_and_from_the_host():
    from sparse_moe_layer_topk_gb300.layer import LatentMoELayer, weights_to_device
    inp = I.make_layer_inputs(0)
    inp["norm"] = torch.ones(inp["cfg"].d)
    cfg, w = inp["cfg"], weights_to_device(inp)
    kw = dict(router=dict(groups=2, group_k=1))
    layer = LatentMoELayer(w, cfg.T, cfg.k, **kw)
    x, g = inp["x"].cuda(), inp["g"].cuda()
    want = layer.step(x, g).clone()
    xs, gs = [inp["x"].pin_memory()] * 3, [inp["g"].pin_memory()] * 3
    back = [torch.empty_like(inp["x"]).pin_memory() for _ in range(3)]
    layer.steps_from_host(xs, gs, back)
    torch.cuda.synchronize()
    for t in back:
        assert torch.equal(t, want.cpu())
    graph = layer.capture_step(x, g)
    layer.dx.zero_()
    graph.replay()
    assert torch.equal(layer.dx, want)


def _scan_reference(w, x, cu, idx):
    """The example's block in 64 bits; `idx` the experts that were chosen."""
    D, S, R = w["W_out"].shape[0], w["log_A"].shape[1], w["W_dt"].shape[0]
    v, z = (_norm(x, w["norm"]) @ w["W_in"]).chunk(2, 1)
    conv, y = [], []
    for a, b in zip(cu[:-1], cu[1:]):
        ext = F.pad(v[a:b], (0, 0, w["conv_w"].shape[1] - 1, 0))
        conv.append(F.silu((ext.unfold(0, w["conv_w"].shape[1], 1) * w["conv_w"]).sum(-1) + w["conv_b"]))
    c = torch.cat(conv)
    p = c @ w["W_x"]
    dt = F.softplus(p[:, :R] @ w["W_dt"] + w["dt_bias"])
    B, C, A = p[:, R:R + S], p[:, R + S:R + 2 * S], -torch.exp(w["log_A"])
    for a, b in zip(cu[:-1], cu[1:]):
        h = torch.zeros(D, S, dtype=F64, device=x.device)
        for t in range(a, b):
            h = torch.exp(dt[t][:, None] * A) * h + (dt[t] * c[t])[:, None] * B[t]
            y.append(h @ C[t] + w["skip"] * c[t])
    u = x + (torch.stack(y) * F.silu(z)) @ w["W_out"]
    return u + _experts(_norm(u, w["moe_norm"]), w, idx)


def test_the_example_blocks_gradients(example):
    lens = [23, 1, 40]
    T, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)]).tolist()
    w = example.ScanWeights(1)
    block = example.ScanBlock(w, T, len(lens), max(lens))
    g = torch.Generator().manual_seed(2)
    x, dout = (torch.randn(T, w.cfg.d, generator=g).to(BF) for _ in range(2))
    out = block.forward(x.cuda(), torch.tensor(cu, dtype=torch.int32, device="cuda"))
    dx = block.backward(dout.cuda())
    ref = _leaf({**{n: getattr(w, n) for n in block.MIXER}, **{n: t for n, t in w.moe.items() if n not in ("bias", "norm")}, "moe_norm": w.moe["norm"]})
    xr = x.cuda().double().requires_grad_()
    want = _scan_reference(ref, xr, cu, block.moe.topk_idx.long())
    (want * dout.cuda().double()).sum().backward()
    _off(out, want.detach(), REL_FRO, "out")
    _off(dx, xr.grad, 2 * REL_FRO, "dx")
    for n in block.MIXER:
        _off(block.grads[n], ref[n].grad, 3 * REL_FRO, n)
    _off(block.moe.grads["norm"], ref["moe_norm"].grad, 3 * REL_FRO, "moe norm")
    assert int(block.mixer.err) | int(block.conv.err) | int(block.moe.err) == 0


@pytest.mark.parametrize("state_bits", [8, 32])
def test_the_example_trains(example, state_bits):
    losses, _ = example.train([100, 1, 155], 6, state_bits=state_bits, mixer="scan")
    assert np.isfinite(losses).all()


def test_the_example_decodes_as_the_packed_pass(example):
    lens = [2, 130, 33]
    w = example.ScanWeights(2)
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randn(n, w.cfg.d, generator=g).to(BF).cuda() for n in lens]
    _, one = example.decode_scan(w, prompts, slots=5)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    block = example.ScanBlock(w, sum(lens), 3, max(lens), backward=False)
    block.forward(torch.cat(prompts), cu)
    _off(one.mixer.y, block.mixer.y[(cu[1:] - 1).long()], 2 * REL_FRO)
    assert int(one.mixer.err) == 0 and int(block.mixer.err) == 0


@pytest.mark.parametrize("router", [None, dict(groups=2, group_k=1)], ids=str)
@pytest.mark.parametrize("res", [BF, F32])
@pytest.mark.parametrize("given", [False, True])
def test_steps_with_a_residual(router, res, given):
    """A step, its graph, its halves and the steps from the host give what forward and backward give one after the other."""
    from sparse_moe_layer_topk_gb300.layer import LatentMoELayer, weights_to_device
    inp = I.make_layer_inputs(0)
    gen = torch.Generator().manual_seed(6)
    inp["norm"] = 1 + 0.2 * torch.randn(inp["cfg"].d, generator=gen)
    cfg, w, n = inp["cfg"], weights_to_device(inp), 3
    make = lambda: LatentMoELayer(w, cfg.T, cfg.k, residual_dtype=res, router=router)  # noqa: E731
    rows = lambda dt: [torch.randn(cfg.T, cfg.d, generator=gen).to(dt).pin_memory() for _ in range(n)]  # noqa: E731
    xs, gs, rs, ds = rows(BF), rows(BF), rows(res), rows(res)
    ref, want = make(), []
    for i in range(n):
        ref.forward(xs[i].cuda(), residual=rs[i].cuda())
        dx = ref.backward(gs[i].cuda(), d_sum=ds[i].cuda() if given else None)
        want.append([t.clone() for t in (dx, ref.norm.d_residual, ref.out, ref.norm.sum, *ref.grads.values())])

    def same(layer, i):
        got = (layer.dx, layer.norm.d_residual, layer.out, layer.norm.sum, *layer.grads.values())
        assert all(torch.equal(a, b) for a, b in zip(got, want[i])) and int(layer.err) == 0

    layer = make()
    x, g, r = (v[0].cuda() for v in (xs, gs, rs))
    kw = dict(d_sum=ds[0].cuda()) if given else {}
    layer.step(x, g, residual=r, **kw)
    same(layer, 0)
    graphs = [layer.capture_step(x, g, residual=r, **kw)], layer.capture_halves(x, g, residual=r, **kw)
    for parts in graphs:
        for i in (1, 2):
            x.copy_(xs[i]), g.copy_(gs[i]), r.copy_(rs[i])
            if given:
                kw["d_sum"].copy_(ds[i])
            for part in parts:
                part.replay()
            same(layer, i)
    for layer, host_graphs in ((layer, True), (layer, False), (make(), False)):
        own = layer.dx, layer.norm.d_residual
        for also in (True, False):
            dx = [torch.empty_like(v).pin_memory() for v in xs]
            dr = [torch.empty_like(v).pin_memory() for v in rs]
            layer.steps_from_host(xs, gs, dx, graphs=host_graphs, residual_host=rs, d_sum_host=ds if given else None,
                                  d_residual_host=dr if also else None)
            torch.cuda.synchronize()
            for i in range(n):
                assert torch.equal(dx[i], want[i][0].cpu()) and (not also or torch.equal(dr[i], want[i][1].cpu())), i
        assert layer.dx is own[0] and (res == BF or layer.norm.d_residual is own[1])
        layer.step(xs[1].cuda(), gs[1].cuda(), residual=rs[1].cuda(), **(dict(d_sum=ds[1].cuda()) if given else {}))
        same(layer, 1)


def test_a_layer_whose_steps_take_a_sums_gradient_only_sometimes():
    """Steps from the host with and without d_sum, in turn, have graphs of their own."""
    from sparse_moe_layer_topk_gb300.layer import LatentMoELayer, weights_to_device
    inp = I.make_layer_inputs(0)
    inp["norm"] = torch.ones(inp["cfg"].d)
    cfg, w, gen = inp["cfg"], weights_to_device(inp), torch.Generator().manual_seed(8)
    layer = LatentMoELayer(w, cfg.T, cfg.k, residual_dtype=BF)
    x, g, r, d = ([torch.randn(cfg.T, cfg.d, generator=gen).to(BF).pin_memory()] for _ in range(4))
    want = []
    for kw in ({}, dict(d_sum=d[0].cuda())):
        layer.step(x[0].cuda(), g[0].cuda(), residual=r[0].cuda(), **kw)
        want.append(layer.dx.cpu())
    assert not torch.equal(*want)
    for turn in (0, 1, 0, 1):
        out = [torch.empty_like(x[0]).pin_memory()]
        layer.steps_from_host(x, g, out, residual_host=r, d_sum_host=d if turn else None)
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[turn])


def test_the_example_chooses_experts_in_groups(example):
    """Some groups of experts are left out for each token, others for other tokens."""
    w = example.ScanWeights(0)
    T = 96
    block = example.ScanBlock(w, T, 1, T)
    x = torch.randn(T, w.cfg.d, generator=torch.Generator().manual_seed(5)).to(BF)
    block.forward(x.cuda(), torch.tensor([0, T], dtype=torch.int32, device="cuda"))
    r = block.moe.router
    assert 1 < r.group_k < r.groups
    groups = block.moe.topk_idx.cpu() // (w.cfg.E // r.groups)
    assert all(len(set(row)) <= r.group_k for row in groups.tolist()) and set(groups.flatten().tolist()) == set(range(r.groups))
