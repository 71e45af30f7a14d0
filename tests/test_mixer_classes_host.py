"""What the classes of routing, norm, convolution and scan refuse, before any call of the library reaches a GPU: every operand
lies in host memory."""
import pytest
import torch

from sparse_moe_layer_topk_gb300 import _lib as M
from sparse_moe_layer_topk_gb300 import build as B
from sparse_moe_layer_topk_gb300 import inputs as I
from sparse_moe_layer_topk_gb300.layer import LatentMoELayer, weights_to_device
from sparse_moe_layer_topk_gb300.norm import RMSNorm
from sparse_moe_layer_topk_gb300.route import Router
from sparse_moe_layer_topk_gb300.scan import CausalConv, SelectiveScan

BF = torch.bfloat16
Z = torch.zeros


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build_library()
    M.load()


@pytest.mark.parametrize("kw,match", [
    (dict(score="tanh"), "score"), (dict(groups=3), "groups"), (dict(groups=0), "groups"), (dict(groups=64), "groups"), (dict(groups=4, group_k=5), "group"),
    (dict(groups=4, group_k=0), "group"), (dict(k=33), "k is"), (dict(k=0), "k is"), (dict(groups=16, group_k=1, k=5), "k is"),
    (dict(group_top=3), "group_top"), (dict(scale=0.0), "scale"), (dict(grad_dtype=torch.float16), "grad_dtype")], ids=str)
def test_router_options(kw, match):
    with pytest.raises(ValueError, match=match):
        Router(4, 64, **{"k": 4, **kw}, device="cpu")


@pytest.mark.parametrize("logits,bias,match", [
    (Z(4, 63), None, "logits"), (Z(3, 64), None, "logits"), (Z(4, 64, dtype=BF), None, "logits"), (Z(64, 4).t(), None, "logits"),
    (Z(4, 64), Z(63), "bias"), (Z(4, 64), Z(64, dtype=torch.float64), "bias"), (Z(4, 64), Z(128)[::2], "bias")], ids=str)
def test_router_operands(logits, bias, match):
    with pytest.raises(ValueError, match=match):
        Router(4, 64, 4, device="cpu").forward(logits, bias)


def test_router_backward_refusals():
    r = Router(4, 64, 4, device="cpu")
    with pytest.raises(ValueError, match="forward before"):
        r.backward(Z(4, 4))
    r.saved = Z(4, 64)
    for args, match in (((Z(4, 5),), "d_w"), ((Z(16), Z(4, 4)), "slot_of"), ((Z(15), Z(4, 4, dtype=torch.int32)), "d_w"),
                        ((Z(4, 4), None, Z(4, 3)), "d_topk_w")):
        with pytest.raises(ValueError, match=match):
            r.backward(*args)


@pytest.mark.parametrize("weight,kw,match", [
    (Z(64, dtype=BF), {}, "weight"), (Z(8, 8), {}, "weight"), (Z(128)[::2], {}, "weight"), (Z(64), dict(residual_dtype=torch.float16), "residual_dtype"),
    (Z(64), dict(out="int8"), "out"), (Z(64), dict(eps=0.0), "eps"), (Z(256), dict(out="fp8", block=32), "block")], ids=str)
def test_norm_options(weight, kw, match):
    with pytest.raises(ValueError, match=match):
        RMSNorm(weight, 4, **kw)


def test_norm_operands():
    n, m = RMSNorm(Z(64), 4), RMSNorm(Z(64), 4, residual_dtype=BF)
    x = Z(4, 64, dtype=BF)
    for call, match in ((lambda: n.forward(Z(4, 64)), "x is"), (lambda: n.forward(Z(3, 64, dtype=BF)), "x is"), (lambda: n.forward(Z(64, 4, dtype=BF).t()), "columns"),
                        (lambda: n.forward(x, x), "residual"), (lambda: m.forward(x), "residual"), (lambda: m.forward(x, Z(4, 64)), "residual"),
                        (lambda: m.forward(x, Z(4, 128, dtype=BF)[:, :64]), "contiguous"), (lambda: n.backward(x), "forward before"),
                        (lambda: RMSNorm(Z(64), 4, backward=False).backward(x), "without a backward")):
        with pytest.raises(ValueError, match=match):
            call()
    n.saved = m.saved = (x, 64)
    for call, match in ((lambda: n.backward(Z(4, 64)), "dy"), (lambda: n.backward(x, x), "no sum"), (lambda: m.backward(x, Z(4, 64)), "d_sum")):
        with pytest.raises(ValueError, match=match):
            call()


@pytest.mark.parametrize("stride", [1 << 31, (1 << 32) + 64])
def test_rows_too_far_apart(stride):
    x = torch.empty_strided((4, 64), (stride, 1), dtype=BF, device="meta")
    with pytest.raises(ValueError, match="apart"):
        RMSNorm(Z(64), 4)._rows("x", x, BF, strided=True)
    with pytest.raises(ValueError, match="apart"):
        CausalConv(Z(64, 4), None, 4).forward(x)


def _conv(T=8, N=2, **kw):
    return CausalConv(Z(16, 4), Z(16), T, N=N, **kw)


def _scan(T=8, N=2, G=2, **kw):
    return SelectiveScan(Z(16, 4), T, groups=G, N=N, max_seqlen=T, **kw)


def test_convolution_and_scan_options():
    for call, match in ((lambda: CausalConv(Z(16, 4, dtype=BF), None, 8), "weight"), (lambda: CausalConv(Z(4, 16).t(), None, 8), "weight"),
                        (lambda: CausalConv(Z(16, 4), Z(15), 8), "bias"), (lambda: SelectiveScan(Z(16), 8), "A is"),
                        (lambda: SelectiveScan(Z(16, 4), 8, skip=Z(4)), "skip"), (lambda: SelectiveScan(Z(16, 4), 8, dt_bias=Z(16, dtype=BF)), "dt_bias"),
                        (lambda: SelectiveScan(Z(16, 4), 8, groups=3), "groups")):
        with pytest.raises(ValueError, match=match):
            call()


@pytest.mark.parametrize("cu", [torch.tensor([0, 3, 8]), torch.tensor([3, 8], dtype=torch.int32), torch.tensor([0, 9, 3, 9, 8], dtype=torch.int32)[::2],
                                torch.tensor([0.0, 3.0, 8.0])], ids=str)
def test_sequence_bounds_of_another_form(cu):
    x, b = Z(8, 16, dtype=BF), Z(8, 2, 4, dtype=BF)
    with pytest.raises(ValueError, match="cu_seqlens"):
        _conv().forward(x, cu)
    with pytest.raises(ValueError, match="cu_seqlens"):
        _scan().forward(x, x, b, b, None, cu)


def test_convolution_and_scan_operands():
    x, b, c, s = Z(8, 16, dtype=BF), Z(8, 2, 4, dtype=BF), _conv(), _scan()
    state, kept = Z(3, 16, 4), Z(3, 3, 16, dtype=BF)
    idx = Z(8, dtype=torch.int32) - 1
    for call, match in ((lambda: c.forward(Z(8, 16)), "x is"), (lambda: c.forward(Z(16, 8, dtype=BF).t()), "contiguous"), (lambda: c.forward(x, None, Z(2, 4, 16, dtype=BF)), "state_in"),
                        (lambda: c.step(x, kept.float(), idx), "state"), (lambda: c.step(x, kept, idx.long()), "state_idx"), (lambda: c.backward(x), "forward before"),
                        (lambda: _conv(backward=False).backward(x), "without a backward"), (lambda: s.forward(x, x, b[:, :1], b), "B is"),
                        (lambda: s.forward(x, x, b, Z(8, 4, 4, dtype=BF)[:, ::2]), "C: the values"), (lambda: s.forward(x, x, b, b, Z(8, 16)), "z is"),
                        (lambda: s.forward(x, x, b, b, None, None, Z(2, 16, 4, dtype=BF)), "state_in"), (lambda: s.step(x, x, b, b, None, Z(3, 4, 16), idx), "state"),
                        (lambda: s.step(x, x, b, b, None, state, idx[:4]), "state_idx"), (lambda: s.backward(x), "forward before"),
                        (lambda: _scan(backward=False).backward(x), "without a backward")):
        with pytest.raises(ValueError, match=match):
            call()
    c.saved, s.saved = (x, None, None), (x, x, b, b, None, None, False)
    for call, match in ((lambda: c.backward(x, Z(2, 3, 16)), "d_state_out"), (lambda: s.backward(x, Z(2, 16, 4, dtype=BF)), "d_state_out"), (lambda: s.backward(Z(8, 16)), "dy")):
        with pytest.raises(ValueError, match=match):
            call()


def test_layer_options():
    inp = I.make_layer_inputs(0)
    w = weights_to_device(inp, "cpu")
    make = lambda w=w, **kw: LatentMoELayer(w, 4, 2, device="cpu", **kw)  # noqa: E731
    with pytest.raises(ValueError, match="auxiliary"):
        make(router={}, aux_scale=0.1)
    with pytest.raises(ValueError, match="norm"):
        make(residual_dtype=BF)
    with pytest.raises(ValueError, match="norm"):
        make({**w, "norm": torch.ones(8)})
    with pytest.raises(ValueError, match="norm"):
        make().forward(inp["x"][:4], residual=inp["x"][:4])
    layer = make({**w, "norm": torch.ones(w["Wr"].shape[0])}, router=dict(score="softmax", groups=2, group_k=1))
    assert layer.grads["norm"] is layer.norm.dw and layer.topk_idx is layer.router.topk_idx
    assert weights_to_device({**inp, "norm": torch.ones(4)}, "cpu")["norm"].tolist() == [1.0] * 4


def test_a_layers_gradient_of_a_sum_that_is_not_there():
    """Refused before anything is computed (a call of the library would refuse the host's tensors)."""
    inp = I.make_layer_inputs(0)
    w = weights_to_device(inp, "cpu")
    normed = {**w, "norm": torch.ones(w["Wr"].shape[0])}
    g = inp["g"][:4]
    for layer in (LatentMoELayer(w, 4, 2, device="cpu"), LatentMoELayer(normed, 4, 2, device="cpu")):
        with pytest.raises(ValueError, match="no sum"):
            layer.backward(g, d_sum=g)
    layer = LatentMoELayer(normed, 4, 2, device="cpu", residual_dtype=BF)
    for d_sum in (g.float(), g[:3], torch.zeros(4, 2 * g.shape[1], dtype=BF)[:, ::2]):
        with pytest.raises(ValueError, match="d_sum"):
            layer.backward(g, d_sum=d_sum)


def test_residuals_of_steps_from_the_host():
    inp = I.make_layer_inputs(0)
    w = weights_to_device(inp, "cpu")
    normed = {**w, "norm": torch.ones(w["Wr"].shape[0])}
    x = [inp["x"][:4].contiguous()]
    plain, layer = LatentMoELayer(w, 4, 2, device="cpu"), LatentMoELayer(normed, 4, 2, device="cpu", residual_dtype=BF)
    for make, kw, match in ((layer, {}, "residual"), (plain, dict(residual_host=x), "residual"), (plain, dict(d_sum_host=x), "no sum"),
                            (plain, dict(d_residual_host=x), "no sum"), (layer, dict(residual_host=x * 2), "residual_host is 1"),
                            (layer, dict(residual_host=[x[0].float()]), "residual_host"), (layer, dict(residual_host=x, d_sum_host=[x[0][:3]]), "d_sum_host"),
                            (layer, dict(residual_host=x, d_residual_host=[x[0].float()]), "d_residual_host")):
        with pytest.raises(ValueError, match=match):
            make.steps_from_host(x, x, x, **kw)
