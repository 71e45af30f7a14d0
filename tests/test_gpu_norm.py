"""The residual norm on the GPU against the fp64 oracle.

A row's sum of squares is fp32 in at most 2^6 additions one after another and a tree: rstd within 2^-17. An output in bf16 is half
a step off besides (2^-8 of it), one in E4M3 2^-4 of it or half the smallest step (2^-10 of the scale)."""
import numpy as np
import pytest
import torch

from oracle import mixer_oracle as O
from gpu_util import f64, need_gpu

pytestmark = pytest.mark.gpu
BF, F32, E8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS, TOL = 1e-6, 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _norm(*a, **k):
    from sparse_moe_layer_topk_gb300.norm import RMSNorm
    return RMSNorm(*a, **k)


def _inputs(T, d, res, seed=0, wide=0):
    g = torch.Generator().manual_seed(seed + d)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (n(T, d + wide) * torch.exp(2 * n(T, 1))).to(BF)[:, :d]
    return x, None if res is None else (3 * n(T, d)).to(res), 1 + 0.3 * n(d), n(T, d).to(BF), None if res is None else n(T, d).to(res)


def _sum(x, r):
    return f64(x) + (0 if r is None else f64(r))


SIZES = [(1, 8), (3, 64), (5, 72), (9, 1000), (4, 1024), (7, 1032), (2, 4096), (3, 4104), (2, 5120), (3, 8192), (2, 8200), (2, 16384), (130, 256)]


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("res", [None, BF, F32])
@pytest.mark.parametrize("wide", [0, 24])
def test_forward(T, d, res, wide):
    x, r, w, _, _ = _inputs(T, d, res, wide=wide)
    n = _norm(w.cuda(), T, EPS, res, backward=False)
    xd = x.cuda() if not wide else torch.cat([x, x[:, :wide]], 1).cuda()[:, :d]
    y = n.forward(xd, None if r is None else r.cuda())
    u = _sum(x, r)
    want = O.rmsnorm(u, f64(w), EPS)
    assert (np.abs(f64(y) - want) <= (2.0 ** -8 + TOL) * np.abs(want) + 1e-30).all()
    if r is not None:
        assert torch.equal(n.sum.cpu(), (x.float() + r.float()).to(res))


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("block", [64, 128, 0])
@pytest.mark.parametrize("res", [None, F32])
def test_forward_in_8_bits(T, d, block, res):
    x, r, w, _, _ = _inputs(T, d, res, 1)
    x[0] = 0
    if r is not None:
        r[0] = 0  # a row of zeros: scale 0, codes 0
    block = block or d
    n = _norm(w.cuda(), T, EPS, res, out="fp8", block=block, backward=False)
    y = n.forward(x.cuda(), None if r is None else r.cuda())
    want = O.rmsnorm(_sum(x, r), f64(w), EPS)
    pad = np.pad(want, ((0, 0), (0, -d % block))).reshape(T, -1, block)
    scale = np.abs(pad).max(-1) / 448
    np.testing.assert_allclose(f64(n.scale), scale, rtol=TOL, atol=1e-33)
    each = np.repeat(f64(n.scale), block, 1)[:, :d]
    got = f64(y.float()) * each
    assert y.dtype == E8 and (np.abs(got - want) <= (2.0 ** -4 + TOL) * np.abs(want) + 2.0 ** -10 * each * (1 + TOL)).all()


@pytest.mark.parametrize("T,d", SIZES + [(1500, 64), (700, 4096)])
@pytest.mark.parametrize("res", [None, BF, F32])
@pytest.mark.parametrize("given", [False, True])
def test_backward(T, d, res, given):
    """dx: fp32 operations on sums of d terms, a rounding to its type. dw: T products in fp32, a few hundred one after another."""
    x, r, w, dy, ds = _inputs(T, d, res, 2)
    n = _norm(w.cuda(), T, EPS, res)
    n.forward(x.cuda(), None if r is None else r.cuda())
    ds = ds if given else None
    dx = n.backward(dy.cuda(), None if ds is None else ds.cuda())
    u = f64(x) if r is None else f64(n.sum)
    want, dw = O.rmsnorm_backward(f64(dy), u, f64(w), EPS, None if ds is None else f64(ds))
    rstd = 1 / np.sqrt((u * u).mean(1, keepdims=True) + EPS)
    gw = np.abs(f64(dy) * f64(w))
    size = rstd * (gw + np.abs(u * rstd) * (gw * np.abs(u * rstd)).mean(1, keepdims=True)) + (0 if ds is None else np.abs(f64(ds)))
    assert (np.abs(f64(dx) - want) <= 2.0 ** -8 * np.abs(want) + TOL * size).all()
    if res is not None:
        half = 2.0 ** -8 if res == BF else 2.0 ** -24
        assert (np.abs(f64(n.d_residual) - want) <= half * np.abs(want) + TOL * size).all()
    size = (np.abs(f64(dy)) * np.abs(u * rstd)).sum(0)
    assert (np.abs(f64(n.dw) - dw) <= 2 * TOL * size).all()


def test_sums_in_place():
    x, r, w, dy, _ = _inputs(6, 512, BF)
    a, b = _norm(w.cuda(), 6, EPS, BF), _norm(w.cuda(), 6, EPS, BF)
    stream = r.cuda()
    ya, yb = a.forward(x.cuda(), stream, in_place=True), b.forward(x.cuda(), r.cuda())
    assert torch.equal(ya, yb) and torch.equal(stream, b.sum)
    assert torch.equal(a.backward(dy.cuda()), b.backward(dy.cuda()))


@pytest.mark.parametrize("size", [1e18, 1e25, 3e38, 1e-30])
def test_values_whose_squares_leave_fp32(size):
    x = (torch.randn(3, 2048, generator=torch.Generator().manual_seed(0)).clamp(-1, 1) * size).to(BF)
    dy = torch.randn(3, 2048, generator=torch.Generator().manual_seed(1)).to(BF)
    w = torch.ones(2048)
    n = _norm(w.cuda(), 3, EPS)
    y, u = n.forward(x.cuda()), f64(x)
    want = O.rmsnorm(u, f64(w), EPS)
    assert (np.abs(f64(y) - want) <= (2.0 ** -8 + TOL) * np.abs(want) + 1e-37).all()
    n.backward(dy.cuda())
    rstd = 1 / np.sqrt((u * u).mean(1, keepdims=True) + EPS)
    dw = (f64(dy) * u * rstd).sum(0)
    assert (np.abs(f64(n.dw) - dw) <= 2 * TOL * (np.abs(f64(dy) * u * rstd)).sum(0) + 1e-37).all()


def test_a_row_with_an_infinity_or_nan_keeps_to_itself():
    x, _, w, _, _ = _inputs(9, 1024, None)
    n = _norm(w.cuda(), 9, EPS)
    clean = n.forward(x.cuda()).clone()
    x[3, 5], x[7, 1000] = float("nan"), float("inf")
    y = n.forward(x.cuda())
    rest = [0, 1, 2, 4, 5, 6, 8]
    assert torch.equal(y[rest], clean[rest]) and bool(y[3].isnan().all()) and bool(y[7, 1000].isnan())


def test_no_rows():
    n = _norm(torch.ones(64, device="cuda"), 0, EPS)
    assert n.forward(torch.empty(0, 64, dtype=BF, device="cuda")).shape == (0, 64)
    n.backward(torch.empty(0, 64, dtype=BF, device="cuda"))
    assert not n.dw.any()


def test_in_a_graph_and_on_another_stream():
    x, r, w, dy, ds = (v.cuda() for v in _inputs(200, 1536, F32))
    n, m = _norm(w, 200, EPS, F32), _norm(w, 200, EPS, F32)
    n.forward(x, r), n.backward(dy, ds)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n.forward(x, r), n.backward(dy, ds)
    x.copy_(x.flip(0).clone())
    n.dw.zero_()
    graph.replay()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    m.forward(x, r, stream=side), m.backward(dy, ds, stream=side)
    torch.cuda.synchronize()
    for a, b in ((n.y, m.y), (n.sum, m.sum), (n.dx, m.dx), (n.dw, m.dw), (n.d_residual, m.d_residual)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,d", [(3, 64), (700, 1000), (2500, 4096), (40, 16384)])
@pytest.mark.parametrize("place", ["dy", "u", "d_sum"])
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=str)
def test_gradients_in_place(T, d, place, dtype):
    """A gradient over what its own row is read from, where the types are the same."""
    from sparse_moe_layer_topk_gb300 import _lib as M
    gen = torch.Generator().manual_seed(T + d)
    make = lambda *s, dt: torch.randn(*s, generator=gen).to(dt).cuda()  # noqa: E731
    ops = dict(dy=make(T, d, dt=BF), u=make(T, d, dt=dtype), d_sum=make(T, d, dt=dtype))
    w = make(d, dt=torch.float32)
    ws_bytes = M.moe_workspace_size(M.MOE_OP_RMSNORM_BWD, T=T, d=d)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
    code = M.MOE_DTYPE_F32 if dtype == torch.float32 else M.MOE_DTYPE_BF16

    def run(dy, u, d_sum, dx, d_residual):
        dw = torch.empty(d, device="cuda")
        M.moe_rmsnorm_bwd(dy, u, w, d_sum, T, d, d, code, 1e-6, dx, d_residual, dw, ws, ws_bytes)
        return dw

    dx, d_residual = torch.empty(T, d, dtype=BF, device="cuda"), torch.empty(T, d, dtype=dtype, device="cuda")
    want = run(**ops, dx=dx, d_residual=d_residual)
    for name, result, other in (("dx", dx, "d_residual"), ("d_residual", d_residual, "dx")):
        if ops[place].dtype != result.dtype:
            continue
        now = {n: t.clone() for n, t in ops.items()}
        dw = run(**now, **{name: now[place], other: None})
        assert torch.equal(now[place], result) and torch.equal(dw, want)


@pytest.mark.parametrize("size", [1e18, 1e25, 3e38, 1e-30])
@pytest.mark.parametrize("res", [None, BF, F32])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("d", [512, 2048, 5120])
def test_gradients_of_values_whose_squares_leave_fp32(size, res, given, d):
    """dx is as small as the values are large (rstd): d_sum, where it is given, is of its size. One row in three has ordinary values."""
    if given and res is None:
        return
    x, r, w, dy, ds = _inputs(7, d, res, 5)
    big = torch.tensor([1.0, 0.0, 0.0, 1.0, 1.0, 0.0, 1.0])[:, None] > 0
    x = torch.where(big, x.float().clamp(-1, 1) * size, x.float()).to(BF)
    if r is not None:
        r = torch.where(big, torch.zeros_like(r), r)
    n = _norm(w.cuda(), 7, EPS, res)
    n.forward(x.cuda(), None if r is None else r.cuda())
    u = f64(x) if r is None else f64(n.sum)
    rstd = 1 / np.sqrt((u * u).mean(1, keepdims=True) + EPS)
    ds = None
    if given:
        ds = (torch.randn(7, d, generator=torch.Generator().manual_seed(9)).double() * torch.from_numpy(rstd)).to(res)
    dx = n.backward(dy.cuda(), None if ds is None else ds.cuda())
    want, dw = O.rmsnorm_backward(f64(dy), u, f64(w), EPS, None if ds is None else f64(ds))
    gw = np.abs(f64(dy) * f64(w))
    bound = TOL * (rstd * (gw + np.abs(u * rstd) * (gw * np.abs(u * rstd)).mean(1, keepdims=True)) + (0 if ds is None else np.abs(f64(ds))))
    # (2^-126 and below: what fp32 and bf16 leave of a gradient is a multiple of 2^-133 there)
    assert (np.abs(f64(dx) - want) <= 2.0 ** -8 * np.abs(want) + bound + 2.0 ** -126).all()
    if res is not None:
        half = 2.0 ** -8 if res == BF else 2.0 ** -24
        assert (np.abs(f64(n.d_residual) - want) <= half * np.abs(want) + bound + 2.0 ** -126).all()
    assert (np.abs(f64(n.dw) - dw) <= 2 * TOL * (np.abs(f64(dy)) * np.abs(u * rstd)).sum(0) + 1e-37).all()
