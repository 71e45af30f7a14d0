"""Causal convolution and selective scan on the GPU against the fp64 oracle: forward, backward and steps.

Inputs are bf16 or fp32 and exact on both sides. Everything in between is fp32. A term of the scan that is t tokens old has
passed t products with decays, each off by at most 2^-21 (the argument's rounding, the exponential's 2 ulp, the product, the time step): with
L tokens, sums are within (L + 16) 2^-21 of the same formulas over magnitudes. Sums over T tokens add T 2^-24. A bf16
output is half a step off besides, 2^-8 of it. The convolution has W <= 4 terms: 2^-18 of the magnitudes.
"""
import numpy as np
import pytest
import torch

from oracle import mixer_oracle as O
from sparse_moe_layer_topk_gb300 import _lib as M
from gpu_util import f64, need_gpu

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _dev(t):
    return None if t is None else t.cuda()


def _np(t):
    return None if t is None else f64(t)


def _close(name, got, want, size, tol, half=2.0 ** -8):
    got = f64(got)
    assert np.isfinite(got).all(), name
    bound = half * np.abs(want) + tol * size + 1e-30
    worst = (np.abs(got - want) / bound).max() if got.size else 0.0
    assert worst <= 1.0, f"{name}: {worst:.2f} of the bound"


# ------------------------------------------------------------------ convolution

def _conv_inputs(lens, D, W, states, wide=0, seed=0):
    g = torch.Generator().manual_seed(seed + D + W)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    T, N = sum(lens), len(lens)
    st = lambda: n(N, W - 1, D).to(BF) if states else None  # noqa: E731
    return dict(x=n(T, D + wide).to(BF)[:, :D], w=n(D, W), b=n(D), st=st(), dy=n(T, D).to(BF), ds=st())


def _conv(v, lens, silu, bias=True, **kw):
    from sparse_moe_layer_topk_gb300.scan import CausalConv
    return CausalConv(v["w"].cuda(), v["b"].cuda() if bias else None, sum(lens), N=len(lens), silu=silu, **kw)


LENS = [[1], [2], [3], [4], [31], [32], [33], [64], [65], [127, 1, 0, 70], [0], [0, 0, 5], [2, 1, 1, 0, 3], [129]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("states", [False, True])
def test_convolution(lens, W, states):
    D, silu = 24, W != 3
    v = _conv_inputs(lens, D, W, states)
    c = _conv(v, lens, silu)
    y = c.forward(v["x"].cuda(), _cu(lens), _dev(v["st"]), want_state=True)
    dx = c.backward(v["dy"].cuda(), _dev(v["ds"]))
    x, w, b, st, dy, ds = (_np(v[k]) for k in ("x", "w", "b", "st", "dy", "ds"))
    ab = lambda a: None if a is None else np.abs(a)  # noqa: E731
    size = O.conv(np.abs(x), np.abs(w), np.abs(b), lens, False, ab(st))[0]
    want, last = O.conv(x, w, b, lens, silu, st)
    _close("y", y, want, size, 2.0 ** -18)
    assert np.array_equal(f64(c.state_out), last)
    want = O.conv_backward(dy, x, w, b, lens, silu, st, ds)
    # silu' and its slope are below 1.1 and 0.5; p is off by 2^-18 of its terms' sizes
    p_size = O.conv(np.abs(x), np.abs(w), np.abs(b), lens, False, ab(st))[0]
    sizes = O.conv_backward(np.abs(dy) * (1.1 + (0.5 * p_size if silu else 0)), np.abs(x), np.abs(w), np.abs(b), lens, False, ab(st), ab(ds))
    names, got = ("dx", "dw", "db", "d_state_in"), (dx, c.dw, c.db, c.d_state_in)
    tol = 2.0 ** -18 + sum(lens) * 2.0 ** -24
    for k in range(4 if states else 3):
        _close(names[k], got[k], want[k], sizes[k], tol, 2.0 ** -8 if k in (0, 3) else 0)
    assert int(c.err) == 0


@pytest.mark.parametrize("D,wide", [(8, 0), (8, 8), (512, 0), (520, 40), (1032, 0)])
@pytest.mark.parametrize("bias", [False, True])
def test_convolution_widths(D, wide, bias):
    lens = [70, 3]
    v = _conv_inputs(lens, D, 4, True, wide)
    c = _conv(v, lens, True, bias)
    x = torch.empty(73, D + wide, dtype=BF, device="cuda")[:, :D]
    x.copy_(v["x"])
    y = c.forward(x, _cu(lens), v["st"].cuda())
    dx = c.backward(v["dy"].cuda())
    b = _np(v["b"]) if bias else None
    args = f64(v["x"]), f64(v["w"]), b, lens, True, f64(v["st"])
    size = O.conv(*(np.abs(a) if isinstance(a, np.ndarray) else a for a in args[:4]), False, np.abs(args[5]))[0]
    _close("y", y, O.conv(*args)[0], size, 2.0 ** -18)
    want = O.conv_backward(f64(v["dy"]), *args)
    norm = np.linalg.norm
    assert norm(f64(dx) - want[0]) <= 2.0 ** -8 * norm(want[0])
    assert norm(f64(c.dw) - want[1]) <= 2.0 ** -16 * norm(want[1])
    assert norm(f64(c.db) - want[2]) <= 2.0 ** -16 * norm(want[2])


def test_convolution_without_bounds_and_in_pieces():
    """Sequences of one length need no bounds; one handed on in two pieces gives what it gives whole."""
    v = _conv_inputs([90, 90], 64, 4, False)
    c = _conv(v, [90, 90], True)
    whole = c.forward(v["x"].cuda()).clone()
    assert torch.equal(c.forward(v["x"].cuda(), _cu([90, 90])), whole)
    x = v["x"].cuda().view(2, 90, 64)
    first, second = _conv(v, [37, 37], True), _conv(v, [53, 53], True)
    a = first.forward(x[:, :37].reshape(-1, 64), want_state=True)
    b = second.forward(x[:, 37:].reshape(-1, 64), state_in=first.state_out)
    assert torch.equal(torch.cat([a.view(2, 37, 64), b.view(2, 53, 64)], 1).view(-1, 64), whole)


def test_convolution_states_in_place():
    v = _conv_inputs([2, 50], 32, 4, True)
    a, b = _conv(v, [2, 50], True), _conv(v, [2, 50], True)
    x, dy, cu = v["x"].cuda(), v["dy"].cuda(), _cu([2, 50])
    a.state_out.copy_(v["st"])
    ya, yb = a.forward(x, cu, a.state_out, want_state=True), b.forward(x, cu, v["st"].cuda(), want_state=True)
    assert torch.equal(ya, yb) and torch.equal(a.state_out, b.state_out)
    assert torch.equal(a.backward(dy), b.backward(dy)) and torch.equal(a.dw, b.dw)


@pytest.mark.parametrize("W", [2, 3, 4])
def test_convolution_steps_follow_the_packed_pass(W):
    lens, D = [9, 14, 6], 136
    v = _conv_inputs(lens, D, W, True)
    x, at = v["x"].cuda(), np.concatenate([[0], np.cumsum(lens)])
    c = _conv(v, lens, True, backward=False)
    want = c.forward(x, _cu(lens), v["st"].cuda(), want_state=True)
    cache = torch.zeros(7, W - 1, D, dtype=BF, device="cuda")
    slot = torch.tensor([4, 0, 6], dtype=torch.int32, device="cuda")
    cache[slot.long()] = v["st"].cuda()
    one = _conv(v, [1, 1, 1], True, backward=False)
    for t in range(max(lens)):
        live = torch.tensor([t < n for n in lens], device="cuda")
        rows = torch.stack([x[at[n] + min(t, lens[n] - 1)] for n in range(3)])
        y = one.step(rows, cache, torch.where(live, slot, -1).int())
        for n in range(3):
            if t < lens[n]:  # (the step rounds every operation, the packed pass does not: a bf16 step apart at most)
                ref = f64(want[at[n] + t])
                assert (np.abs(f64(y[n]) - ref) <= 2.0 ** -7 * np.abs(ref) + 1e-6).all()
            else:
                assert not y[n].any()
    assert torch.equal(cache[slot.long()], c.state_out)
    assert not cache[[1, 2, 3, 5]].any() and int(one.err) == 0


# ------------------------------------------------------------------ scan

def _scan_inputs(lens, D, S, G, states=True, gate=True, seed=0, slow=False):
    g = torch.Generator().manual_seed(seed + D + S)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    T, N = sum(lens), len(lens)
    st = lambda: n(N, D, S) if states else None  # noqa: E731
    return dict(u=n(T, D).to(BF), delta=n(T, D).to(BF), A=-torch.exp(n(D, S)), B=n(T, G, S).to(BF), C=n(T, G, S).to(BF), skip=n(D),
                z=n(T, D).to(BF) if gate else None, bias=n(D) - (5 if slow else 2), st=st(), dy=n(T, D).to(BF), ds=st())


def _scan(v, lens, **kw):
    from sparse_moe_layer_topk_gb300.scan import SelectiveScan
    kw = dict(skip=v["skip"].cuda(), dt_bias=v["bias"].cuda(), groups=v["B"].shape[1], N=len(lens), max_seqlen=max(lens, default=0), **kw)
    return SelectiveScan(v["A"].cuda(), sum(lens), **kw)


def _operands(v):
    return [_dev(v[k]) for k in ("u", "delta", "B", "C", "z")]


def _check_scan(v, lens, s=None, bwd=True):
    s = s or _scan(v, lens, backward=bwd)
    y = s.forward(*_operands(v), _cu(lens), _dev(v["st"]), want_state=True)
    a = {k: _np(t) for k, t in v.items()}
    ab = {k: None if t is None else np.abs(t) for k, t in a.items()}
    rest = (a["A"], a["B"], a["C"], lens, a["skip"], a["z"], a["bias"], a["st"])
    sizes = (a["A"], ab["B"], ab["C"], lens, ab["skip"], None, a["bias"], ab["st"])
    T, tol = sum(lens), (max(lens, default=0) + 16) * 2.0 ** -21
    want, last = O.scan(a["u"], a["delta"], *rest)
    size, last_size = O.scan(ab["u"], a["delta"], *sizes)
    gate = 1.0 if a["z"] is None else np.abs(a["z"] * O.sigmoid(a["z"]))
    _close("y", y, want, size * gate, tol)
    _close("state_out", s.state_out, last, last_size, tol, 2.0 ** -24)
    assert int(s.err) == 0
    if not bwd:
        return s
    got = dict(zip(("du", "ddelta", "dB", "dC", "dz"), s.backward(v["dy"].cuda(), _dev(v["ds"]))))
    got.update(dA=s.dA, dskip=s.dskip, d_dt_bias=s.d_dt_bias)
    if v["st"] is not None or v["ds"] is not None:
        got["d_state_in"] = s.d_state_in
    want = O.scan_backward(a["dy"], a["u"], a["delta"], *rest, d_state=a["ds"])
    g = np.abs(a["dy"]) * gate
    bound = O.scan_backward(g, ab["u"], a["delta"], *sizes, d_state=ab["ds"], size=True)
    if a["z"] is not None:
        sg = O.sigmoid(a["z"])
        bound["dz"] = np.abs(a["dy"]) * size * np.abs(sg * (1 + a["z"] * (1 - sg)))
    else:
        assert got.pop("dz") is None
    for k, t in got.items():
        half = 2.0 ** -8 if t.dtype == BF else 2.0 ** -24
        _close(k, t, want[k], bound[k], 2 * tol + T * 2.0 ** -24, half)
    assert int(s.err) == 0
    return s


SCAN_LENS = [[1], [2], [31], [32], [33], [64], [65], [100, 0, 1, 37], [0], [0, 0, 3], [129, 5]]


@pytest.mark.parametrize("lens", SCAN_LENS, ids=str)
@pytest.mark.parametrize("states,gate", [(True, True), (False, False)])
def test_scan(lens, states, gate):
    _check_scan(_scan_inputs(lens, 16, 16, 1, states, gate), lens)


@pytest.mark.parametrize("D,S,G", [(8, 16, 1), (8, 4, 2), (64, 8, 1), (72, 12, 1), (24, 16, 2), (40, 4, 5), (136, 16, 1), (264, 8, 2), (48, 16, 12)])
def test_scan_widths(D, S, G):
    _check_scan(_scan_inputs([45, 20], D, S, G), [45, 20])


@pytest.mark.parametrize("D,N,length", [(8, 1, 1500), (64, 2, 700), (24, 1, 900)])
@pytest.mark.parametrize("slow", [False, True])
def test_long_sequences_in_parts(D, N, length, slow):
    """Few channels: the time axis is cut, sums first. With memories of a few tokens and of hundreds."""
    lens = [length] * N
    lens[-1] -= 77
    _check_scan(_scan_inputs(lens, D, 8, 1, slow=slow), lens)


@pytest.mark.parametrize("lens,most", [([40, 3], 2 ** 31 - 1), ([900], 2 ** 31 - 1), ([900], 10 ** 12), ([0], 5000), ([0, 0], 9000)], ids=str)
def test_any_bound_of_the_lengths(lens, most):
    from sparse_moe_layer_topk_gb300.scan import SelectiveScan
    v = _scan_inputs(lens, 16, 4, 1)
    s = SelectiveScan(v["A"].cuda(), sum(lens), v["skip"].cuda(), v["bias"].cuda(), N=len(lens), max_seqlen=most)
    _check_scan(v, lens, s)


@pytest.mark.parametrize("skip,bias,soft", [(False, True, True), (True, False, True), (True, True, False)])
def test_parts_that_may_be_left_out(skip, bias, soft):
    from sparse_moe_layer_topk_gb300.scan import SelectiveScan
    lens = [50, 9]
    v = _scan_inputs(lens, 32, 16, 1)
    if not soft:
        v["delta"], v["bias"] = (0.1 * v["delta"].float().abs()).to(BF), 0.05 * v["bias"].abs()
    s = SelectiveScan(v["A"].cuda(), 59, v["skip"].cuda() if skip else None, v["bias"].cuda() if bias else None, N=2, max_seqlen=50, softplus=soft)
    y = s.forward(*_operands(v), _cu(lens), v["st"].cuda())
    got = s.backward(v["dy"].cuda())
    a = {k: _np(t) for k, t in v.items()}
    rest = (a["A"], a["B"], a["C"], lens, a["skip"] if skip else None, a["z"], a["bias"] if bias else None, a["st"])
    want = O.scan(a["u"], a["delta"], *rest, soft=soft)[0]
    norm = np.linalg.norm
    assert norm(f64(y) - want) <= 2.0 ** -8 * norm(want)
    ref = O.scan_backward(a["dy"], a["u"], a["delta"], *rest, soft=soft)
    for k, t in zip(("du", "ddelta", "dB", "dC", "dz"), got):
        assert norm(f64(t) - ref[k]) <= 2.0 ** -8 * norm(ref[k]), k
    for k in ("dA", "dskip", "d_dt_bias"):
        assert norm(f64(getattr(s, k)) - ref[k]) <= 2.0 ** -14 * norm(ref[k]), k


def test_time_steps_of_all_sizes():
    """softplus keeps the relative precision of small steps and passes into the line for large ones."""
    from sparse_moe_layer_topk_gb300.scan import SelectiveScan
    x = torch.linspace(-80, 80, 4096).to(BF)
    D = 4096
    s = SelectiveScan(torch.zeros(D, 4, device="cuda"), 1, backward=False)
    one = torch.ones(1, 1, 4, dtype=BF, device="cuda")
    s.forward(torch.ones(1, D, dtype=BF, device="cuda"), x[None].cuda(), one, one, want_state=True)
    np.testing.assert_allclose(f64(s.state_out)[0, :, 0], O.softplus(f64(x)), rtol=2.0 ** -20, atol=1e-37)


def test_slices_of_wider_rows():
    lens, D, G, S = [33, 40], 24, 2, 8
    v = _scan_inputs(lens, D, S, G)
    s, ref = _scan(v, lens), _scan(v, lens)
    u, d, B, C, z = _operands(v)
    ref.forward(u, d, B, C, z, _cu(lens), v["st"].cuda())
    T = 73
    xz, bc = torch.cat([u, z, d], 1), torch.cat([torch.zeros(T, 4, dtype=BF, device="cuda"), B.flatten(1), C.flatten(1)], 1)
    parts = xz[:, :D], xz[:, 2 * D:], bc[:, 4:4 + G * S].unflatten(1, (G, S)), bc[:, 4 + G * S:].unflatten(1, (G, S)), xz[:, D:2 * D]
    assert torch.equal(s.forward(*parts, _cu(lens), v["st"].cuda()), ref.y)
    dy = v["dy"].cuda()
    for a, b in zip(s.backward(dy), ref.backward(dy)):
        assert torch.equal(a, b)


def test_states_in_place_and_in_pieces():
    v = _scan_inputs([80], 32, 16, 1)
    whole = _scan(v, [80])
    ops = _operands(v)
    whole.forward(*ops, state_in=v["st"].cuda(), want_state=True)
    dy = v["dy"].cuda()
    d_whole = [t.clone() for t in whole.backward(dy)]
    first, second = _scan(v, [32]), _scan(v, [48])
    first.state_out.copy_(v["st"])
    a = first.forward(*(t[:32] for t in ops), state_in=first.state_out, want_state=True)
    second.state_out.copy_(first.state_out)
    b = second.forward(*(t[32:] for t in ops), state_in=second.state_out, want_state=True)
    assert torch.equal(torch.cat([a, b]), whole.y) and torch.equal(second.state_out, whole.state_out)
    db = second.backward(dy[32:])
    da = first.backward(dy[:32], second.d_state_in)
    for w, x, y in zip(d_whole, da, db):
        assert torch.equal(w, torch.cat([x, y]))
    assert torch.equal(first.d_state_in, whole.d_state_in)


@pytest.mark.parametrize("D,S,G,gate", [(136, 16, 1, True), (24, 4, 2, False), (64, 12, 1, True)])
def test_scan_steps_follow_the_packed_pass(D, S, G, gate):
    lens = [9, 14, 6]
    v = _scan_inputs(lens, D, S, G, gate=gate)
    ops, at = _operands(v), np.concatenate([[0], np.cumsum(lens)])
    s = _scan(v, lens, backward=False)
    want = s.forward(*ops, _cu(lens), v["st"].cuda(), want_state=True)
    cache = torch.zeros(7, D, S, device="cuda")
    slot = torch.tensor([4, 0, 6], dtype=torch.int32, device="cuda")
    cache[slot.long()] = v["st"].cuda()
    one = _scan(v, [1, 1, 1], backward=False)
    for t in range(max(lens)):
        live = torch.tensor([t < n for n in lens], device="cuda")
        pick = [int(at[n] + min(t, lens[n] - 1)) for n in range(3)]
        y = one.step(*(None if x is None else x[pick] for x in ops), cache, torch.where(live, slot, -1).int())
        for n in range(3):
            ref = f64(want[at[n] + t]) if t < lens[n] else 0 * f64(y[n])
            # two fp32 computations of the same value, rounded: a bf16 step apart at most, and their own errors
            assert (np.abs(f64(y[n]) - ref) <= 2.0 ** -7 * np.abs(ref) + 1e-3).all()
    np.testing.assert_allclose(f64(cache[slot.long()]), f64(s.state_out), rtol=1e-4, atol=1e-4)
    assert not cache[[1, 2, 3, 5]].any() and int(one.err) == 0


# ------------------------------------------------------------------ both

BAD = [([0, 50, 40, 73], [1, 0, 0]), ([0, 30, 200, 73], [1, 0, 0]), ([-3, 30, 60, 73], [0, 1, 1]), ([0, 73, 73, 9], [1, 1, 0])]


@pytest.mark.parametrize("bounds,good", BAD, ids=str)
def test_sequences_out_of_place_are_skipped_and_flagged(bounds, good):
    """Nothing of them is written, in the backward either, and they add nothing to the weights' gradients."""
    from sparse_moe_layer_topk_gb300.scan import CausalConv, SelectiveScan
    T, D, N = 73, 16, 3
    v = _scan_inputs([T], D, 16, 1, states=False)
    w = _conv_inputs([T], D, 4, False)
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    s = SelectiveScan(v["A"].cuda(), T, v["skip"].cuda(), v["bias"].cuda(), N=N, max_seqlen=T)
    c = CausalConv(w["w"].cuda(), w["b"].cuda(), T, N=N)
    rows = [t for n in range(N) if good[n] for t in range(bounds[n], bounds[n + 1])]
    lens = [bounds[n + 1] - bounds[n] for n in range(N) if good[n]]
    other = sorted(set(range(T)) - set(rows))
    for t in (s.y, s.du, s.ddelta, s.dB, s.dC, s.dz, c.y, c.dx, s.state_out, c.state_out):
        t.fill_(7.0)
    y, yc = s.forward(*_operands(v), cu, want_state=True), c.forward(w["x"].cuda(), cu, want_state=True)
    assert int(s.err) == M.MOE_FLAG_BAD_INDEX and int(c.err) == M.MOE_FLAG_BAD_INDEX
    g = s.backward(v["dy"].cuda())
    gc = c.backward(w["dy"].cuda())
    for t in (y, yc, gc, *g):
        assert bool((t[other] == 7.0).all())
    skipped = [n for n in range(N) if not good[n]]
    assert bool((s.state_out[skipped] == 7.0).all()) and bool((c.state_out[skipped] == 7.0).all())
    pick = {k: t if k in ("A", "skip", "bias") or t is None else t[rows] for k, t in v.items()}
    r = _scan(pick, lens)
    assert torch.equal(r.forward(*_operands(pick), _cu(lens)), y[rows])
    for a, b in zip(r.backward(pick["dy"].cuda()), g):
        assert torch.equal(a, b[rows])
    np.testing.assert_allclose(f64(r.dA), f64(s.dA), rtol=1e-5, atol=1e-5)
    rc = _conv({**w, "x": w["x"][rows]}, lens, True)
    assert torch.equal(rc.forward(w["x"][rows].cuda(), _cu(lens)), yc[rows])
    rc.backward(w["dy"][rows].cuda())
    np.testing.assert_allclose(f64(rc.dw), f64(c.dw), rtol=1e-5, atol=1e-5)


def test_a_sequence_longer_than_its_bound_is_skipped():
    from sparse_moe_layer_topk_gb300.scan import SelectiveScan
    v = _scan_inputs([70], 16, 16, 1, states=False)
    s = SelectiveScan(v["A"].cuda(), 70, v["skip"].cuda(), v["bias"].cuda(), N=2, max_seqlen=40)
    s.y.fill_(7.0)
    y = s.forward(*_operands(v), _cu([25, 45]))
    assert int(s.err) == M.MOE_FLAG_BAD_INDEX
    assert bool((y[25:] == 7.0).all()) and not bool((y[:25] == 7.0).all())


def test_slots_out_of_range_are_flagged():
    v, w = _scan_inputs([1, 1], 16, 4, 1), _conv_inputs([1, 1], 16, 3, False)
    s, c = _scan(v, [1, 1], backward=False), _conv(w, [1, 1], True, backward=False)
    idx = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    state, kept = torch.ones(3, 16, 4, device="cuda"), torch.ones(3, 2, 16, dtype=BF, device="cuda")
    y, yc = s.step(*_operands(v), state, idx), c.step(w["x"].cuda(), kept, idx)
    assert int(s.err) == M.MOE_FLAG_BAD_INDEX and int(c.err) == M.MOE_FLAG_BAD_INDEX
    assert not y[0].any() and not yc[0].any() and y[1].any() and yc[1].any()
    assert bool((state[[0, 2]] == 1).all()) and bool((kept[[0, 2]] == 1).all())


def test_results_do_not_depend_on_timing():
    lens = [300, 41, 500]
    v, w = _scan_inputs(lens, 200, 16, 1), _conv_inputs(lens, 200, 4, True)
    s, c = _scan(v, lens), _conv(w, lens, True)
    runs = []
    for _ in range(3):
        s.forward(*_operands(v), _cu(lens), v["st"].cuda())
        c.forward(w["x"].cuda(), _cu(lens), w["st"].cuda())
        out = [*s.backward(v["dy"].cuda(), v["ds"].cuda()), s.dA, s.dskip, s.d_dt_bias, c.backward(w["dy"].cuda(), w["ds"].cuda()), c.dw, c.db]
        runs.append([t.clone() for t in out])
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


def test_in_a_graph_and_on_another_stream():
    lens = [900]  # in parts
    v, w = _scan_inputs(lens, 24, 8, 1), _conv_inputs(lens, 24, 4, True)
    made = [(_scan(v, lens), _conv(w, lens, True)) for _ in range(2)]
    ops, cu, st, cst = _operands(v), _cu(lens), v["st"].cuda(), w["st"].cuda()
    x, dy, ds, dcs = w["x"].cuda(), v["dy"].cuda(), v["ds"].cuda(), w["ds"].cuda()

    def run(s, c, stream=None):
        u = c.forward(x, cu, cst, want_state=True, stream=stream)
        s.forward(u, *ops[1:], cu, st, want_state=True, stream=stream)
        du = s.backward(dy, ds, stream=stream)[0]
        c.backward(du, dcs, stream=stream)

    (s, c), (s2, c2) = made
    run(s, c), run(s2, c2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(s, c)
    x.copy_(x.flip(0).clone())
    graph.replay()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    run(s2, c2, side)
    torch.cuda.synchronize()
    for name in ("y", "du", "ddelta", "dB", "dC", "dz", "dA", "dskip", "d_dt_bias", "state_out", "d_state_in"):
        assert torch.equal(getattr(s, name), getattr(s2, name)), name
    for name in ("y", "dx", "dw", "db", "state_out", "d_state_in"):
        assert torch.equal(getattr(c, name), getattr(c2, name)), name


@pytest.mark.parametrize("at", [0, 64, 128])
def test_results_between_the_rows_that_are_read(at):
    """Inputs and outputs that are columns of one wide buffer share none of them."""
    from sparse_moe_layer_topk_gb300 import _lib as M
    T, D, W, wide = 70, 64, 4, 256
    gen = torch.Generator().manual_seed(at)
    buf = torch.randn(T, wide, generator=gen).to(torch.bfloat16).cuda()
    w = torch.randn(D, W, generator=gen).cuda()
    keep = buf.clone()
    x, y = buf[:, 192:], buf[:, at:at + D]
    want = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    call = lambda x, y, ldy: M.moe_conv_fwd(x, w, None, None, None, 1, T, D, W, wide, ldy, True, y, None, None)  # noqa: E731
    call(x, want, D)
    call(x, y, wide)
    assert torch.equal(y, want)
    keep[:, at:at + D] = want
    assert torch.equal(buf, keep)


@pytest.mark.parametrize("B", [1, 5, 61])
@pytest.mark.parametrize("place", ["u", "delta", "z"])
def test_a_step_in_place(B, place):
    """The outputs of the steps over what their own rows are read from."""
    from sparse_moe_layer_topk_gb300 import _lib as M
    D, S, W, G = 520, 16, 4, 2
    gen = torch.Generator().manual_seed(B)
    make = lambda *s, dt=torch.bfloat16: torch.randn(*s, generator=gen).to(dt).cuda()  # noqa: E731
    f32 = torch.float32
    u, delta, z, b, c = make(B, D), make(B, D), make(B, D), make(B, G * S), make(B, G * S)
    A, skip, bias, state = -make(D, S, dt=f32).abs(), make(D, dt=f32), make(D, dt=f32), make(B, D, S, dt=f32)

    def scan(u, delta, z, state, y):
        M.moe_scan_step(u, delta, A, b, c, skip, z, bias, state, None, B, B, D, S, G, D, D, G * S, G * S, D, D, True, y)
        return y

    want, apart, over = torch.empty_like(u), state.clone(), state.clone()
    scan(u, delta, z, apart, want)
    ops = dict(u=u.clone(), delta=delta.clone(), z=z.clone())
    assert torch.equal(scan(**ops, state=over, y=ops[place]), want) and torch.equal(over, apart)

    w, inputs = make(D, W, dt=f32), make(B, W - 1, D)
    apart, over, x = inputs.clone(), inputs.clone(), u.clone()
    M.moe_conv_step(u, w, skip, apart, None, B, B, D, W, D, D, True, want)
    M.moe_conv_step(x, w, skip, over, None, B, B, D, W, D, D, True, x)
    assert torch.equal(x, want) and torch.equal(over, apart)


@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(BF).min, -2e38, -1e30, -130.0, -88.0])
def test_tokens_masked_by_their_time_step(low):
    """A token whose time step is softplus of -infinity, or of the type's lowest value, leaves the state as it is and has no gradient of
    its own: the others get what they get without it. (softplus(-88) is 6e-39: nothing, in a state of fp32.)"""
    from sparse_moe_layer_topk_gb300.scan import SelectiveScan
    lens, D, S = [70, 200, 1, 900], 24, 16
    T, g = sum(lens), torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    u, z, dy, delta = (n(T, D).to(BF) for _ in range(4))
    B, C, A, bias = n(T, 1, S).to(BF), n(T, 1, S).to(BF), -torch.exp(n(D, S)), n(D) - 2
    out = torch.rand(T, generator=g) < 0.3
    out[:2], out[70 + 199], out[270] = True, True, True
    delta[out] = low
    keep = ~out
    at = np.concatenate([[0], np.cumsum(lens)])
    kept = [int(keep[a:b].sum()) for a, b in zip(at[:-1], at[1:])]
    cu, cu_kept = _cu(lens), _cu(kept)

    def run(u, delta, B, C, z, dy, cu, longest):
        s = SelectiveScan(A.cuda(), u.shape[0], n0.cuda(), bias.cuda(), N=len(lens), max_seqlen=longest)
        y = s.forward(u.cuda(), delta.cuda(), B.cuda(), C.cuda(), z.cuda(), cu, want_state=True)
        grads = s.backward(dy.cuda())
        assert int(s.err) == 0
        return s, y, grads

    n0 = n(D)
    dy[out] = 0  # (y of a masked token is C . h all the same; the loss does not see it)
    s, y, grads = run(u, delta, B, C, z, dy, cu, max(lens))
    want = O.scan(*(f64(t) for t in (u, delta.clamp(min=-1e4), A, B, C)), lens, f64(n0), f64(z), f64(bias))
    size = O.scan(*(f64(t) for t in (u.abs(), delta.clamp(min=-1e4), A, B.abs(), C.abs())), lens, f64(n0.abs()), None, f64(bias))
    gate = np.abs(f64(z) * O.sigmoid(f64(z)))
    tol = (900 + 16) * 2.0 ** -21
    _close("y", y, want[0], size[0] * gate, tol)
    _close("state", s.state_out, want[1], size[1], tol, 0)
    t, yk, gk = run(*(v[keep] for v in (u, delta, B, C, z, dy)), cu_kept, max(max(kept), 1))
    rows = keep.cuda()
    norm = torch.linalg.vector_norm
    for name, a, b in zip(("du", "ddelta", "dB", "dC", "dz"), grads, gk):
        a, b = a.float()[rows], b.float()
        # (the tiles lie elsewhere, and sums go another way: a rounding to bf16 apart, 2^-8 of a value at most)
        assert bool(a.isfinite().all()) and float(norm(a - b)) <= 2.0 ** -8 * float(norm(b)), name
    assert not grads[1][out.cuda()].any() or low >= -88.0
    for name in ("dA", "dskip", "d_dt_bias"):
        a, b = getattr(s, name), getattr(t, name)
        assert bool(a.isfinite().all()) and float(norm(a - b)) <= 2.0 ** -10 * float(norm(b)), name


@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(BF).min])
def test_steps_masked_by_their_time_step(low):
    from sparse_moe_layer_topk_gb300.scan import SelectiveScan
    R, D, S, g = 7, 40, 16, torch.Generator().manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    u, delta, z = (n(R, D).to(BF).cuda() for _ in range(3))
    B, C, state = n(R, 1, S).to(BF).cuda(), n(R, 1, S).to(BF).cuda(), n(R, D, S).cuda()
    delta[[1, 4]] = low
    s = SelectiveScan(-torch.exp(n(D, S)).cuda(), R, n(D).cuda(), n(D).cuda(), backward=False)
    before = state.clone()
    y = s.step(u, delta, B, C, z, state)
    assert bool(y.isfinite().all()) and bool(state.isfinite().all())
    # (a decay of no time at all is 1, to the bit that raising the exponential's argument by 2.2e-8 leaves it)
    assert torch.equal(state[[1, 4]], before[[1, 4]]) and not torch.equal(state[0], before[0])


def test_time_steps_that_are_no_numbers_stay_so():
    """softplus(NaN) is NaN, and of +infinity infinite: neither is taken for a number."""
    from sparse_moe_layer_topk_gb300.scan import SelectiveScan
    D, S = 8, 16
    one = torch.ones(4, D, dtype=BF, device="cuda")
    b = torch.ones(4, 1, S, dtype=BF, device="cuda")
    s = SelectiveScan(-torch.ones(D, S, device="cuda"), 4, N=4, backward=False)
    delta = torch.zeros(4, D, dtype=BF, device="cuda")
    delta[1], delta[2] = float("nan"), float("inf")
    y = s.forward(one, delta, b, b)
    assert bool(y[1].isnan().all()) and bool(y[2].isinf().all()) and bool(y[[0, 3]].isfinite().all())


@pytest.mark.parametrize("captured", [False, True])
def test_a_scan_step_directly_behind_its_convolution(captured):
    """The scan's step reads what the convolution's has just written (their starts overlap), row after row and token after token, as a
    decoding loop and as a graph that is replayed: the same bits as with a wait between them."""
    from sparse_moe_layer_topk_gb300.scan import CausalConv, SelectiveScan
    R, D, S, W, steps, g = 61, 1032, 16, 4, 12, torch.Generator().manual_seed(6)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    taps, cb, A, skip, bias = n(D, W).cuda(), n(D).cuda(), -torch.exp(n(D, S)).cuda(), n(D).cuda(), (n(D) - 2).cuda()
    xs = n(steps, R, D).to(BF).cuda()
    delta, z = n(R, D).to(BF).cuda(), n(R, D).to(BF).cuda()
    B, C = n(R, 1, S).to(BF).cuda(), n(R, 1, S).to(BF).cuda()
    idx = torch.randperm(R + 3, generator=g)[:R].to(torch.int32).cuda()
    idx[5] = -1
    first = n(R + 3, W - 1, D).to(BF).cuda(), n(R + 3, D, S).cuda()

    def run(wait):
        conv, scan = CausalConv(taps, cb, R, backward=False), SelectiveScan(A, R, skip, bias, backward=False)
        x, inputs, states, ys = torch.empty_like(xs[0]), first[0].clone(), first[1].clone(), []

        def token():
            v = conv.step(x, inputs, idx)
            if wait:
                torch.cuda.synchronize()
            return scan.step(v, delta, B, C, z, states, idx)
        if captured and not wait:
            x.copy_(xs[0])
            token()  # (kernels' attributes are set outside the capture)
            inputs.copy_(first[0]), states.copy_(first[1])
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                token()
            inputs.copy_(first[0]), states.copy_(first[1])
        for t in range(steps):
            x.copy_(xs[t])
            if captured and not wait:
                graph.replay()
            else:
                token()
            ys.append(scan.y.clone())
        assert int(conv.err) == 0 and int(scan.err) == 0
        return torch.stack(ys), inputs, states

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b) and bool(a.isfinite().all())


@pytest.mark.parametrize("bad", [[], [70], [3, 40, 255]], ids=str)
@pytest.mark.parametrize("longest", [5, 90])
def test_many_short_sequences(bad, longest):
    """Hundreds of sequences, some empty and a few out of place: outputs, last states and gradients are those of the good ones alone."""
    from sparse_moe_layer_topk_gb300.scan import CausalConv, SelectiveScan
    g = torch.Generator().manual_seed(len(bad) + longest)
    N, D = 300, 16
    lens = torch.randint(0, 5, (N,), generator=g)
    lens[torch.randint(0, N, (6,), generator=g)] = longest
    bounds = [0, *lens.cumsum(0).tolist()]
    T = bounds[-1] + 4
    good = [True] * N
    for n in bad:  # a bound behind the one before it: the sequences on either side of it are skipped
        while n == 0 or bounds[n] == bounds[n - 1] or bounds[n] - bounds[n - 1] == bounds[n] + 1:
            n += 1
        bounds[n] = bounds[n - 1] - 1
        good[n - 1] = good[n] = False
    v, w = _scan_inputs([T], D, 16, 1, states=False), _conv_inputs([T], D, 4, False)
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    s = SelectiveScan(v["A"].cuda(), T, v["skip"].cuda(), v["bias"].cuda(), N=N, max_seqlen=90)
    c = CausalConv(w["w"].cuda(), w["b"].cuda(), T, N=N)
    kept = [n for n in range(N) if good[n]]
    rows = [t for n in kept for t in range(bounds[n], bounds[n + 1])]
    left = [bounds[n + 1] - bounds[n] for n in kept]
    other = sorted(set(range(T)) - set(rows))
    for t in (s.y, s.du, s.ddelta, s.dB, s.dC, s.dz, c.y, c.dx, s.state_out, c.state_out):
        t.fill_(7.0)
    y, yc = s.forward(*_operands(v), cu, want_state=True), c.forward(w["x"].cuda(), cu, want_state=True)
    flag = M.MOE_FLAG_BAD_INDEX if bad else 0
    assert int(s.err) == flag and int(c.err) == flag
    grads, gc = s.backward(v["dy"].cuda()), c.backward(w["dy"].cuda())
    for t in (y, yc, gc, *grads):
        assert bool((t[other] == 7.0).all())
    pick = {k: t if k in ("A", "skip", "bias") or t is None else t[rows] for k, t in v.items()}
    r, rc = _scan(pick, left), _conv({**w, "x": w["x"][rows]}, left, True)
    assert torch.equal(r.forward(*_operands(pick), _cu(left), want_state=True), y[rows]) and torch.equal(r.state_out, s.state_out[kept])
    assert torch.equal(rc.forward(w["x"][rows].cuda(), _cu(left), want_state=True), yc[rows]) and torch.equal(rc.state_out, c.state_out[kept])
    for a, b in zip(r.backward(pick["dy"].cuda()), grads):
        assert torch.equal(a, b[rows])
    assert torch.equal(rc.backward(w["dy"][rows].cuda()), gc[rows])
    for a, b in ((r.dA, s.dA), (r.d_dt_bias, s.d_dt_bias), (rc.dw, c.dw), (rc.db, c.db)):
        np.testing.assert_allclose(f64(a), f64(b), rtol=1e-5, atol=1e-4)
    skipped = [n for n in range(N) if not good[n]]
    assert bool((s.state_out[skipped] == 7.0).all()) and bool((c.state_out[skipped] == 7.0).all())


@pytest.mark.parametrize("N", [127, 128, 129, 400])
def test_long_sequences_among_many(N):
    """Sequences that are cut, their sums and joins, behind and between runs of 128 short ones."""
    g = torch.Generator().manual_seed(N)
    lens = torch.randint(0, 4, (N,), generator=g)
    lens[torch.tensor([5, 126, N - 1])] = torch.tensor([900, 333, 1200])
    lens = lens.tolist()
    _check_scan(_scan_inputs(lens, 8, 8, 1), lens)


@pytest.mark.parametrize("W,silu", [(2, True), (2, False), (3, True), (3, False), (4, True), (4, False)])
def test_convolution_of_many_sequences(W, silu):
    lens = [0, 1, 2, 3, 5, 70] * 50
    v = _conv_inputs(lens, 24, W, True)
    c = _conv(v, lens, silu)
    y = c.forward(v["x"].cuda(), _cu(lens), _dev(v["st"]), want_state=True)
    dx = c.backward(v["dy"].cuda(), _dev(v["ds"]))
    args = f64(v["x"]), f64(v["w"]), f64(v["b"]), lens, silu, f64(v["st"])
    size = O.conv(*(np.abs(a) for a in args[:3]), lens, False, np.abs(args[5]))[0]
    want, last = O.conv(*args)
    _close("y", y, want, size, 2.0 ** -18)
    assert np.array_equal(f64(c.state_out), last)
    want = O.conv_backward(f64(v["dy"]), *args, f64(v["ds"]))
    norm = np.linalg.norm
    for got, ref, tol in zip((dx, c.dw, c.db, c.d_state_in), want, (2.0 ** -8, 2.0 ** -16, 2.0 ** -16, 2.0 ** -8)):
        assert norm(f64(got) - ref) <= tol * norm(ref)
    assert int(c.err) == 0
