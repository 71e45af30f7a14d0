"""AdamW on the GPU against the fp64 oracle.

Tolerances. fp32 states: m and v are one or two fp32 operations on exact inputs (|error| <=
2^-22 of the sum of magnitudes); the update divides and takes a root with errors of a few
units (2^-20 of its magnitude, computed with |m|), and the new weight is rounded once more
(2^-22). A clip factor adds its own 2^-21. bf16 weights: one rounding step, 2^-7 of the
magnitude. 8-bit states: each value is one of the two E4M3 neighbours of the exact one, and
the one that the rounding number picks, except where fp32 and fp64 fall on different
sides of the cut (a 2^-20th part of the steps: at most 1e-4 of the values).
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as O
from sparse_moe_layer_topk_gb300 import _lib as M
from gpu_util import f64, need_gpu

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.97, eps=1e-8)
E8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _tensors(sizes, p_dtype, g_dtype, seed=0, offset=0):
    """Weights and gradients; with an offset they are views that start `offset` values into a buffer."""
    g = torch.Generator().manual_seed(seed)
    make = lambda n, s, dt: (s * torch.randn(n + offset, generator=g)).to(dt).cuda()[offset:]  # noqa: E731
    return [make(n, 0.05, p_dtype) for n in sizes], [make(n, 0.2, g_dtype) for n in sizes]


def _adamw(params, grads, **kw):
    from sparse_moe_layer_topk_gb300.optim import AdamW
    return AdamW(params, grads, lr=HYPER["lr"], betas=(HYPER["beta1"], HYPER["beta2"]), eps=HYPER["eps"], **kw)


def _values8(codes, scales):
    c = f64(codes.view(E8).float())
    return c * np.repeat(f64(scales), 256)[:c.size]


def _bounded(name, got, ref, bound):
    err = np.abs(f64(got) - ref)
    assert np.isfinite(f64(got)).all(), name
    assert (err <= bound + 1e-37).all(), f"{name}: {np.max(err / (bound + 1e-37)):.2f} of the bound"


def _check_steps(params, grads, steps, max_norm=0.0, bits=32, master=False, decay=0.1, seed=3):
    opt = _adamw(params, grads, max_norm=max_norm, state_bits=bits, master=master, weight_decay=decay, seed=seed)
    decays = decay if isinstance(decay, list) else [decay] * len(params)
    for step in range(1, steps + 1):
        before = [(f64(opt.master[i] if master else p).ravel(),
                   f64(opt.m[i]) if bits == 32 else _values8(opt.m[i], opt.m_scale[i]),
                   f64(opt.v[i]) if bits == 32 else _values8(opt.v[i], opt.v_scale[i]) ** 2)
                  for i, p in enumerate(params)]
        opt.step()
        torch.cuda.synchronize()
        clip, extra = 1.0, 0.0
        if max_norm > 0:
            norm, clip = O.clip_factor([f64(g) for g in grads], max_norm)
            extra = 2.0 ** -21
            assert abs(float(opt.grad_norm) - norm) <= 2.0 ** -21 * norm
        for i, (p0, m0, v0) in enumerate(before):
            g = f64(grads[i]).ravel()
            if not g.size:
                continue
            args = (step, HYPER["lr"], HYPER["beta1"], HYPER["beta2"], HYPER["eps"], decays[i], clip)
            p, m, v = O.adamw_update(p0, g, m0, v0, *args)
            mag = HYPER["beta1"] * np.abs(m0) + (1 - HYPER["beta1"]) * clip * np.abs(g)
            u = O.rounding_numbers(seed, step, i, g.size)
            if bits == 32:
                _bounded("m", opt.m[i], m, (2.0 ** -22 + extra) * mag)
                _bounded("v", opt.v[i], v, (2.0 ** -22 + 2 * extra) * v)
            else:
                for name, x, codes, scales, k in (("m", m, opt.m[i], opt.m_scale[i], 0),
                                                  ("r", np.sqrt(v), opt.v[i], opt.v_scale[i], 1)):
                    want = O.block_scales(x)
                    np.testing.assert_allclose(f64(scales), want, rtol=2.0 ** -20 + 2 * extra)
                    y = x / np.repeat(want, 256)[:x.size]
                    got = f64(codes.view(E8).float())
                    unit = O.e4m3_unit(y)
                    assert (np.abs(got - y) <= unit * (1 + 2.0 ** -16) + 1e-30).all(), name
                    picked = np.clip(O.round_stochastic(y, unit, u[k]), -448, 448)
                    assert np.mean(got != picked) <= 1e-4 + 1.0 / x.size * (x.size < 10000), name
            size = np.abs(HYPER["lr"] * (mag / (1 - HYPER["beta1"] ** step))
                          / (np.sqrt(v / (1 - HYPER["beta2"] ** step)) + HYPER["eps"]))
            fine = 2.0 ** -22 * np.abs(p0) + (2.0 ** -20 + 2 * extra) * size
            if master and params[i].dtype == BF:
                _bounded("master", opt.master[i], p, fine)
                _bounded("p", params[i].flatten(), p, fine + 2.0 ** -8 * np.abs(p))
                assert torch.equal(params[i].flatten(), opt.master[i].to(BF))
            elif params[i].dtype == BF:
                _bounded("p", params[i].flatten(), p, fine + 2.0 ** -7 * np.abs(p))
                picked = O.round_stochastic(p, np.ldexp(1.0, np.frexp(p)[1] - 8), u[2])
                assert np.mean(f64(params[i]).ravel() != picked) <= 1e-3 + 1.0 / p.size * (p.size < 10000)
            else:
                _bounded("p", params[i].flatten(), p, fine)
    assert int(opt.step_count) == steps and int(opt.err) == 0
    return opt


SIZES = [1, 2, 7, 8, 9, 255, 256, 257, 0, 2047, 2048, 2049, 70_001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_dtype,g_dtype,master", [(F32, F32, False), (F32, BF, False), (BF, F32, True),
                                                    (BF, BF, False), (BF, F32, False)], ids=str)
@pytest.mark.parametrize("max_norm", [0.0, 1.0])
def test_sizes_and_types(bits, p_dtype, g_dtype, master, max_norm):
    _check_steps(*_tensors(SIZES, p_dtype, g_dtype), 3, max_norm=max_norm, bits=bits, master=master)


@pytest.mark.parametrize("offset", [1, 4])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_dtype", [F32, BF], ids=str)
def test_views_with_any_alignment(offset, bits, p_dtype):
    _check_steps(*_tensors([5, 300, 3001], p_dtype, F32, offset=offset), 2, bits=bits, max_norm=0.5)


def test_weights_that_lie_side_by_side():
    """Slices of one buffer without a gap, an empty one between them, and one gradient for two of them."""
    flat = torch.randn(1300, device="cuda")
    g = 0.1 * torch.randn(500, device="cuda")
    _check_steps([flat[:500], flat[500:500], flat[500:1000], flat[1000:]], [g, g[:0], g, g[:300]], 2, max_norm=1.0)


def test_decay_for_each_tensor_and_shapes():
    params, grads = _tensors([600, 600], F32, F32)
    params, grads = [p.view(20, 30) for p in params], [g.view(20, 30) for g in grads]
    _check_steps(params, grads, 2, decay=[0.0, 0.3])


def test_mixed_types_in_one_step():
    a, b = _tensors([5000], F32, BF), _tensors([4097], BF, F32, seed=1)
    opt = _adamw(a[0] + b[0], a[1] + b[1], state_bits=8, master=True, max_norm=1.0)
    opt.step()
    assert opt.master[0] is None and opt.master[1].dtype == F32
    assert torch.equal(b[0][0], opt.master[1].to(BF))


@pytest.mark.parametrize("max_norm", [0.0, 1.0])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
def test_mixed_types_against_the_oracle(bits, master, max_norm):
    """Tensors of different types behind one another, long enough that a warp's run goes from one type's code
    into another's (over 608 chunks of 2,048 values), with this file's bounds for each."""
    kinds = [(700_001, F32, BF), (300, BF, F32), (500_017, BF, BF), (5, F32, F32), (4096, BF, BF), (600_000, F32, F32),
             (257, BF, F32)]
    params, grads = map(list, zip(*((p[0], g[0]) for p, g in (_tensors([n], pt, gt, seed=i)
                                                              for i, (n, pt, gt) in enumerate(kinds)))))
    seed = 11
    opt = _adamw(params, grads, state_bits=bits, master=master, max_norm=max_norm, weight_decay=0.1, seed=seed)
    for step in (1, 2):
        wide = [x if master and x is not None else p for x, p in zip(opt.master or params, params)]
        state = lambda x, sc, i: f64(x[i]) if bits == 32 else _values8(x[i], sc[i])  # noqa: E731
        before = [(f64(wide[i]), state(opt.m, opt.m_scale, i), state(opt.v, opt.v_scale, i) ** (1 if bits == 32 else 2))
                  for i in range(len(kinds))]
        opt.step()
        norm, clip = O.clip_factor([f64(g) for g in grads], max_norm) if max_norm else (0.0, 1.0)
        extra = 2.0 ** -21 if max_norm else 0.0
        if max_norm:
            assert abs(float(opt.grad_norm) - norm) <= 2.0 ** -21 * norm
        for i, (p0, m0, v0) in enumerate(before):
            g = f64(grads[i])
            p, m, v = O.adamw_update(p0, g, m0, v0, step, HYPER["lr"], HYPER["beta1"], HYPER["beta2"], HYPER["eps"], 0.1, clip)
            mag = HYPER["beta1"] * np.abs(m0) + (1 - HYPER["beta1"]) * clip * np.abs(g)
            u = O.rounding_numbers(seed, step, i, g.size)
            if bits == 32:
                _bounded("m", opt.m[i], m, (2.0 ** -22 + extra) * mag)
                _bounded("v", opt.v[i], v, (2.0 ** -22 + 2 * extra) * v)
            else:
                for x, codes, scales, k in ((m, opt.m[i], opt.m_scale[i], 0), (np.sqrt(v), opt.v[i], opt.v_scale[i], 1)):
                    y = x / np.repeat(O.block_scales(x), 256)[:x.size]
                    picked = np.clip(O.round_stochastic(y, O.e4m3_unit(y), u[k]), -448, 448)
                    assert np.mean(f64(codes.float()) != picked) <= 1e-4 + 1.0 / x.size * (x.size < 10000), i
                    np.testing.assert_allclose(f64(scales), O.block_scales(x), rtol=2.0 ** -20 + 2 * extra)
            size = np.abs(HYPER["lr"] * (mag / (1 - HYPER["beta1"] ** step))
                          / (np.sqrt(v / (1 - HYPER["beta2"] ** step)) + HYPER["eps"]))
            fine = 2.0 ** -22 * np.abs(p0) + (2.0 ** -20 + 2 * extra) * size
            if params[i].dtype == F32:
                _bounded("p", params[i], p, fine)
            elif master:
                _bounded("master", opt.master[i], p, fine)
                assert torch.equal(params[i], opt.master[i].to(BF))
            else:
                _bounded("p", params[i], p, fine + 2.0 ** -7 * np.abs(p))
    assert int(opt.step_count) == 2 and int(opt.err) == 0


def test_large_norm_is_one_sum():
    """Twenty million gradients: the fp32 partial sums keep the norm to 2^-21."""
    _check_steps(*_tensors([20_000_003, 17], F32, BF), 1, max_norm=1.0)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("g_dtype", [F32, BF], ids=str)
@pytest.mark.parametrize("big,max_norm", [(1e19, 1.0), (1e20, 1.0), (-3e25, 1e5), (3e38, 1e12)])
def test_a_finite_norm_whose_squares_pass_fp32(big, max_norm, g_dtype, bits):
    """The step is taken and clipped: a norm counts as not finite only where itself is past fp32."""
    params, grads = _tensors([3000, 17], F32, g_dtype)
    grads[0][1234] = big
    grads[1][3] = big / 2
    if bits == 32:
        _check_steps(params, grads, 2, max_norm=max_norm)
        return
    # (clipped, the other values' v lies below fp32's normal numbers, and with it what 8-bit r can be held to)
    opt = _adamw(params, grads, max_norm=max_norm, state_bits=8)
    for step in (1, 2):
        opt.step()
        norm, clip = O.clip_factor([f64(g) for g in grads], max_norm)
        assert abs(float(opt.grad_norm) - norm) <= 2.0 ** -21 * norm
        assert int(opt.step_count) == step and int(opt.err) == 0
    for i, at in ((0, 1234), (1, 3)):
        want = (1 - HYPER["beta1"] ** 2) * clip * f64(grads[i])[at]  # two steps' m, rounded twice to E4M3
        assert abs(_values8(opt.m[i], opt.m_scale[i])[at] - want) <= 2 * 2.0 ** -3 * abs(want)
        assert bool(torch.isfinite(params[i]).all())


def test_a_norm_past_fp32_is_not_finite():
    params, grads = _tensors([3000], F32, F32)
    grads[0][:2] = 3e38
    opt, was = _adamw(params, grads, max_norm=1.0), params[0].clone()
    opt.step()
    assert int(opt.err) == M.MOE_FLAG_NONFINITE and int(opt.step_count) == 0 and torch.equal(params[0], was)


@pytest.mark.parametrize("p_dtype,master", [(F32, False), (BF, True), (BF, False)], ids=str)
@pytest.mark.parametrize("n", [600, 603])
def test_a_second_moment_past_fp32_leaves_the_weight_to_its_decay(n, p_dtype, master):
    """v = inf takes the update to zero and not the weight to NaN, at this step and the next."""
    params, grads = _tensors([n], p_dtype, F32)
    grads[0][300], grads[0][n - 1] = 1e21, -3e25
    opt = _adamw(params, grads, master=master, weight_decay=0.5)
    keep = 1 - HYPER["lr"] * 0.5
    for step in (1, 2):
        before = f64(opt.master[0] if master else params[0])
        opt.step()
        got = f64(opt.master[0] if master else params[0])
        for at in (300, n - 1):
            assert float(opt.v[0][at]) == float("inf") and np.isfinite(float(opt.m[0][at]))
            # one rounding of the weight, or one step of bf16
            assert abs(got[at] - keep * before[at]) <= (2.0 ** -7 if p_dtype == BF and not master else 2.0 ** -22) * abs(before[at])
        assert np.isfinite(got).all() and int(opt.step_count) == step


def test_a_second_moment_past_fp32_in_8_bits_is_lost_alone():
    params, grads = _tensors([600], F32, F32)
    grads[0][300] = 1e21
    opt = _adamw(params, grads, state_bits=8)
    opt.step()
    other = torch.arange(600, device="cuda") != 300
    assert bool(torch.isnan(params[0][300])) and bool(torch.isfinite(params[0][other]).all())


def test_no_clipping_below_the_norm():
    params, grads = _tensors([1000], F32, F32)
    a = _check_steps([params[0].clone()], grads, 1, max_norm=1e6)
    b = _check_steps([params[0].clone()], grads, 1)
    assert torch.equal(a.params[0], b.params[0])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_clipped_step_with_a_bad_gradient_changes_nothing(bad, bits):
    params, grads = _tensors([3000, 40], BF, F32)
    opt = _check_steps(params, grads, 2, bits=bits, master=True, max_norm=1.0)
    lists = [params, opt.m, opt.v, opt.master] + ([opt.m_scale, opt.v_scale] if bits == 8 else [])
    keep = [[t.clone() for t in ts] for ts in lists]
    grads[1][7] = bad
    opt.step()
    torch.cuda.synchronize()
    assert int(opt.err) == M.MOE_FLAG_NONFINITE and int(opt.step_count) == 2
    for ts, old in zip(lists, keep):
        for t, o in zip(ts, old):
            assert torch.equal(t.view(torch.uint8), o.view(torch.uint8))
    grads[1][7] = 0.1
    opt.err.zero_()
    opt.step()
    assert int(opt.err) == 0 and int(opt.step_count) == 3


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_without_a_clip_bad_values_stay_in_their_place(bad):
    """8 bits: the value gets the NaN code, the rest of its block keeps its scale and values."""
    a, ga = _tensors([600], F32, F32)
    b = [a[0].clone()]
    opt_a = _adamw(a, ga, state_bits=8)
    opt_a.step()
    gb = [ga[0].clone()]
    gb[0][300] = bad
    opt_b = _adamw(b, gb, state_bits=8)
    opt_b.step()
    other = torch.arange(600, device="cuda") != 300
    mb, ma = opt_b.m[0].float(), opt_a.m[0].float()
    assert torch.isnan(mb[300]) and torch.isnan(opt_b.v[0].float()[300])
    if abs(ga[0][300]) < ga[0][256:512].abs().max():  # it did not set its block's scale
        assert torch.equal(mb[other], ma[other]) and torch.equal(a[0][other], b[0][other])


def test_zero_gradients_and_zero_states():
    params, grads = _tensors([700], F32, F32)
    grads[0].zero_()
    for bits in (32, 8):
        p = params[0].clone()
        opt = _adamw([p], grads, state_bits=bits, weight_decay=0.0, max_norm=1.0)
        opt.step()
        assert torch.equal(p, params[0]) and float(opt.grad_norm) == 0.0
        assert (opt.m[0].float() == 0).all() and (opt.v[0].float() == 0).all()


def test_results_repeat_bit_for_bit_and_seeds_differ():
    outs = []
    for seed in (1, 1, 2):
        params, grads = _tensors([100_000], BF, F32)
        opt = _adamw(params, grads, state_bits=8, max_norm=1.0, seed=seed)
        for _ in range(3):
            opt.step()
        outs.append((params[0].clone(), opt.m[0].view(torch.uint8).clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert not torch.equal(outs[0][1], outs[2][1])


def test_stochastic_rounding_does_not_freeze_the_second_moment():
    """With beta2 = 0.999 and no gradient sqrt(v) shrinks by 0.05% a step, far below a step of its
    format; on average over the values it still does."""
    from sparse_moe_layer_topk_gb300.optim import AdamW
    n, steps = 51200, 200
    p, g = [torch.zeros(n, device="cuda")], [torch.full((n,), 0.01, device="cuda")]
    opt = AdamW(p, g, lr=0.0, betas=(0.9, 0.999), state_bits=8)
    opt.step()
    g[0].copy_(0.01 * torch.rand(n, device="cuda"))
    opt.step()
    first = _values8(opt.v[0], opt.v_scale[0])
    g[0].zero_()
    for _ in range(steps):
        opt.step()
    # each value's rounding errors have zero mean; over n values the mean has 1 / sqrt(n) of their spread
    assert abs(_values8(opt.v[0], opt.v_scale[0]).mean() / first.mean() / 0.999 ** (steps / 2) - 1) < 0.02


def test_captured_steps_count_and_follow_the_schedule():
    params, grads = _tensors([5000], BF, F32)
    twin = [params[0].clone()]
    opt, ref = _adamw(params, grads, master=True, max_norm=1.0), _adamw(twin, grads, master=True, max_norm=1.0)
    lr = torch.tensor([HYPER["lr"]], device="cuda")
    opt.schedule_on_device(lr)
    opt.step()
    ref.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    for k in range(3):
        lr.fill_(HYPER["lr"] / (k + 1))
        graph.replay()
        ref.lr = float(torch.tensor(HYPER["lr"] / (k + 1)))
        ref.step()
    torch.cuda.synchronize()
    assert int(opt.step_count) == 4
    assert torch.equal(opt.master[0], ref.master[0]) and torch.equal(params[0], twin[0])


def test_state_dict_round_trip():
    params, grads = _tensors([3000, 11], BF, BF)
    opt = _check_steps(params, grads, 2, bits=8, master=True)
    d, w = opt.state_dict(), [p.clone() for p in params]
    opt.step()
    want = [p.clone() for p in params]
    for p, old in zip(params, w):
        p.copy_(old)
    again = _adamw(params, grads, state_bits=8, master=True, weight_decay=0.1, seed=3)
    again.load_state(**d)
    again.step()
    assert int(again.step_count) == 3
    for p, x in zip(params, want):
        assert torch.equal(p, x)


@pytest.mark.parametrize("change", [dict(m=-1), dict(v=-1), dict(m_scale=-1), dict(v_scale=-1), dict(master=-1),
                                    dict(master=0), dict(v=1), dict(v_scale=1)], ids=str)
def test_a_state_that_does_not_fit_is_not_taken_over_in_part(change):
    """A list without its last entry (-1), an entry missing (0), one of another size (1)."""
    params, grads = _tensors([3000, 11], BF, BF)
    opt = _check_steps(params, grads, 2, bits=8, master=True)
    (name, how), = change.items()
    was, d = opt.state_dict(), opt.state_dict()
    for xs in (d["m"], d["v"]):
        for x in xs:
            x.zero_()
    d["step"] = 7
    d[name] = d[name][:-1] if how == -1 else [d[name][0], None if how == 0 else d[name][1][:-1]]
    with pytest.raises(ValueError, match=name):
        opt.load_state(**d)
    now = opt.state_dict()
    assert now["step"] == was["step"] == 2
    for n in ("m", "v", "m_scale", "v_scale", "master"):
        for a, b in zip(now[n], was[n]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_parameters_of_a_module():
    """torch.nn.Parameter weights: the master copies stay out of autograd, and a state loads without no_grad."""
    params, grads = _tensors([3000, 11], BF, F32)
    params = [torch.nn.Parameter(p) for p in params]
    opt = _adamw(params, grads, master=True, max_norm=1.0)
    assert not any(x.requires_grad for x in opt.master)
    opt.step()
    opt.load_state(**opt.state_dict())
    opt.load_state(1, opt.m, opt.v)
    assert torch.equal(opt.master[0], params[0].detach().float())


@pytest.mark.parametrize("bits,master", [(8, False), (8, True), (32, False)])
def test_a_resumed_run_rounds_as_the_run_it_resumes(bits, master):
    """The rounding numbers' seed is part of the state."""
    params, grads = _tensors([3000], BF, F32)
    opt = _adamw(params, grads, state_bits=bits, master=master, seed=12345)
    opt.step()
    twin, d = [params[0].clone()], opt.state_dict()
    again = _adamw(twin, grads, state_bits=bits, master=master)
    again.load_state(**d)
    opt.step()
    again.step()
    assert torch.equal(params[0], twin[0])
    assert torch.equal(opt.m[0].view(torch.uint8), again.m[0].view(torch.uint8))


def test_a_tensor_past_32_bits():
    """Indexes past 2^31 reach their own values (bf16, 8-bit states)."""
    n = (1 << 31) + 5000
    p, g = torch.zeros(n, dtype=BF, device="cuda"), torch.zeros(n, dtype=BF, device="cuda")
    g[-4000:] = 0.25
    opt = _adamw([p], [g], state_bits=8)
    opt.step()
    # first step: update = lr * g / (|g| + eps), so -lr in bf16's neighbours
    lr = HYPER["lr"]
    assert ((p[-4000:].float() + lr).abs() <= 2.0 ** -7 * lr).all()
    assert int((p[:-4000] != 0).sum()) == 0


def test_class_refusals():
    p, g = _tensors([10], F32, F32)
    for bad in (([], []), (p, []), (p, [g[0][:5]]), (p, [g[0].half()]), (p, [g[0].cpu()])):
        with pytest.raises(ValueError):
            _adamw(*bad)
    with pytest.raises(ValueError):
        _adamw([torch.zeros(4, 4, device="cuda").t()], [torch.zeros(4, 4, device="cuda")[:, :].t()])
    with pytest.raises(ValueError):
        _adamw(p, g, state_bits=4)
    with pytest.raises(ValueError):
        _adamw(p, g, weight_decay=[0.1, 0.2])
    opt = _adamw(p, g, state_bits=8)
    with pytest.raises(ValueError):
        opt.load_state(1, opt.m, opt.v)
