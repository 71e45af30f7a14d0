"""Routing with scores, bias and groups on the GPU against the fp64 oracle.

Ids are exact: the choice is that of 64-bit values. Scores and weights are fp32 of a few operations on exact logits,
the exponential's argument up to 100 in magnitude (2^-24 of it): within 2^-17 of their values.
"""
import numpy as np
import pytest
import torch

from oracle import mixer_oracle as O
from sparse_moe_layer_topk_gb300 import _lib as M
from gpu_util import f64, need_gpu

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _router(*a, **k):
    from sparse_moe_layer_topk_gb300.route import Router
    return Router(*a, **k)


def _check(logits, bias, k, score="sigmoid", renorm=True, scale=1.0, flag=0, **groups):
    T, E = logits.shape
    r = _router(T, E, k, score=score, renorm=renorm, scale=scale, **groups)
    idx, w = r.forward(logits.cuda(), None if bias is None else bias.cuda())
    torch.cuda.synchronize()
    want = O.route(f64(logits), None if bias is None else f64(bias), k, score, renorm=renorm, scale=scale, **groups)
    np.testing.assert_array_equal(idx.cpu().numpy(), want[0])
    np.testing.assert_allclose(f64(w), want[1], rtol=TOL, atol=1e-37)
    np.testing.assert_allclose(f64(r.topk_s), want[2], rtol=TOL, atol=1e-37)
    assert int(r.err) == flag
    return r


def _logits(T, E, seed=0, std=1.5):
    return std * torch.randn(T, E, generator=torch.Generator().manual_seed(seed))


def _bias(E, seed=0, std=0.05):
    return std * torch.randn(E, generator=torch.Generator().manual_seed(seed + 1000))


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 3), (5, 8, 8), (2, 33, 32), (7, 64, 6), (9, 100, 7), (4, 255, 31), (33, 896, 16),
                                   (5, 1024, 32), (3, 1023, 17), (2, 36, 32), (3, 896, 32)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_without_groups(T, E, k, score, bias, renorm):
    _check(_logits(T, E, E + k), _bias(E, k) if bias else None, k, score, renorm, 2.5 if renorm else 1.0)


@pytest.mark.parametrize("E,groups,group_k,k", [(896, 8, 4, 16), (896, 8, 1, 32), (896, 7, 3, 9), (896, 14, 13, 16), (256, 8, 4, 8), (60, 4, 2, 6),
                                                (1024, 32, 5, 32), (1024, 32, 31, 3), (1000, 5, 2, 32), (96, 32, 1, 3), (8, 2, 1, 4), (64, 4, 4, 8),
                                                (35, 5, 2, 14), (32, 32, 8, 8), (1023, 3, 2, 20), (1020, 17, 9, 32)])
@pytest.mark.parametrize("score,bias,group_top", [("sigmoid", True, 2), ("sigmoid", False, 2), ("softmax", True, 1),
                                                  ("softmax", False, 2), ("sigmoid", False, 1), ("softmax", True, 2)])
def test_groups(E, groups, group_k, k, score, bias, group_top):
    _check(_logits(21, E, E + groups), _bias(E, k) if bias else None, k, score, groups=groups, group_k=group_k, group_top=group_top)


@pytest.mark.parametrize("groups,group_k", [(1, 1), (8, 3), (7, 2)])
@pytest.mark.parametrize("bias", [None, "zero", "some", "two"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_rows_of_equal_logits(groups, group_k, bias, score):
    """A padded batch: the same logit everywhere, so that only the bias and the order of the experts choose."""
    l = torch.cat([torch.zeros(5, 896), torch.full((3, 896), -3.25), _logits(3, 896)])
    b = {None: None, "zero": torch.zeros(896), "some": _bias(896), "two": (torch.arange(896) % 3 == 0).float() * 0.125}[bias]
    _check(l, b, 16, score, groups=groups, group_k=group_k)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,group_k", [(1, 1), (8, 4)])
def test_values_nearer_than_32_bits_tell_apart(score, groups, group_k):
    """Score and bias meet: bias = const - score up to a few 2^-24 of noise, so that the order lies below fp32's
    rounding of the sums, and many pairs differ in logit and bias yet nearly not in their sum."""
    g = torch.Generator().manual_seed(5)
    l = torch.randn(40, 896, generator=g).repeat_interleave(3, 0)[:64]
    s = torch.sigmoid(l.double()) if score == "sigmoid" else torch.softmax(l.double(), 1)
    b = (0.75 - s[0] + 1e-8 * torch.randn(896, generator=g, dtype=torch.float64)).float()
    _check(l, b, 16, score, groups=groups, group_k=group_k)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,group_k", [(1, 1), (4, 2)])
@pytest.mark.parametrize("by", ["logit", "bias"])
def test_experts_out_of_service(score, groups, group_k, by):
    """-infinity takes an expert out; where too few others are left, such experts fill the list with weight 0."""
    l, b = _logits(12, 64, 3), _bias(64)
    out = torch.rand(12, 64, generator=torch.Generator().manual_seed(8)) < torch.linspace(0.05, 1.0, 12)[:, None]
    out[-1] = True
    if by == "logit":
        l[out] = -torch.inf
    else:
        b[out[6]] = -torch.inf
    r = _check(l, b if by == "bias" else None, 8, score, groups=groups, group_k=group_k)
    assert not r.topk_w.isnan().any()


def test_values_that_are_no_numbers_are_flagged_and_taken_out():
    for bad in (float("nan"), float("inf")):
        l = _logits(4, 128)
        l[2, 7] = bad
        r = _check(l, None, 8, flag=M.MOE_FLAG_NONFINITE)
        assert 7 not in r.topk_idx[2].tolist()
        b = _bias(128)
        b[9] = bad
        r = _check(_logits(4, 128), b, 8, "softmax", flag=M.MOE_FLAG_NONFINITE)
        assert 9 not in r.topk_idx.flatten().tolist()


def test_extreme_logits():
    l = torch.tensor([[-100.0, -101.0, -102.5, -90.0] * 16, [100.0, 99.0, 80.0, -3e38] * 16, [3e38, 1.0, -3e38, 0.0] * 16,
                      [-300.0, -301.0, -302.0, -303.0] * 16])
    for score in ("sigmoid", "softmax"):
        _check(l[[0, 3]], None, 6, score)
    r = _router(4, 64, 6)
    idx, w = r.forward(l.cuda())
    np.testing.assert_allclose(f64(w).sum(1), 1.0, rtol=1e-6)
    assert idx[1].tolist() == [0, 4, 8, 12, 16, 20]


@pytest.mark.parametrize("E", [64, 100, 896, 1023])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient(E, score, renorm, dtype):
    """fp32: within 2^-17 of the terms of each entry (g_j and the weighted sum of all g); bf16: a rounding more, 2^-8."""
    T, k = 37, 7
    l, g = _logits(T, E, E), torch.randn(T, k, generator=torch.Generator().manual_seed(1))
    l[3, 5:9] = -torch.inf
    r = _router(T, E, k, score=score, renorm=renorm, scale=2.5, grad_dtype=dtype)
    r.forward(l.cuda(), _bias(E).cuda())
    idx, w, s = r.topk_idx.cpu().numpy(), f64(r.topk_w), f64(r.topk_s)
    got = f64(r.backward(g.cuda()))
    args = f64(g), f64(l), idx, w, s, score, renorm, 2.5
    want = O.route_backward(*args)
    size = np.abs(want)
    if renorm:
        np.put_along_axis(size, idx.astype(np.int64), w * (np.abs(f64(g)) + (w * np.abs(f64(g))).sum(1, keepdims=True) / 2.5), 1)
    elif score == "softmax":
        size = size + 2.5 * O.scores(f64(l), score) * (s * np.abs(f64(g))).sum(1, keepdims=True)
    bound = TOL * size + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0) + 1e-37
    assert (np.abs(got - want) <= bound).all()
    assert int(r.err) == 0


def test_gradient_from_permuted_rows():
    T, E, k = 20, 64, 4
    r = _router(T, E, k)
    r.forward(_logits(T, E).cuda())
    slot = torch.randperm(T * k, generator=torch.Generator().manual_seed(0)).to(torch.int32).view(T, k)
    slot[3, 1] = -1
    rows = torch.randn(T * k, generator=torch.Generator().manual_seed(2))
    d_w = torch.empty(T, k, device="cuda")
    got = r.backward(rows.cuda(), slot.cuda(), d_w).clone()
    want = torch.where(slot >= 0, rows[slot.long().clamp(min=0)], 0.0)
    assert torch.equal(d_w.cpu(), want)
    assert torch.equal(r.backward(want.cuda()), got)


@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("softmax", False)])
def test_gradient_of_bad_and_repeated_ids(score, renorm):
    """An id out of range and one that its row names twice are flagged, and nothing is written out of bounds."""
    T, E, k = 6, 64, 4
    r = _router(T, E, k, score=score, renorm=renorm)
    r.forward(_logits(T, E).cuda())
    d_w = torch.ones(T, k, device="cuda")
    good = r.backward(d_w).clone()
    assert int(r.err) == 0
    r.topk_idx[1, 2] = E
    r.topk_idx[2, 3] = -5
    r.topk_idx[4, 3] = r.topk_idx[4, 0]
    got = r.backward(d_w)
    assert int(r.err) == M.MOE_FLAG_BAD_EXPERT
    rows = [0, 3, 5]
    assert torch.equal(got[rows], good[rows]) and bool(got.isfinite().all())


def test_no_tokens():
    r = _router(0, 64, 4)
    idx, w = r.forward(torch.empty(0, 64, device="cuda"))
    assert idx.shape == (0, 4) and r.backward(torch.empty(0, 4, device="cuda")).shape == (0, 64)


def test_in_a_graph_and_on_another_stream():
    T, E, k = 300, 896, 16
    l, b, g = _logits(T, E).cuda(), _bias(E).cuda(), torch.randn(T, k, device="cuda")
    kw = dict(score="softmax", renorm=False, groups=8, group_k=4)
    r = _router(T, E, k, **kw)
    r.forward(l, b), r.backward(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.forward(l, b), r.backward(g)
    l.copy_(_logits(T, E, 7).cuda())
    graph.replay()
    side = torch.cuda.Stream()
    other = _router(T, E, k, **kw)
    torch.cuda.synchronize()
    other.forward(l, b, stream=side), other.backward(g, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(r.topk_idx, other.topk_idx) and torch.equal(r.topk_w, other.topk_w)
    assert torch.equal(r.d_logits, other.d_logits)


@pytest.mark.parametrize("groups,group_k", [(1, 1), (8, 4)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_logits_at_both_ends_of_the_range(score, groups, group_k):
    """Differences of logits that pass the largest float, next to experts that only 64 bits tell apart."""
    l = _logits(9, 256, 3)
    l[:, ::5] = -3e38
    l[3:6, 7] = 3e38
    b = torch.full((256,), 0.25)
    b[1::3] += 2.0 ** -24
    _check(l, b, 12, score, groups=groups, group_k=group_k)


def test_more_tokens_than_lanes_number_in_32_bits():
    T = 2 ** 27 + 9  # (x 32 lanes is more than 2^32)
    logits = torch.zeros(T, 2, device="cuda")
    logits[::3, 1] = 1.0
    r = _router(T, 2, 1, renorm=False, grad_dtype=torch.bfloat16)
    idx, w = r.forward(logits)
    assert torch.equal(idx[:, 0].long(), logits.argmax(1))
    one = 1 / (1 + np.exp(-1.0))
    assert float((w[::3] - one).abs().max()) < 1e-6 and float((w[1::3] - 0.5).abs().max()) < 1e-6
    d = r.backward(torch.ones_like(w))
    # d sigmoid: 0.25 at 0, 0.1966 at 1, rounded to 8 bits
    assert bool((d[1::3, 0] == 0.25).all()) and float((d[::3, 1].float() - one * (1 - one)).abs().max()) < 2.0 ** -11
    assert not d[1::3, 1].any() and not d[::3, 0].any()


@pytest.mark.parametrize("groups,group_k", [(1, 1), (8, 4)])
def test_logits_and_biases_that_start_anywhere(groups, group_k):
    """Rows and biases of a multiple of four values that begin on four bytes."""
    logits, bias = _logits(9, 256, 5), _bias(256, 5)
    for at_l, at_b in ((0, 1), (1, 0), (3, 2)):
        l, b = torch.zeros(9 * 256 + at_l, device="cuda"), torch.zeros(256 + at_b, device="cuda")
        l, b = l[at_l:].view(9, 256).copy_(logits), b[at_b:].copy_(bias)
        _check(l, b, 8, groups=groups, group_k=group_k)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_biases_whose_sums_pass_32_bits(score):
    """Groups whose two largest values add up to more than the largest float."""
    b = torch.cat([torch.full((16,), v) for v in (2.0e38, 2.5e38, -3e38, 2.25e38)])
    _check(_logits(6, 64, 8), b, 6, score, groups=4, group_k=2)


@pytest.mark.parametrize("k", [17, 20, 25, 31, 32])
@pytest.mark.parametrize("E,groups,group_k", [(896, 1, 1), (1000, 5, 3), (64, 1, 1), (100, 1, 1), (256, 8, 4)])
@pytest.mark.parametrize("score,bias", [("sigmoid", False), ("sigmoid", True), ("softmax", True)])
def test_many_experts_a_token(E, groups, group_k, k, score, bias):
    """More than 16, where the lanes' largest values alone do not bound them: values of their own, of few levels, all but some the
    same, and masked."""
    l = _logits(24, E, E + k)
    l[6:12] = (l[6:12] * 4).round() / 4  # many equal values
    l[12:18] = torch.where(torch.arange(E) % 7 == 0, l[12:18], torch.tensor(-0.5))
    l[18:20, E // 3:] = -torch.inf
    l[20:22] = 0.25
    l[22:, ::2] = -torch.inf
    b = (_bias(E, k) * 8).round() / 8 if bias else None
    _check(l, b, k, score, groups=groups, group_k=group_k)


@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("softmax", True), ("softmax", False)])
def test_slots_that_do_not_exist(score, renorm):
    """A dropped row's slot is negative; one behind the last row is flagged. Both have no gradient of their own."""
    T, E, k = 11, 60, 4
    r = _router(T, E, k, score=score, renorm=renorm)
    r.forward(_logits(T, E, 2).cuda())
    g = torch.randn(T * k, generator=torch.Generator().manual_seed(3)).cuda()
    slots = torch.randperm(T * k, generator=torch.Generator().manual_seed(4)).to(torch.int32).view(T, k)
    slots[1, 2] = slots[5, 0] = -1
    by_token = torch.where(slots >= 0, g.cpu()[slots.clamp(min=0).long()], torch.tensor(0.0)).cuda()
    want = r.backward(by_token).clone()
    seen = torch.empty(T, k, device="cuda")
    assert torch.equal(r.backward(g, slots.cuda(), seen), want) and torch.equal(seen, by_token) and int(r.err) == 0
    slots[5, 0] = T * k
    assert torch.equal(r.backward(g, slots.cuda(), seen), want) and torch.equal(seen, by_token)
    assert int(r.err) == M.MOE_FLAG_BAD_INDEX


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,group_k", [(8, 4), (7, 2), (32, 8)])
def test_groups_by_one_value_that_32_bits_cannot_tell(score, groups, group_k):
    """group_top = 1: a group's largest value is found in 64 bits where members lie within fp32's rounding of one another."""
    g = torch.Generator().manual_seed(5)
    l = torch.randn(40, 896, generator=g).repeat_interleave(3, 0)[:64]
    s = torch.sigmoid(l.double()) if score == "sigmoid" else torch.softmax(l.double(), 1)
    b = (0.75 - s[0] + 1e-8 * torch.randn(896, generator=g, dtype=torch.float64)).float()
    _check(l, b, 16, score, groups=groups, group_k=group_k, group_top=1)


@pytest.mark.parametrize("bias", [0.0, 64.0, -1000.0])
@pytest.mark.parametrize("groups,group_k,group_top", [(8, 4, 1), (8, 4, 2), (5, 2, 1), (32, 7, 1), (1, 1, 1)])
def test_scores_next_to_one_and_biases_that_quantise_them(bias, groups, group_k, group_top):
    """Sigmoid scores that are all 1 in fp32, or equal once a large bias is added."""
    l = 15 + 14 * torch.rand(48, 160, generator=torch.Generator().manual_seed(7))
    l[40:] = l[40:, :1]  # padded rows: one logit everywhere
    _check(l, torch.full((160,), bias), 5, groups=groups, group_k=group_k, group_top=group_top)
    l = torch.tensor([[18.0, 30.0, 25.0, 20.0]])
    if groups == 8:
        _check(l, torch.full((4,), bias), 1, groups=2, group_k=1, group_top=group_top)


@pytest.mark.parametrize("bias", ["zero", "some", "two"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_rows_of_equal_logits_by_one_value(bias, score):
    l = torch.cat([torch.zeros(5, 896), torch.full((3, 896), -3.25), _logits(3, 896)])
    b = {"zero": torch.zeros(896), "some": _bias(896), "two": (torch.arange(896) % 3 == 0).float() * 0.125}[bias]
    for groups, group_k in ((8, 3), (7, 2), (32, 20)):
        _check(l, b, 16, score, groups=groups, group_k=group_k, group_top=1)


@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("groups,group_k", [(8, 4), (16, 3)])
def test_members_on_either_side_of_a_rounding(group_top, groups, group_k):
    """Scores within a few 2^-24 of the middle between two sums of fp32: which of a group's members comes second is not what their
    rounded sums say."""
    g = torch.Generator().manual_seed(11)
    size, T = 128 // groups, 400
    middle = 0.5 + 2.0 ** -18  # (100.5 and 100.5 + 2^-17 are neighbours)
    l = np.log(middle / (1 - middle)) + 4e-7 * torch.randn(T, groups, size, generator=g, dtype=torch.float64)
    l = l + 8e-7 * (2 * torch.rand(T, 1, 1, generator=g, dtype=torch.float64) - 1)
    if group_top == 2:
        l[:, :, 0] = 2.0
    l[:, :, 4:] = -5.0
    _check(l.float().view(T, 128), torch.full((128,), 100.0), 8, groups=groups, group_k=group_k, group_top=group_top)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_members_whose_scores_round_differently(score, group_top):
    """As above, with scores of different sizes and biases that make up for it: each score has an error of its own."""
    g = torch.Generator().manual_seed(14)
    T, groups, size = 1500, 8, 8
    rand = lambda *s: torch.rand(*s, generator=g, dtype=torch.float64)  # noqa: E731
    noise = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    unit = 2.0 ** -17 if score == "sigmoid" else 2.0 ** -24  # between two sums next to 100.5, or to 0.75
    steps = torch.round((0.2 + 0.6 * rand(groups, size)) / unit if score == "sigmoid" else (0.003 + 0.006 * rand(groups, size)) / unit)
    b = (100.5 if score == "sigmoid" else 0.75) - steps * unit
    scatter = 1e-7 if score == "sigmoid" else 1e-9
    s = (steps + 0.5) * unit + scatter * noise(T, groups, size) + 2 * scatter * (2 * rand(T, 1, 1) - 1)
    if group_top == 2:
        b[:, 0] = 101 if score == "sigmoid" else 1
        s[:, :, 0] = 0.5 if score == "sigmoid" else 0.004
    s[:, :, 4:] *= 0.01
    if score == "sigmoid":
        l = torch.log(s / (1 - s)).view(T, 64)
    else:  # (an expert that is never chosen takes the rest of the row)
        s = s.view(T, 64)
        s[:, 63] = 0
        s[:, 63] = 1 - s.sum(1)
        b[-1, -1] = -10
        l = torch.log(s)
    _check(l.float(), b.float().view(64), 6, score, groups=groups, group_k=4, group_top=group_top)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_two_members_on_either_side_of_a_rounding(score):
    """Two groups whose second member is one of two that differ by less than the error of their scores, while their sums with the bias
    are neighbours in fp32, further apart than any score's error."""
    g = torch.Generator().manual_seed(15)
    T, E = 6000, 1024
    rand = lambda *s: torch.rand(*s, generator=g, dtype=torch.float64)  # noqa: E731
    unit, sums, scatter = (2.0 ** -17, 100.5, 5e-8) if score == "sigmoid" else (2.0 ** -24, 0.75, 1.5e-10)
    span = 0.2 + 0.6 * rand(2, 2) if score == "sigmoid" else 0.0007 + 0.0004 * rand(2, 2)
    steps = torch.round(span / unit)
    b, s = torch.zeros(2, E // 2, dtype=torch.float64), torch.full((T, 2, E // 2), 0.01 if score == "sigmoid" else 0.0, dtype=torch.float64)
    b[:, 1:3] = sums - steps * unit
    s[:, :, 1:3] = (steps + 0.5) * unit + scatter * torch.randn(T, 2, 2, generator=g, dtype=torch.float64)
    b[:, 0], s[:, :, 0] = sums + 0.25, 0.001
    if score == "softmax":
        s[:, :, 3:] = ((1 - s.sum((1, 2))) / (E - 6))[:, None, None]
    l = torch.log(s / (1 - s)) if score == "sigmoid" else torch.log(s) + 7
    _check(l.float().view(T, E), b.float().view(E), 2, score, groups=2, group_k=1, group_top=2)


def test_groups_of_opposite_biases():
    """The two largest members of a group cancel: the sum is small, and its error that of its terms."""
    g = torch.Generator().manual_seed(12)
    T, groups, size = 400, 8, 8
    middle = 0.5 + 2.0 ** -18
    l = np.log(middle / (1 - middle)) + 4e-6 * torch.randn(T, groups, size, generator=g, dtype=torch.float64)
    b = torch.full((groups, size), -100.0)
    b[:, 0] = 100.0
    _check(l.float().view(T, 64), b.view(64), 6, groups=groups, group_k=4)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("k", [1, 3])
@pytest.mark.parametrize("groups,group_k", [(1, 1), (2, 1)])
def test_a_large_score_beside_small_ones(score, k, groups, group_k):
    """An expert whose bias all but cancels its large score ends within that score's rounding of experts with small scores, which fp32
    tells apart far more finely."""
    rng, T, E = np.random.default_rng(13), 3000, 64
    f32 = lambda x: np.asarray(x, dtype=np.float32).astype(np.float64)  # noqa: E731
    sig = lambda x: 1 / (1 + np.exp(-x))  # noqa: E731
    target = sig(-7.0)
    cs = np.arange(8, 32, 4)
    bias = np.zeros(E)
    bias[cs] = f32(target - rng.uniform(0.55, 0.8, cs.size))
    bias[30] = -10.0  # takes up the rest of a softmax, and is never chosen
    l = np.full((T, E), -40.0)
    c = rng.choice(cs, T)
    rows = np.arange(T)
    p = target - bias[c] + 3e-7 * rng.standard_normal(T)  # what the expert's score should be
    near = 8e-9 * rng.standard_normal(T)
    if score == "sigmoid":
        l[rows, c] = f32(np.log(p / (1 - p)))
        first = sig(l[rows, c]) + bias[c] + near
        at = lambda v: f32(np.log(v / (1 - v)))  # noqa: E731
    else:
        l[rows, c] = 0.0
        l[:, 30] = f32(np.log(1 / p - 1))
        first = p + bias[c] + near
        at = lambda v: f32(np.log(v / p))  # noqa: E731
    wanted = p
    for again in range(6):
        l[:, 0] = at(first)
        l[:, 4] = at(first - 1.8e-8)
        for j in range(k - 1):
            l[:, 1 + 8 * j] = at(first * (1.5 + j))
        if score == "softmax":
            small = np.exp(np.delete(l, 30, 1)).sum(1) - 1
            l[:, 30] = f32(np.log(1 / wanted - 1 - small))
            p = 1 / np.exp(l).sum(1)
            first = p + bias[c] + near
    assert np.isfinite(l).all()
    _check(torch.from_numpy(l).float(), torch.from_numpy(bias).float(), k, score, groups=groups, group_k=group_k)


def test_scores_below_the_smallest_normal_number():
    """exp of them is flushed to zero in fp32, beside biases as small."""
    l = torch.full((3, 64), -120.0)
    l[0, 5], l[1, 9], l[2, 40] = -88.0, -88.5, -89.0
    b = torch.zeros(64)
    b[20], b[21] = 4e-39, 3e-39
    for k in (1, 2, 3):
        _check(l, b, k)
        _check(torch.cat([l, torch.zeros(3, 64)], 1), torch.cat([b, torch.full((64,), -1.0)]), k, "softmax")


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_of_scores_next_to_one(renorm, dtype):
    """With the logits, 1 - s keeps its relative precision where s itself is 1 in fp32. Against scores and weights in 64 bits from the logits:
    w and s are off by 2^-17 of themselves and the sum of them by as much, 1 - s by 2^-21 (|l| < 32: the argument's rounding 2^-20)."""
    T, E, k = 64, 64, 6
    l = 2 + 24 * torch.rand(T, E, generator=torch.Generator().manual_seed(21))
    l[9, 3:60], l[10, 4] = -torch.inf, -30.0
    g = torch.randn(T, k, generator=torch.Generator().manual_seed(22))
    r = _router(T, E, k, renorm=renorm, scale=2.5, grad_dtype=dtype)
    r.forward(l.cuda(), _bias(E).cuda())
    got = f64(r.backward(g.cuda(), logits=l.cuda()))
    idx = r.topk_idx.cpu().numpy().astype(np.int64)
    assert (np.take_along_axis(f64(l), idx, 1) > 17).mean() > 0.2
    chosen = np.take_along_axis(f64(l), idx, 1)
    s, rest = O.sigmoid(chosen), O.sigmoid(-chosen)
    w = 2.5 * (s / s.sum(1, keepdims=True) if renorm else s)
    v = w * (f64(g) - (w * f64(g)).sum(1, keepdims=True) / 2.5) if renorm else w * f64(g)
    size = w * (np.abs(f64(g)) + ((w * np.abs(f64(g))).sum(1, keepdims=True) / 2.5 if renorm else 0))
    want, bound = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(want, idx, v * rest, 1)
    np.put_along_axis(bound, idx, (4 * TOL + 2.0 ** -19) * size * rest, 1)
    bound = bound + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0) + 1e-37
    assert (np.abs(got - want) <= bound).all()
    assert int(r.err) == 0


@pytest.mark.parametrize("E", [62, 63, 65])
def test_dense_gradient_of_logits_that_start_anywhere(E):
    T, k = 9, 5
    logits, g = _logits(T, E, 3), torch.randn(T, k, generator=torch.Generator().manual_seed(4)).cuda()
    grads = []
    for at in range(4):
        l = torch.zeros(T * E + at, device="cuda")[at:].view(T, E).copy_(logits)
        r = _router(T, E, k, score="softmax", renorm=False)
        r.forward(l)
        grads.append(r.backward(g).clone())
    assert all(torch.equal(d, grads[0]) for d in grads) and bool(grads[0].any())
