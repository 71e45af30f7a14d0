"""Linear attention on the GPU against the fp64 oracle: forward, backward and step.

Tolerances. Inputs are bf16 and exact on both sides. An output passes at most two
roundings to bf16: a product's operand (the scores or the state) and the
output itself, each within 2^-9 of its value; so elementwise |error| <= 2^-8 A * 1.05,
with A the same formula over the operands' magnitudes and 5% for sums and decays in fp32.
An fp32 state is a sum of products whose scaled operand keeps at least 16 bits: |error| <=
2^-16 A. The layer's relative Frobenius bound (1e-2) holds as well.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as O
from sparse_moe_layer_topk_gb300 import _lib as M
from gpu_util import REL_FRO, f64, need_gpu

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _make(lens, Hs, r, Dk, Dv, decays=None, seed=0, states=True):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    T, N, Hq = sum(lens), len(lens), Hs * r
    ld = -torch.rand(Hs, generator=g) if decays is None else torch.tensor(decays, dtype=F32)
    x = dict(lens=lens, ld=ld, q=n(T, Hq, Dk).to(BF), k=n(T, Hs, Dk).to(BF), v=n(T, Hs, Dv).to(BF),
             do=n(T, Hq, Dv).to(BF), S0=n(N, Hs, Dk, Dv) if states else None,
             X=n(N, Hs, Dk, Dv) if states else None,
             scale=Dk ** -0.5, dims=(Hs, r, Dk, Dv))
    return x


def _cuda(x):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _layer(x, **kw):
    from sparse_moe_layer_topk_gb300.linattn import LinearAttention
    Hs, r, Dk, Dv = x["dims"]
    return LinearAttention(x["ld"].cuda(), sum(x["lens"]), Dk, Dv, r=r, N=len(x["lens"]),
                           max_seqlen=max(x["lens"], default=0), scale=x["scale"], **kw)


def _close(name, got, ref, mag, bits):
    got = f64(got)
    assert np.isfinite(got).all(), name
    err = np.abs(got - ref)
    bound = 2.0 ** -bits * 1.05 * mag + 1e-30
    worst = (err / bound).max() if err.size else 0.0
    assert worst <= 1.0, f"{name}: {worst:.2f} of the bound"
    norm = np.linalg.norm(ref)
    assert np.linalg.norm(err) <= REL_FRO * norm + 1e-30, f"{name}: {np.linalg.norm(err) / norm:.2e}"


def _ref(x):
    d = lambda t: None if t is None else f64(t)  # noqa: E731
    args = [d(x[n]) for n in ("q", "k", "v")]
    mags = [np.abs(a) for a in args]
    ab = lambda t: None if t is None else np.abs(d(t))  # noqa: E731
    ld, S0, X, do = f64(x["ld"]), d(x["S0"]), d(x["X"]), d(x["do"])
    out = dict(zip(["o", "S"], O.linattn_forward(*args, ld, x["lens"], x["scale"], S0)))
    mag = dict(zip(["o", "S"], O.linattn_forward(*mags, ld, x["lens"], x["scale"], ab(x["S0"]))))
    names = ["dq", "dk", "dv", "dS"]
    out.update(zip(names, O.linattn_backward(do, *args, ld, x["lens"], x["scale"], S0, X)))
    mag.update(zip(names, O.linattn_backward(np.abs(do), *mags, ld, x["lens"], x["scale"], ab(x["S0"]), ab(x["X"]))))
    return out, mag


def _check(x, la=None, states=True):
    la = la or _layer(x)
    y = _cuda(x)
    o = la.forward(y["q"], y["k"], y["v"], _cu(x["lens"]), y["S0"], want_state=states)
    dq, dk, dv = la.backward(y["do"], y["X"])
    torch.cuda.synchronize()
    ref, mag = _ref(x)
    _close("o", o, ref["o"], mag["o"], 8)
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _close(n, t, ref[n], mag[n], 8)
    if states:
        _close("state_out", la.state_out, ref["S"], mag["S"], 16)
        if x["S0"] is not None or x["X"] is not None:
            _close("d_state_in", la.d_state_in, ref["dS"], mag["dS"], 16)
    assert int(la.err) == 0
    return la


LENS = [[1], [2], [63], [64], [65], [127], [128], [129], [255], [256], [300], [385],
        [0], [0, 0], [1, 1, 1], [0, 5, 0, 200, 1], [128, 128], [130, 0, 126, 257]]


@pytest.mark.parametrize("lens", LENS, ids=str)
def test_lengths(lens):
    _check(_make(lens, 2, 1, 128, 128))


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (64, 128), (128, 64), (8, 8), (16, 128), (40, 72),
                                   (96, 104), (120, 56), (128, 8)])
def test_widths(Dk, Dv):
    _check(_make([150, 37], 2, 1, Dk, Dv, seed=Dk + Dv))


@pytest.mark.parametrize("Hs,r", [(1, 1), (3, 1), (1, 2), (2, 3), (1, 8), (5, 4)])
@pytest.mark.parametrize("Dk,Dv", [(64, 128), (128, 128)])
def test_grouped_heads(Hs, r, Dk, Dv):
    _check(_make([131, 1, 140], Hs, r, Dk, Dv, seed=Hs * 10 + r))


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("lens,Hs,r", [([127, 255, 126, 383], 3, 2), ([255, 127, 1, 127], 2, 4),
                                       ([4095], 1, 2), ([2047, 127, 1663], 1, 3)], ids=str)
def test_grouped_heads_of_nearly_whole_chunks(lens, Hs, r, Dk, Dv):
    """Chunks short of a token, for each head of a group in turn; the long ones in segments."""
    _check(_make(lens, Hs, r, Dk, Dv, seed=sum(lens) + r))


@pytest.mark.parametrize("N,max_seqlen", [(1, 20000), (3, 5000)])
def test_empty_sequences_where_long_ones_were_expected(N, max_seqlen):
    from sparse_moe_layer_topk_gb300.linattn import LinearAttention
    x = _make([0] * N, 2, 2, 64, 128)
    _check(x, LinearAttention(x["ld"].cuda(), 0, 64, 128, r=2, N=N, max_seqlen=max_seqlen, scale=x["scale"]))


@pytest.mark.parametrize("most", [2 ** 31 - 1, 2 ** 31 - 100, 2 ** 31 - 128, 10 ** 12])
@pytest.mark.parametrize("lens,Hs", [([300, 0, 129], 2), ([2900], 3)], ids=str)
def test_any_bound_of_the_lengths(lens, Hs, most):
    """A bound that says nothing, up to the last number of its type."""
    from sparse_moe_layer_topk_gb300.linattn import LinearAttention
    x = _make(lens, Hs, 1, 64, 128, seed=Hs)
    _check(x, LinearAttention(x["ld"].cuda(), sum(lens), 64, 128, N=len(lens), max_seqlen=most, scale=x["scale"]))


def test_without_states():
    x = _make([200, 90], 2, 2, 64, 64, states=False)
    la = _check(x)
    # (no state given on either side: d_state_in was not asked for)
    assert la._d_state_in is None


@pytest.mark.parametrize("decays", [[0.0, -1e-6], [-float("inf"), -0.5], [-100.0, -20.0], [-1e-3, -88.0]],
                         ids=str)
def test_extreme_decays(decays):
    """No decay, total decay, and slopes whose powers underflow inside a chunk."""
    _check(_make([260, 3], 2, 1, 64, 64, decays=decays))


def test_bad_decay_is_flagged_and_counts_as_none():
    x = _make([40], 3, 1, 64, 64, decays=[0.5, float("nan"), -0.5])
    la, y = _layer(x), _cuda(x)
    o = la.forward(y["q"], y["k"], y["v"], _cu([40]), y["S0"])
    torch.cuda.synchronize()
    assert int(la.err) == M.MOE_FLAG_NONFINITE
    x["ld"] = torch.tensor([0.0, 0.0, -0.5])
    ref, mag = _ref(x)
    _close("o", o, ref["o"], mag["o"], 8)


def test_many_chunks_keep_the_state():
    """Over 40 chunks with hardly any decay the fp32 state keeps its 16 bits."""
    _check(_make([5200], 1, 1, 64, 64, decays=[-1e-5]))


@pytest.mark.parametrize("N,T", [(1, 700), (3, 600)])
def test_equal_lengths_without_bounds(N, T):
    """cu_seqlens None: N sequences of T / N tokens."""
    x = _make([T // N] * N, 2, 1, 64, 128)
    la, y = _layer(x), _cuda(x)
    o = la.forward(y["q"], y["k"], y["v"], None, y["S0"], want_state=True)
    dq, dk, dv = la.backward(y["do"], y["X"])
    ref, mag = _ref(x)
    for n, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        _close(n, t, ref[n], mag[n], 8)
    _close("state_out", la.state_out, ref["S"], mag["S"], 16)


def test_slices_of_a_fused_projection():
    x = _make([133, 60], 2, 2, 64, 128)
    Hs, r, Dk, Dv = x["dims"]
    T = sum(x["lens"])
    w = [Hs * r * Dk, Hs * Dk, Hs * Dv]
    fused = torch.full((T, sum(w) + 24), float("nan"), dtype=BF, device="cuda")
    at = 8
    for n, wid in zip("qkv", w):
        fused[:, at:at + wid] = x[n].cuda().flatten(1)
        x[n + "_view"] = fused[:, at:at + wid].unflatten(1, x[n].shape[1:])
        at += wid
    la, y = _layer(x), _cuda(x)
    o = la.forward(x["q_view"], x["k_view"], x["v_view"], _cu(x["lens"]), y["S0"], want_state=True)
    dq, dk, dv = la.backward(y["do"], y["X"])
    ref, mag = _ref(x)
    for n, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        _close(n, t, ref[n], mag[n], 8)


@pytest.mark.parametrize("r", [1, 3])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_other_sequences_values_stay_out(bad, r):
    """A sequence of NaN or infinities leaves its neighbours in the same tiles as they were."""
    lens = [70, 50, 75]
    x = _make(lens, 1, r, 64, 64)
    ref, mag = _ref(x)
    for n in ("q", "k", "v", "do"):
        x[n][70:120] = bad
    la, y = _layer(x), _cuda(x)
    o = la.forward(y["q"], y["k"], y["v"], _cu(lens), y["S0"], want_state=True)
    dq, dk, dv = la.backward(y["do"], y["X"])
    for part, seq in ((slice(0, 70), 0), (slice(120, 195), 2)):
        for n, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
            _close(n, t[part], ref[n][part], mag[n][part], 8)
        _close("state", la.state_out[seq], ref["S"][seq], mag["S"][seq], 16)
        _close("d_state", la.d_state_in[seq], ref["dS"][seq], mag["dS"][seq], 16)


def test_bad_bounds_are_flagged_and_skipped():
    """Sequences out of order, past T or longer than max_seqlen: flagged, nothing of them written."""
    x = _make([60, 60, 60], 1, 1, 64, 64)
    la, y = _layer(x), _cuda(x)
    la.max_seqlen = 64
    ref, mag = _ref(x)
    for cu in ([0, 60, 50, 180], [0, 60, 120, 181], [0, 60, -1, 1]):
        la.err.zero_()
        la.o.fill_(7.0)
        la.state_out.fill_(7.0)
        la.forward(y["q"], y["k"], y["v"], torch.tensor(cu, dtype=torch.int32, device="cuda"), y["S0"],
                   want_state=True)
        torch.cuda.synchronize()
        assert int(la.err) == M.MOE_FLAG_BAD_INDEX, cu
        _close("o", la.o[:60], ref["o"][:60], mag["o"][:60], 8)
        bad = 1 if cu[2] < cu[1] else 2
        assert (la.state_out[bad] == 7.0).all()


def test_outputs_stay_inside_their_rows():
    """Rows that belong to no sequence keep what they hold."""
    x = _make([100, 30], 1, 2, 64, 64)
    la, y = _layer(x), _cuda(x)
    cu = torch.tensor([0, 90, 110], dtype=torch.int32, device="cuda")  # tokens 110.. unused
    for t in (la.o, la.dq, la.dk, la.dv):
        t.fill_(3.0)
    la.forward(y["q"], y["k"], y["v"], cu, y["S0"])
    la.backward(y["do"], y["X"])
    for t in (la.o, la.dq, la.dk, la.dv):
        assert (t[110:] == 3.0).all() and not (t[:110] == 3.0).all(dim=(1, 2)).any()


def test_same_result_on_a_side_stream_and_in_a_graph():
    x = _make([300, 77], 2, 1, 128, 64)
    la, y = _layer(x), _cuda(x)
    cu = _cu(x["lens"])

    def both():
        la.forward(y["q"], y["k"], y["v"], cu, y["S0"], want_state=True)
        la.backward(y["do"], y["X"])

    keep = lambda: [t.clone() for t in (la.o, la.state_out, la.dq, la.dk, la.dv, la.d_state_in)]  # noqa: E731
    both()
    want = keep()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(keep(), want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for t in (la.o, la.dq, la.dk, la.dv):
        t.zero_()
    graph.replay()
    for a, b in zip(keep(), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("lens,r,Dk,Dv", [([4000], 2, 128, 128), ([2900, 0, 513], 1, 64, 128)], ids=str)
def test_segments_in_a_graph(lens, r, Dk, Dv):
    """Several launches a call, each behind the one before it: the same bits in a graph and a second time."""
    x = _make(lens, 1, r, Dk, Dv, seed=9)
    la = _check(x)
    assert la.ws_bytes > 0  # (in segments)
    y, cu = _cuda(x), _cu(lens)

    def both():
        la.forward(y["q"], y["k"], y["v"], cu, y["S0"], want_state=True)
        la.backward(y["do"], y["X"])

    keep = lambda: [t.clone() for t in (la.o, la.state_out, la.dq, la.dk, la.dv, la.d_state_in)]  # noqa: E731
    want = keep()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
        both()
    for t in (la.o, la.dq, la.dk, la.dv, la.ws):
        t.zero_()
    for _ in range(2):
        graph.replay()
        for a, b in zip(keep(), want):
            assert torch.equal(a, b)


def test_states_in_place():
    """state_out may be state_in."""
    x = _make([200, 0, 15], 2, 1, 64, 64)
    la, y = _layer(x), _cuda(x)
    la.forward(y["q"], y["k"], y["v"], _cu(x["lens"]), y["S0"], want_state=True)
    want = la.state_out.clone()
    la.state_out.copy_(y["S0"])
    la.forward(y["q"], y["k"], y["v"], _cu(x["lens"]), la.state_out, want_state=True)
    assert torch.equal(la.state_out, want)


@pytest.mark.parametrize("how", ["current", "stream", "handle", "graph"])
@pytest.mark.parametrize("lens,Hs,r", [([200, 0, 15], 2, 1), ([4000], 1, 2)], ids=str)
def test_backward_of_a_forward_in_place(lens, Hs, r, how):
    """Consecutive segments by one instance, the states handed on in place: each segment's backward starts from
    the states before that segment."""
    parts = [_make(lens, Hs, r, 64, 64, seed=s) for s in (1, 2, 3)]
    la, cu = _layer(parts[0]), _cu(lens)
    ys = [_cuda(x) for x in parts]
    side = torch.cuda.Stream() if how in ("stream", "handle") else None
    stream = side.cuda_stream if how == "handle" else side

    def segment(y, state):
        la.forward(y["q"], y["k"], y["v"], cu, state, want_state=True, stream=stream)
        la.backward(y["do"], y["X"], stream=stream)

    for i, x in enumerate(parts):
        parts[i] = x = {**x, "ld": parts[0]["ld"], "S0": x["S0"] if i == 0 else la.state_out.clone().cpu()}
        state = ys[0]["S0"] if i == 0 else la.state_out
        torch.cuda.synchronize()
        if how == "graph" and i > 0:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                segment(ys[i], state)
            graph.replay()
        else:
            segment(ys[i], state)
        torch.cuda.synchronize()
        ref, mag = _ref(x)
        _close("o", la.o, ref["o"], mag["o"], 8)
        for n, t in (("dq", la.dq), ("dk", la.dk), ("dv", la.dv)):
            _close(n, t, ref[n], mag[n], 8)
        _close("state_out", la.state_out, ref["S"], mag["S"], 16)
        _close("d_state_in", la.d_state_in, ref["dS"], mag["dS"], 16)


@pytest.mark.parametrize("stream", [0, None])
def test_a_forward_in_place_keeps_states_that_are_still_being_written(stream):
    """The states come from work that is still under way on the call's stream, the default one."""
    x = _make([150], 1, 1, 64, 64)
    la, y, cu = _layer(x), _cuda(x), _cu(x["lens"])
    la.state_out.zero_()
    la.forward(y["q"], y["k"], y["v"], cu, la.state_out, want_state=True)
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)
    la.state_out.copy_(y["S0"])
    la.forward(y["q"], y["k"], y["v"], cu, la.state_out, want_state=True, stream=stream)
    dq, _, _ = la.backward(y["do"], y["X"], stream=stream)
    torch.cuda.synchronize()
    ref, mag = _ref(x)
    _close("dq", dq, ref["dq"], mag["dq"], 8)


def test_prompt_in_parts_and_tokens_resume_the_state():
    """A prompt at once, in two parts with the state handed on, and its last tokens by the step form
    give the same state and outputs."""
    from sparse_moe_layer_topk_gb300.linattn import LinearAttention
    x = _make([210], 2, 2, 64, 64, states=False)
    ref, mag = _ref(x)
    y = _cuda(x)
    ld = x["ld"].cuda()
    part = lambda t, a, b: t[a:b]  # noqa: E731
    first = LinearAttention(ld, 200, 64, 64, r=2, scale=x["scale"])
    o1 = first.forward(*(part(y[n], 0, 200) for n in "qkv"), want_state=True)
    cache = first.state_out.clone()
    one = LinearAttention(ld, 1, 64, 64, r=2, scale=x["scale"], backward=False)
    outs = [o1]
    for t in range(200, 210):
        outs.append(one.step(*(part(y[n], t, t + 1) for n in "qkv"), cache).clone())
    _close("o", torch.cat(outs), ref["o"], mag["o"], 8)
    _close("state", cache, ref["S"], mag["S"], 16)


@pytest.mark.parametrize("T,lens_of", [(4000, [4000]), (4096, [1000, 3, 3093])])
def test_long_axis(T, lens_of):
    """One and few long sequences with one head: the time axis is split over the GPU."""
    _check(_make(lens_of, 1, 1, 128, 128, decays=[-2e-3]))


@pytest.mark.parametrize("Hs,r,T,most", [(80, 1, 8190, 8192), (80, 2, 8192, 8192), (32, 1, 16300, 16384),
                                         (80, 1, 3001, 8192), (80, 1, 0, 8192), (151, 1, 20000, 20000)])
def test_long_axis_of_many_heads(Hs, r, T, most):
    """One sequence of heads that do not divide the SMs: segments of unequal lengths (151 heads fill the SMs
    and are not split)."""
    from sparse_moe_layer_topk_gb300.linattn import LinearAttention
    x = _make([T], Hs, r, 8, 16, decays=(-0.3 * 1000.0 ** (-np.arange(Hs) / Hs)).tolist(), seed=T + Hs)
    la = LinearAttention(x["ld"].cuda(), T, 8, 16, r=r, max_seqlen=most, scale=x["scale"], backward=False)
    assert (la.ws_bytes > 0) == (Hs < 151)
    y = _cuda(x)
    o = la.forward(y["q"], y["k"], y["v"], _cu([T]), y["S0"], want_state=True)
    torch.cuda.synchronize()
    d = {n: f64(x[n]) for n in ("q", "k", "v", "S0", "ld")}
    run = lambda f: O.linattn_forward(f(d["q"]), f(d["k"]), f(d["v"]), d["ld"], [T], x["scale"], f(d["S0"]))  # noqa: E731
    ref, mag = run(lambda a: a), run(np.abs)
    _close("o", o, ref[0], mag[0], 8)
    _close("state_out", la.state_out, ref[1], mag[1], 16)
    assert int(la.err) == 0


def test_offsets_past_32_bits():
    """Tokens 2^20 elements apart: the last ones lie past 2^31 elements."""
    T, ld = 2100, 1 << 20
    x = _make([T], 1, 1, 64, 64, decays=[-0.05], states=False)
    buf = torch.zeros(T * ld, dtype=BF, device="cuda")
    q = buf.as_strided((T, 1, 64), (ld, 64, 1), 0)
    k = buf.as_strided((T, 1, 64), (ld, 64, 1), 64)
    v = buf.as_strided((T, 1, 64), (ld, 64, 1), 128)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        t.copy_(x[n].cuda())
    la = _layer(x)
    o = la.forward(q, k, v, want_state=True)
    dq, dk, dv = la.backward(x["do"].cuda())
    ref, mag = _ref(x)
    for n, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        _close(n, t, ref[n], mag[n], 8)


# ------------------------------------------------------------------ step

def _step_ref(x, state, idx):
    o = np.zeros((x["q"].shape[0], x["q"].shape[1], x["v"].shape[2]))
    mag, S, A = o.copy(), f64(state).copy(), np.abs(f64(state))
    for b, slot in enumerate(idx):
        if 0 <= slot < S.shape[0]:
            row = {n: f64(x[n][b:b + 1]) for n in "qkv"}
            ld = f64(x["ld"])
            o[b:b + 1], s = O.linattn_forward(row["q"], row["k"], row["v"], ld, [1], x["scale"], S[slot][None])
            mag[b:b + 1], a = O.linattn_forward(*(np.abs(row[n]) for n in "qkv"), ld, [1], x["scale"], A[slot][None])
            S[slot], A[slot] = s[0], a[0]
    return o, mag, S, A


@pytest.mark.parametrize("B,Hs,r,Dk,Dv", [(1, 1, 1, 64, 64), (1, 32, 1, 128, 128), (3, 2, 4, 128, 64), (37, 5, 2, 96, 128),
                                          (2, 3, 1, 8, 8), (9, 2, 1, 40, 72), (130, 4, 1, 64, 128)])
def test_step(B, Hs, r, Dk, Dv):
    """fp32 state and output sums: the output is rounded once (2^-9), the state has fp32's error."""
    x = _make([1] * B, Hs, r, Dk, Dv, states=False)
    la, y = _layer(x, backward=False), _cuda(x)
    slots = B + 3
    g = torch.Generator().manual_seed(5)
    state = torch.randn(slots, Hs, Dk, Dv, generator=g)
    idx = torch.randperm(slots, generator=g)[:B].to(torch.int32)
    if B > 2:
        idx[1] = -1
    s = state.cuda()
    la.o.fill_(5.0)
    o = la.step(y["q"], y["k"], y["v"], s, idx.cuda())
    ref, mag, S, A = _step_ref(x, state, idx.tolist())
    _close("o", o, ref, mag, 9)
    _close("state", s, S, A, 21)
    assert int(la.err) == 0


def test_step_without_indexes_and_with_a_slot_past_the_cache():
    x = _make([1] * 4, 2, 1, 64, 64, states=False)
    la, y = _layer(x, backward=False), _cuda(x)
    state = torch.randn(4, 2, 64, 64)
    s = state.cuda()
    o = la.step(y["q"], y["k"], y["v"], s)
    ref, mag, S, A = _step_ref(x, state, range(4))
    _close("o", o, ref, mag, 9)
    _close("state", s, S, A, 21)
    s = state.cuda()
    o = la.step(y["q"], y["k"], y["v"], s, torch.tensor([0, 4, 3, -7], dtype=torch.int32, device="cuda"))
    assert int(la.err) == M.MOE_FLAG_BAD_INDEX
    ref, mag, S, A = _step_ref(x, state, [0, 4, 3, -7])
    _close("o", o, ref, mag, 9)
    _close("state", s, S, A, 21)


def test_step_on_a_cache_past_32_bits():
    slots = 140_000  # x 128 x 128 values: past 2^31
    state = torch.empty(slots, 1, 128, 128, device="cuda")
    x = _make([1, 1], 1, 1, 128, 128, states=False)
    la, y = _layer(x, backward=False), _cuda(x)
    init = torch.randn(2, 1, 128, 128)
    state[0], state[slots - 1] = init[0].cuda(), init[1].cuda()
    o = la.step(y["q"], y["k"], y["v"], state, torch.tensor([slots - 1, 0], dtype=torch.int32, device="cuda"))
    ref, mag, S, A = _step_ref(x, init, [1, 0])
    _close("o", o, ref, mag, 9)
    _close("state", state[[0, slots - 1]], S, A, 21)


# ------------------------------------------------------------------ refusals of the Python class

def test_class_refusals():
    x = _make([10], 2, 1, 64, 64)
    la, y = _layer(x), _cuda(x)
    with pytest.raises(ValueError):
        la.backward(y["do"])
    with pytest.raises(ValueError):
        la.forward(y["q"][:5], y["k"], y["v"])
    with pytest.raises(ValueError):
        la.forward(y["q"].float(), y["k"], y["v"])
    with pytest.raises(ValueError):
        la.forward(y["q"].transpose(1, 2).contiguous().transpose(1, 2), y["k"], y["v"])
    with pytest.raises(ValueError):
        la.forward(y["q"], y["k"], y["v"], state_in=y["S0"].double())
    with pytest.raises(M.MoEError):
        la.forward(y["q"].cpu(), y["k"], y["v"])


def test_an_instance_without_a_backward():
    """It says so, and keeps none of a prompt's operands alive."""
    x = _make([10], 2, 1, 64, 64)
    la, y = _layer(x, backward=False), _cuda(x)
    held = torch.cuda.memory_allocated()
    q = y["q"].clone()
    la.forward(q, y["k"], y["v"], state_in=y["S0"])
    del q
    assert torch.cuda.memory_allocated() == held
    with pytest.raises(ValueError, match="without a backward"):
        la.backward(y["do"])
