"""Out-of-bounds write checks of the sequence mixer and the optimizer step: every array that a call writes, its
workspace among them, lies inside a larger buffer whose 4 KB before and after it hold a byte pattern, rows are
further apart than they are wide, and pattern and gaps must be intact after the call."""
import ctypes

import numpy as np
import pytest
import torch

from sparse_moe_layer_topk_gb300 import _lib as M

from gpu_util import need_gpu
from test_gpu_guards import CANARY, Guarded

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


class Guards(Guarded):
    def __init__(self):
        super().__init__()
        self.gaps = []

    def rows(self, T, heads, width, gap):
        """A [T, heads, width] bf16 output whose tokens lie heads * width + gap apart, and that distance."""
        n = heads * width
        buf = self.empty(T, n + gap, dtype=BF)
        buf.view(torch.uint8).fill_(CANARY)
        self.gaps.append(buf[:, n:])
        return buf[:, :n].unflatten(1, (heads, width)), n + gap

    def check(self):
        super().check()
        for i, gap in enumerate(self.gaps):
            assert bool((gap.contiguous().view(torch.uint8) == CANARY).all()), f"rows {i}"


def _written(t):
    """No value still holds the pattern (a bf16 or fp32 value of four 0xA5 bytes does not come up here)."""
    word = torch.int16 if t.dtype == BF else torch.int32
    return not bool((t.contiguous().view(word) == (-23131 if t.dtype == BF else -1515870811)).any())


@pytest.mark.parametrize("gap", [0, 8, 24])
@pytest.mark.parametrize("lens,Hs,r,Dk,Dv", [
    ([1], 1, 1, 8, 8), ([129, 0, 127, 300], 2, 1, 128, 128), ([130, 255], 2, 3, 104, 96), ([257, 1, 70], 3, 1, 64, 64),
    ([200, 56], 1, 2, 40, 72), ([300], 2, 2, 120, 56), ([4000], 1, 2, 128, 128), ([3900], 2, 1, 64, 104)], ids=str)
def test_mixer_writes_stay_in_bounds(lens, Hs, r, Dk, Dv, gap):
    T, N, Hq = sum(lens), len(lens), Hs * r
    gen = torch.Generator().manual_seed(T + Dk)
    make = lambda *s, dt=BF: torch.randn(*s, generator=gen).to(dt).cuda()  # noqa: E731
    q, k, v, do = make(T, Hq, Dk), make(T, Hs, Dk), make(T, Hs, Dv), make(T, Hq, Dv)
    S0, X = make(N, Hs, Dk, Dv, dt=F32), make(N, Hs, Dk, Dv, dt=F32)
    decay = -torch.rand(Hs, generator=gen).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    g = Guards()
    o, ldo = g.rows(T, Hq, Dv, gap)
    dq, lddq = g.rows(T, Hq, Dk, gap)
    dk, lddk = g.rows(T, Hs, Dk, gap)
    dv, lddv = g.rows(T, Hs, Dv, gap)
    S, dS = g.empty(N, Hs, Dk, Dv, dtype=F32), g.empty(N, Hs, Dk, Dv, dtype=F32)
    err = g.empty(1, dtype=torch.int32)
    err.zero_()
    dims = dict(T=max(lens), d=Dk, l=Dv, E=Hs, k=r, f=T, S=N)
    fws, bws = (M.moe_workspace_size(op, **dims) for op in (M.MOE_OP_LINATTN_FWD, M.MOE_OP_LINATTN_BWD))
    assert fws > 0 or max(lens) < 2000  # (the long ones are split)
    ws = [g.empty(max(n, 32), dtype=torch.uint8) for n in (fws, bws)]
    M.moe_linattn_fwd(q, k, v, decay, cu, S0, N, T, max(lens), Hs, r, Dk, Dv, Hq * Dk, Hs * Dk, Hs * Dv, ldo, 0.3, o, S,
                      ws[0], fws, err)
    M.moe_linattn_bwd(do, q, k, v, decay, cu, S0, X, N, T, max(lens), Hs, r, Dk, Dv, Hq * Dv, Hq * Dk, Hs * Dk, Hs * Dv,
                      0.3, dq, dk, dv, lddq, lddk, lddv, dS, ws[1], bws, err)
    g.check()
    assert int(err) == 0
    for t in (o, dq, dk, dv, S, dS):
        assert _written(t)


def test_states_that_lie_side_by_side():
    """A state gradient directly behind the states that the call reads shares no memory with them."""
    T, n = 200, 2 * 64 * 64
    gen = torch.Generator().manual_seed(1)
    x = [torch.randn(T, 2, 64, generator=gen).to(BF).cuda() for _ in range(4)]
    states = torch.randn(3 * n, generator=gen).cuda()
    S0, X, dS = (states[i * n:(i + 1) * n].view(1, 2, 64, 64) for i in (0, 2, 1))
    keep = states.clone()
    out = [torch.empty_like(t) for t in x[:3]]
    decay = torch.tensor([-0.1, -0.2], device="cuda")
    M.moe_linattn_bwd(x[3], *x[:3], decay, None, S0, X, 1, T, T, 2, 1, 64, 64, 128, 128, 128, 128, 0.3, *out, 128, 128, 128,
                      dS, None, 0)
    apart = torch.empty_like(dS)
    M.moe_linattn_bwd(x[3], *x[:3], decay, None, S0, X, 1, T, T, 2, 1, 64, 64, 128, 128, 128, 128, 0.3, *out, 128, 128, 128,
                      apart, None, 0)
    assert torch.equal(states[:n], keep[:n]) and torch.equal(states[2 * n:], keep[2 * n:]) and torch.equal(dS, apart)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("B,Hs,r,Dk,Dv", [(1, 1, 1, 8, 8), (5, 3, 2, 40, 72), (37, 2, 5, 128, 104), (160, 8, 1, 64, 128)])
def test_step_writes_stay_in_bounds(B, Hs, r, Dk, Dv, graph):
    Hq, slots = Hs * r, B + 2
    gen = torch.Generator().manual_seed(B)
    make = lambda *s, dt=BF: torch.randn(*s, generator=gen).to(dt).cuda()  # noqa: E731
    q, k, v, decay = make(B, Hq, Dk), make(B, Hs, Dk), make(B, Hs, Dv), -torch.rand(Hs, generator=gen).cuda()
    first = make(slots, Hs, Dk, Dv, dt=F32)
    idx = torch.randperm(slots, generator=gen)[:B].to(torch.int32)
    if B > 3:
        idx[2] = -1
    idx = idx.cuda()
    want, state_want = torch.empty(B, Hq, Dv, dtype=BF, device="cuda"), first.clone()
    g = Guards()
    o, ldo = g.rows(B, Hq, Dv, 8)
    state = g.empty(slots, Hs, Dk, Dv, dtype=F32)
    state.copy_(first)
    call = lambda s, o, ld: M.moe_linattn_step(q, k, v, decay, s, idx, slots, B, Hs, r, Dk, Dv, Hq * Dk, Hs * Dk, Hs * Dv,  # noqa: E731
                                               ld, 0.3, o)
    steps = 3
    for _ in range(steps):
        call(state_want, want, Hq * Dv)
    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            call(state, o, ldo)
        for _ in range(steps):
            captured.replay()
    else:
        for _ in range(steps):
            call(state, o, ldo)
    g.check()
    assert _written(o) and torch.equal(o, want) and torch.equal(state, state_want)
    free = torch.ones(slots, dtype=torch.bool, device="cuda")
    free[idx[idx >= 0].long()] = False
    assert torch.equal(state[free], first[free])


@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_dtype,master", [(F32, False), (BF, False), (BF, True)], ids=str)
def test_optimizer_writes_stay_in_bounds(p_dtype, master, bits, shift):
    """Arrays of the very sizes that the header names; `shift` values further on, so that they are walked by value."""
    sizes = [1, 7, 255, 256, 257, 2049, 5003]
    gen = torch.Generator().manual_seed(bits + shift)
    g = Guards()

    def array(n, dtype, fill):
        whole = g.empty(n + shift, dtype=dtype)
        g.gaps.append(whole[:shift])
        t = whole[shift:]
        return t.copy_(fill) if isinstance(fill, torch.Tensor) else t.zero_()

    rows, grads, keep, outs = (M.AdamWTensor * len(sizes))(), [], [], []
    for i, n in enumerate(sizes):
        w = torch.randn(n, generator=gen)
        grads.append(torch.randn(n, generator=gen).cuda())
        p = array(n, p_dtype, w)
        ms = array(n, F32, p.float()) if master else None
        state = torch.uint8 if bits == 8 else F32
        m, v = array(n, state, 0), array(n, state, 0)
        scales = [g.empty(-(-n // 256), dtype=F32).zero_() for _ in range(2)] if bits == 8 else [None, None]
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        rows[i] = M.AdamWTensor(ptr(p), ptr(grads[i]), ptr(m), ptr(v), ptr(scales[0]), ptr(scales[1]), ptr(ms), n, 0.1,
                                M.MOE_DTYPE_F32 if p_dtype == F32 else M.MOE_DTYPE_BF16, M.MOE_DTYPE_F32)
        keep.append(p.clone())
        outs.append(p)
    plan = torch.empty(M.moe_workspace_size(M.MOE_OP_ADAMW_PLAN, T=len(sizes)), dtype=torch.uint8)
    chunks = ctypes.c_longlong()
    M.moe_adamw_plan(rows, len(sizes), bits, plan.data_ptr(), plan.numel(), chunks)
    plan = plan.cuda()
    ctl = g.empty(M.MOE_ADAMW_CTL_BYTES, dtype=torch.uint8).zero_()
    need = M.moe_workspace_size(M.MOE_OP_ADAMW_STEP)
    ws = g.empty(need, dtype=torch.uint8)
    for max_norm in (0.0, 1.0):
        M.moe_adamw_step(plan, len(sizes), chunks.value, bits, 0.1, None, 0.1, 0.05, 1e-8, max_norm, 5, ctl, ws, need)
    g.check()
    assert int(ctl[:8].view(torch.int64)) == 2
    for p, was in zip(outs, keep):
        assert not torch.equal(p, was) and bool(torch.isfinite(p.float()).all())
