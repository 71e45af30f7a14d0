"""Out-of-bounds write checks of routing, norm, convolution and scan: every array that a call writes, its workspace among
them, lies inside a larger buffer whose 4 KB before and after it hold a byte pattern, output rows are further apart than
they are wide where the call allows it, and pattern and gaps must be intact after the call."""
import numpy as np
import pytest
import torch

from sparse_moe_layer_topk_gb300 import _lib as M

from gpu_util import need_gpu
from test_gpu_block_guards import Guards, _written

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _make(seed):
    gen = torch.Generator().manual_seed(seed)
    return lambda *s, dt=BF: torch.randn(*s, generator=gen).to(dt).cuda()


@pytest.mark.parametrize("T,E,k,groups,group_k", [(1, 1, 1, 1, 1), (9, 100, 7, 1, 1), (33, 896, 16, 8, 4), (5, 1024, 32, 32, 31), (7, 1023, 9, 3, 2)])
@pytest.mark.parametrize("score,renorm", [(0, 1), (1, 0)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_routing(T, E, k, groups, group_k, score, renorm, dtype):
    make, g = _make(E), Guards()
    logits, bias, d_w = make(T, E, dt=F32), make(E, dt=F32), make(T, k, dt=F32)
    idx, w, s = g.empty(T, k, dtype=I32), g.empty(T, k, dtype=F32), g.empty(T, k, dtype=F32)
    dL, dk = g.empty(T, E, dtype=dtype), g.empty(T, k, dtype=F32)
    err = g.empty(1, dtype=I32).zero_()
    M.moe_route_scores(logits, bias, T, E, k, score, groups, group_k, 2, renorm, 1.5, idx, w, s, err)
    M.moe_route_scores_bwd(d_w, None, logits, idx, w, s, T, E, k, score, renorm, 1.5, dL,
                           M.MOE_DTYPE_F32 if dtype == F32 else M.MOE_DTYPE_BF16, dk, err)
    g.check()
    assert int(err) == 0 and _written(w) and _written(s) and _written(dL) and torch.equal(dk, d_w)
    assert bool(((idx >= 0) & (idx < E)).all())


@pytest.mark.parametrize("T,d", [(1, 8), (5, 1000), (131, 72), (3, 4104), (2, 16384), (700, 2048)])
@pytest.mark.parametrize("res", [None, BF, F32])
@pytest.mark.parametrize("block", [0, 64, 128, -1])
def test_norm(T, d, res, block):
    make, g = _make(d), Guards()
    x, w, dy = make(T, d), make(d, dt=F32), make(T, d)
    r = None if res is None else make(T, d, dt=res)
    code = M.MOE_DTYPE_F32 if res == F32 else M.MOE_DTYPE_BF16
    total = None if res is None else g.empty(T, d, dtype=res)
    block = d if block < 0 else block
    y = g.empty(T, d, dtype=torch.uint8 if block else BF)
    scale = g.empty(T, -(-d // block), dtype=F32) if block else None
    M.moe_rmsnorm_fwd(x, r, w, T, d, d, code, 1e-6, total, y, M.MOE_DTYPE_E4M3 if block else M.MOE_DTYPE_BF16, scale, block)
    dx, dr = g.empty(T, d, dtype=BF), None if res is None else g.empty(T, d, dtype=res)
    dw, need = g.empty(d, dtype=F32), M.moe_workspace_size(M.MOE_OP_RMSNORM_BWD, T=T, d=d)
    ws = g.empty(need, dtype=torch.uint8)
    M.moe_rmsnorm_bwd(dy, x if total is None else total, w, None if total is None else total, T, d, d, code, 1e-6, dx, dr, dw, ws, need)
    g.check()
    for t in [dx, dw] + ([] if res is None else [total, dr]) + ([scale] if block else [y]):
        assert _written(t)


@pytest.mark.parametrize("lens,D,W", [([1], 8, 4), ([33, 0, 2, 70], 24, 3), ([129], 520, 2), ([64, 65], 136, 4), ([0, 0], 16, 4)], ids=str)
@pytest.mark.parametrize("gap", [0, 8, 24])
def test_convolution(lens, D, W, gap):
    make, g, T, N = _make(D), Guards(), sum(lens), len(lens)
    x, dy, w, b = make(T, D), make(T, D), make(D, W, dt=F32), make(D, dt=F32)
    st, ds = make(N, W - 1, D), make(N, W - 1, D)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=I32, device="cuda")
    (y, ldy), (dx, lddx) = g.rows(T, 1, D, gap), g.rows(T, 1, D, gap)
    out, d_in, dw, db = g.empty(N, W - 1, D, dtype=BF), g.empty(N, W - 1, D, dtype=BF), g.empty(D, W, dtype=F32), g.empty(D, dtype=F32)
    err = g.empty(1, dtype=I32).zero_()
    need = M.moe_workspace_size(M.MOE_OP_CONV_BWD, T=T, d=D, l=W, S=N)
    ws = g.empty(need, dtype=torch.uint8)
    M.moe_conv_fwd(x, w, b, cu, st, N, T, D, W, D, ldy, 1, y, out, err)
    M.moe_conv_bwd(dy, x, w, b, cu, st, ds, N, T, D, W, D, D, lddx, 1, dx, dw, db, d_in, ws, need, err)
    slots = N + 2
    cache = g.empty(slots, W - 1, D, dtype=BF)
    cache.zero_()
    idx = torch.arange(N - 1, -1, -1, dtype=I32, device="cuda")
    one, ld1 = g.rows(N, 1, D, gap)
    M.moe_conv_step(make(N, D), w, b, cache, idx, slots, N, D, W, D, ld1, 1, one, err)
    g.check()
    assert int(err) == 0 and not cache[N:].any()
    for t in (y, dx, out, d_in, dw, db, one):
        assert _written(t)


@pytest.mark.parametrize("lens,D,S,G", [([1], 8, 4, 1), ([33, 0, 2, 70], 24, 16, 2), ([129], 520, 8, 1), ([64, 65], 136, 12, 1), ([0, 0], 16, 16, 1),
                                        ([1500], 8, 16, 2), ([900, 700], 40, 4, 5), ([64], 264, 16, 2)], ids=str)
@pytest.mark.parametrize("gap", [0, 8, 24])
def test_scan(lens, D, S, G, gap):
    make, g, T, N = _make(D + S), Guards(), sum(lens), len(lens)
    u, delta, z, dy, B, C = (make(T, w) for w in (D, D, D, D, G * S, G * S))
    A, skip, bias = -torch.exp(make(D, S, dt=F32)), make(D, dt=F32), make(D, dt=F32)
    st, ds = make(N, D, S, dt=F32), make(N, D, S, dt=F32)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=I32, device="cuda")
    (y, ldy), (du, lddu), (dd, lddd), (dz, lddz) = (g.rows(T, 1, D, gap) for _ in range(4))
    dB, dC = g.empty(T, G, S, dtype=BF), g.empty(T, G, S, dtype=BF)
    out, d_in, dA = g.empty(N, D, S, dtype=F32), g.empty(N, D, S, dtype=F32), g.empty(D, S, dtype=F32)
    dskip, dbias = g.empty(D, dtype=F32), g.empty(D, dtype=F32)
    err = g.empty(1, dtype=I32).zero_()
    dims = dict(T=max(lens), d=D, l=S, E=G, f=T, S=N)
    fws, bws, tws = (M.moe_workspace_size(op, **dims) for op in (M.MOE_OP_SCAN_FWD, M.MOE_OP_SCAN_BWD, M.MOE_OP_SCAN_TILE_STATES))
    assert fws > 0 or max(lens) < 700  # (the long ones are cut)
    ws, tiles = [g.empty(max(n, 16), dtype=torch.uint8) for n in (fws, bws)], g.empty(tws, dtype=torch.uint8)
    M.moe_scan_fwd(u, delta, A, B, C, skip, z, bias, cu, st, N, T, max(lens), D, S, G, D, D, G * S, G * S, D, ldy, 1, y, out, tiles, ws[0], fws, err)
    M.moe_scan_bwd(dy, u, delta, A, B, C, skip, z, bias, cu, tiles, ds, N, T, max(lens), D, S, G, D, D, D, G * S, G * S, D, 1, du, dd, dB, dC, dz,
                   lddu, lddd, lddz, dA, dskip, dbias, d_in, ws[1], bws, err)
    slots = N + 2
    cache = g.empty(slots, D, S, dtype=F32)
    cache.zero_()
    idx = torch.arange(N - 1, -1, -1, dtype=I32, device="cuda")
    one, ld1 = g.rows(N, 1, D, gap)
    M.moe_scan_step(make(N, D), make(N, D), A, make(N, G * S), make(N, G * S), skip, make(N, D), bias, cache, idx, slots, N, D, S, G, D, D, G * S, G * S,
                    D, ld1, 1, one, err)
    g.check()
    assert int(err) == 0 and not cache[N:].any()
    for t in (y, du, dd, dz, dB, dC, out, d_in, dA, dskip, dbias, one):
        assert _written(t)
