"""Refusals of the entry points of routing, norm, convolution and scan, found on the host before any CUDA call."""
import pytest

from sparse_moe_layer_topk_gb300 import _lib as M
from sparse_moe_layer_topk_gb300 import build as B

P = 0x1000
ARG, ALIGN, WS, UNS, OK = M.MOE_ERR_ARG, M.MOE_ERR_ALIGN, M.MOE_ERR_WORKSPACE, M.MOE_ERR_UNSUPPORTED, M.MOE_OK


@pytest.fixture(scope="module")
def lib():
    B.build_library()
    return M.load()


def _far(*names, step=1 << 24):
    return {n: (i + 1) * step for i, n in enumerate(names)}


ROUTE = dict(logits=P, bias=P, T=4, E=64, k=4, score=0, groups=4, group_k=2, group_top=2, renorm=1, scale=1.0, topk_idx=P,
             topk_w=P, topk_s=P, err_flag=None, stream=None)
ROUTE_BWD = dict(d_w=P, slot_of=None, logits=P, topk_idx=P, topk_w=P, topk_s=P, T=4, E=64, k=4, score=1, renorm=0, scale=1.0,
                 d_logits=P, dtype=0, d_topk_w=None, err_flag=None, stream=None)
GRADS = dict(d_logits=P, x=P, Wr=P, T=4, d=64, E=64, dx_accum=P, dWr=P, wgrad_dtype=0, dz=P, W_dn=P, l=64, stream=None)
LATENT = dict(x=P, Wr=P, W_dn=P, T=4, d=64, E=64, l=64, logits=P, z=P, stream=None)
NORM = dict(**_far("x", "residual", "weight"), T=4, d=128, ldx=128, res_dtype=1, eps=1e-6, **_far("sum", "y", step=1 << 28),
            y_dtype=1, y_scale=None, block=0, stream=None)
NORM_BWD = dict(dy=P, u=P, weight=P, d_sum=P, T=4, d=128, ldu=128, res_dtype=1, eps=1e-6, dx=P, d_residual=P, dw=P, ws=P,
                ws_bytes=1 << 40, stream=None)
CONV = dict(x=P, weight=P, bias=P, cu_seqlens=P, state_in=None, N=2, T=8, D=64, W=4, ldx=64, ldy=64, silu=1, y=P, state_out=None,
            err_flag=None, stream=None)
CONV_BWD = dict(dy=P, x=P, weight=P, bias=P, cu_seqlens=P, state_in=None, d_state_out=None, N=2, T=8, D=64, W=4, lddy=64, ldx=64,
                lddx=64, silu=1, dx=P, dw=P, db=P, d_state_in=None, ws=P, ws_bytes=1 << 40, err_flag=None, stream=None)
CONV_STEP = dict(x=P, weight=P, bias=P, state=P, state_idx=None, n_slots=4, B=4, D=64, W=4, ldx=64, ldy=64, silu=1, y=P,
                 err_flag=None, stream=None)
SCAN = dict(u=P, delta=P, A=P, B=P, C=P, skip=P, z=P, dt_bias=P, cu_seqlens=P, state_in=None, N=2, T=8, max_seqlen=8, D=64, states=16,
            G=2, ldu=64, lddelta=64, ldB=32, ldC=32, ldz=64, ldy=64, softplus=1, y=P, state_out=None, tile_states=P, ws=P,
            ws_bytes=1 << 40, err_flag=None, stream=None)
SCAN_BWD = dict(dy=P, u=P, delta=P, A=P, B=P, C=P, skip=P, z=P, dt_bias=P, cu_seqlens=P, tile_states=P, d_state_out=None, N=2, T=8,
                max_seqlen=8, D=64, states=16, G=2, lddy=64, ldu=64, lddelta=64, ldB=32, ldC=32, ldz=64, softplus=1, du=P, ddelta=P, dB=P,
                dC=P, dz=P, lddu=64, ldddelta=64, lddz=64, dA=P, dskip=P, d_dt_bias=P, d_state_in=None, ws=P, ws_bytes=1 << 40,
                err_flag=None, stream=None)
SCAN_STEP = dict(u=P, delta=P, A=P, B=P, C=P, skip=P, z=P, dt_bias=P, state=P, state_idx=None, n_slots=4, rows=4, D=64, states=16, G=2,
                 ldu=64, lddelta=64, ldB=32, ldC=32, ldz=64, ldy=64, softplus=1, y=P, err_flag=None, stream=None)

NAN, INF = float("nan"), float("inf")
CASES = {
    "moe_route_scores": (ROUTE, [
        (dict(logits=None), ARG), (dict(topk_idx=None), ARG), (dict(topk_w=None), ARG), (dict(topk_s=None), ARG), (dict(T=-1), ARG),
        (dict(E=0), ARG), (dict(E=1028), ARG), (dict(k=0), ARG), (dict(k=33), ARG), (dict(score=2), ARG), (dict(groups=0), ARG),
        (dict(groups=3), ARG), (dict(E=66, groups=33, group_k=33), UNS), (dict(group_k=0), ARG), (dict(group_k=5), ARG), (dict(group_top=0), ARG),
        (dict(group_top=3), ARG), (dict(k=17, group_k=1), ARG), (dict(scale=NAN), ARG), (dict(scale=INF), ARG), (dict(logits=P + 2), ALIGN),
        (dict(bias=P + 1), ALIGN), (dict(T=0), OK)]),
    "moe_route_scores_bwd": (ROUTE_BWD, [
        (dict(d_w=None), ARG), (dict(logits=None), ARG), (dict(topk_idx=None), ARG), (dict(d_logits=None), ARG), (dict(scale=0.0), ARG),
        (dict(dtype=2), ARG), (dict(d_logits=P + 8), ALIGN), (dict(logits=P + 4), ALIGN), (dict(T=0), OK), (dict(T=0, logits=None, renorm=1), OK)]),
    "moe_router_grads": (GRADS, [
        (dict(d_logits=None), ARG), (dict(Wr=None), ARG), (dict(x=None), ARG), (dict(W_dn=None), ARG), (dict(d=60), ALIGN), (dict(E=60), ALIGN),
        (dict(l=60), ALIGN), (dict(wgrad_dtype=2), ARG), (dict(dx_accum=P + 8), ALIGN), (dict(T=0, dWr=None), OK)]),
    "moe_router_logits_latent": (LATENT, [
        (dict(x=None), ARG), (dict(z=None), ARG), (dict(logits=None), ARG), (dict(E=1088), ARG), (dict(d=32), ALIGN), (dict(logits=P + 4), ALIGN), (dict(T=0), OK)]),
    "moe_rmsnorm_fwd": (NORM, [
        (dict(x=None), ARG), (dict(weight=None), ARG), (dict(y=None), ARG), (dict(sum=None), ARG), (dict(residual=None), ARG), (dict(eps=0.0), ARG),
        (dict(eps=NAN), ARG), (dict(d=0), ARG), (dict(d=16392, ldx=16392), UNS), (dict(d=100), ALIGN), (dict(ldx=120), ARG), (dict(ldx=132), ALIGN),
        (dict(res_dtype=2), ARG), (dict(y_dtype=0), ARG), (dict(y_dtype=2), ARG), (dict(y_dtype=2, y_scale=P, block=32), UNS), (dict(x=(1 << 24) + 8), ALIGN),
        (dict(sum=(2 << 24) + 16), ARG), (dict(sum=1 << 24), ARG), (dict(y=1 << 24), ARG), (dict(y=2 << 24), ARG), (dict(y=(1 << 28) + 256), ARG),
        (dict(T=0), OK), (dict(T=0, y_dtype=2, y_scale=P, block=128), OK), (dict(T=0, residual=None, sum=None), OK)]),
    "moe_rmsnorm_bwd": (NORM_BWD, [
        (dict(dy=None), ARG), (dict(u=None), ARG), (dict(weight=None), ARG), (dict(eps=0.0), ARG), (dict(ldu=64), ARG), (dict(ldu=132), ALIGN),
        (dict(d=16392, ldu=16392), UNS), (dict(res_dtype=3), ARG), (dict(dx=P + 8), ALIGN), (dict(ws=None), WS), (dict(ws_bytes=16), WS),
        (dict(T=0, dw=None), OK)]),
    "moe_conv_fwd": (CONV, [
        (dict(x=None), ARG), (dict(weight=None), ARG), (dict(y=None), ARG), (dict(W=1), UNS), (dict(W=5), UNS), (dict(W=0), ARG), (dict(D=60), ALIGN),
        (dict(D=0), ARG), (dict(ldx=56), ARG), (dict(ldy=68), ALIGN), (dict(y=P + 8), ALIGN), (dict(N=-1), ARG), (dict(T=-1), ARG),
        (dict(cu_seqlens=None, T=9), ARG), (dict(state_in=P, state_out=P), ARG), (dict(state_in=P, state_out=P + 16), ARG), (dict(state_in=P + 8), ALIGN),
        (dict(T=2 ** 31 - 1, D=1 << 20, ldx=1 << 20, ldy=1 << 20), ARG), (dict(N=0), OK)]),
    "moe_conv_bwd": (CONV_BWD, [
        (dict(dy=None), ARG), (dict(dx=None), ARG), (dict(lddx=32), ARG), (dict(d_state_in=P, state_in=P), ARG), (dict(d_state_in=P, d_state_out=P + 32), ARG),
        (dict(ws=None), WS), (dict(ws_bytes=64), WS), (dict(W=6), UNS), (dict(N=0, dw=None, db=None), OK)]),
    "moe_conv_step": (CONV_STEP, [
        (dict(x=None), ARG), (dict(state=None), ARG), (dict(B=5), ARG), (dict(B=-1), ARG), (dict(state=P + 8), ALIGN), (dict(W=8), UNS), (dict(B=0), OK)]),
    "moe_scan_fwd": (SCAN, [
        (dict(u=None), ARG), (dict(delta=None), ARG), (dict(A=None), ARG), (dict(B=None), ARG), (dict(C=None), ARG), (dict(y=None), ARG), (dict(states=0), ARG),
        (dict(states=20), UNS), (dict(states=6), ALIGN), (dict(G=3), ARG), (dict(G=0), ARG), (dict(G=32, ldB=512, ldC=512), ALIGN), (dict(D=60), ALIGN),
        (dict(ldB=16), ARG), (dict(ldB=34), ALIGN), (dict(C=P + 4), ALIGN), (dict(ldz=60), ARG), (dict(u=P + 8), ALIGN), (dict(A=P + 4), ALIGN),
        (dict(max_seqlen=-1), ARG), (dict(cu_seqlens=None, max_seqlen=3), ARG), (dict(state_in=P, state_out=P + 16), ARG), (dict(tile_states=P + 8), ALIGN),
        (dict(T=1 << 20, max_seqlen=1 << 20, N=1, ws=None), WS), (dict(N=0), OK)]),
    "moe_scan_bwd": (SCAN_BWD, [
        (dict(dy=None), ARG), (dict(tile_states=None), ARG), (dict(dB=None), ARG), (dict(dC=None), ARG), (dict(dA=None), ARG), (dict(du=None), ARG),
        (dict(ddelta=None), ARG), (dict(lddu=32), ARG), (dict(lddz=60), ARG), (dict(ldddelta=68), ALIGN), (dict(dB=P + 4), ALIGN),
        (dict(d_state_in=P, d_state_out=P + 16), ARG), (dict(ws=None), WS), (dict(ws_bytes=64), WS)]),
    "moe_scan_step": (SCAN_STEP, [
        (dict(u=None), ARG), (dict(state=None), ARG), (dict(rows=5), ARG), (dict(rows=-1), ARG), (dict(state=P + 8), ALIGN), (dict(states=32), UNS),
        (dict(rows=0), OK)]),
}


APART = {  # arguments that no two of share memory
    "moe_rmsnorm_bwd": {**NORM_BWD, **_far("dy", "u", "weight", "d_sum", "dx", "d_residual", "dw", "ws")},
    "moe_conv_fwd": {**CONV, **_far("x", "weight", "y")},
    "moe_conv_bwd": {**CONV_BWD, **_far("dy", "x", "weight", "dx", "ws")},
    "moe_conv_step": {**CONV_STEP, **_far("x", "weight", "state", "y")},
    "moe_scan_fwd": {**SCAN, **_far("u", "delta", "B", "C", "z", "y", "ws")},
    "moe_scan_bwd": {**SCAN_BWD, **_far("dy", "u", "delta", "B", "C", "z", "du", "ddelta", "dz", "ws")},
    "moe_scan_step": {**SCAN_STEP, **_far("u", "delta", "B", "C", "z", "y")},
}
ROW = 64 * 2  # bytes of a row of the sizes above


@pytest.mark.parametrize("name,out,others", [
    ("moe_rmsnorm_bwd", "dx", ["dy", "u", "d_sum"]), ("moe_rmsnorm_bwd", "d_residual", ["dy", "u", "d_sum"]), ("moe_conv_fwd", "y", ["x"]),
    ("moe_conv_bwd", "dx", ["dy", "x"]), ("moe_conv_step", "y", ["x"]), ("moe_scan_fwd", "y", ["u", "delta", "z", "B", "C"]),
    ("moe_scan_bwd", "du", ["dy", "u", "delta", "z", "B", "C"]), ("moe_scan_bwd", "ddelta", ["dy", "u", "delta", "z", "B", "C"]),
    ("moe_scan_bwd", "dz", ["dy", "u", "delta", "z", "B", "C"]), ("moe_scan_step", "y", ["u", "delta", "z", "B", "C"])], ids=str)
def test_results_over_what_is_read(lib, name, out, others):
    """A result that begins inside what other rows are still read from, at either end."""
    base = APART[name]
    for other in others:
        for shift in (ROW // 2, -ROW // 2, ROW):
            assert getattr(lib, name)(*{**base, out: base[other] + shift}.values()) == ARG, (other, shift)
    if name in ("moe_conv_fwd", "moe_conv_bwd", "moe_scan_fwd", "moe_scan_bwd"):  # neighbours' rows are read: not in place either
        assert getattr(lib, name)(*{**base, out: base[others[0]]}.values()) == ARG


def test_results_among_the_columns_that_are_read(lib):
    """Columns of one wide buffer of which some are both read and written."""
    base = {**APART["moe_conv_fwd"], "ldx": 192, "ldy": 192}
    at = base["x"]
    for columns in (32, 136, -32, -184):  # a part of y's columns lies in x's
        assert lib.moe_conv_fwd(*{**base, "y": at + 2 * columns}.values()) == ARG


@pytest.mark.parametrize("name,change,want", [(n, c, w) for n, (_, rows) in CASES.items() for c, w in rows], ids=str)
def test_refusals(lib, name, change, want):
    base = CASES[name][0]
    assert len(base) == len(M.SIGNATURES[name][0])
    assert getattr(lib, name)(*{**base, **change}.values()) == want


def test_workspaces_of_nothing(lib):
    """Sizes that no call allows ask for no workspace, and do not divide by zero."""
    for op in (M.MOE_OP_RMSNORM_BWD, M.MOE_OP_CONV_BWD, M.MOE_OP_SCAN_FWD, M.MOE_OP_SCAN_BWD, M.MOE_OP_SCAN_TILE_STATES):
        assert M.moe_workspace_size(op) == 0
        assert M.moe_workspace_size(op, T=-1, d=-8, l=-4, E=-2, f=-1, S=-3) == 0
        assert M.moe_workspace_size(op, T=5, d=0, l=16, E=1, f=5, S=1) == 0


def test_tile_states_hold_every_tile(lib):
    """Tiles of 32 tokens of sequences placed one behind the other never share a place, and fit."""
    size = M.moe_workspace_size(M.MOE_OP_SCAN_TILE_STATES, d=8, l=4, f=100, S=5)
    assert size >= (100 // 32 + 5) * 8 * 4 * 4
    at, taken = 0, []
    for n, length in enumerate([1, 32, 33, 0, 34]):
        taken += [at // 32 + n + k for k in range(-(-length // 32))]
        at += length
    assert at == 100 and len(set(taken)) == len(taken) and max(taken) < 100 // 32 + 5


@pytest.mark.parametrize("E,logits,want", [(64, P + 4, ALIGN), (66, P + 4, OK), (63, P + 8, OK), (63, P + 2, ALIGN), (64, P, OK)])
@pytest.mark.parametrize("renorm", [0, 1])
def test_logits_that_the_dense_gradient_reads(lib, E, logits, want, renorm):
    """Expert counts that are not a multiple of 4 are read one by one, from any place of a float; renormalised scores need no logits."""
    got = lib.moe_route_scores_bwd(*{**ROUTE_BWD, "E": E, "logits": logits, "renorm": renorm, "T": 0}.values())
    assert got == (OK if renorm and logits % 4 == 0 else want)
