"""Refusals of the mixer's and optimizer's entry points, found on the host before any CUDA call."""
import ctypes

import pytest

from sparse_moe_layer_topk_gb300 import _lib as M
from sparse_moe_layer_topk_gb300 import build as B

P = 0x1000


@pytest.fixture(scope="module")
def lib():
    B.build_library()
    return M.load()


FWD = dict(q=P, k=P, v=P, log_decay=P, cu_seqlens=P, state_in=None, N=2, T=8, max_seqlen=8, Hs=2, r=1, Dk=64,
           Dv=64, ldq=128, ldk=128, ldv=128, ldo=128, scale=1.0, o=P, state_out=None, ws=P,
           ws_bytes=1 << 40, err_flag=None, stream=None)
BWD = dict(dout=P, q=P, k=P, v=P, log_decay=P, cu_seqlens=P, state_in=None, d_state_out=None, N=2, T=8,
           max_seqlen=8, Hs=2, r=1, Dk=64, Dv=64, lddo=128, ldq=128, ldk=128, ldv=128, scale=1.0, dq=P,
           dk=P, dv=P, lddq=128, lddk=128, lddv=128, d_state_in=None, ws=P, ws_bytes=1 << 40, err_flag=None,
           stream=None)
STEP = dict(q=P, k=P, v=P, log_decay=P, state=P, state_idx=None, n_slots=4, B=4, Hs=2, r=1, Dk=64, Dv=64, ldq=128,
            ldk=128, ldv=128, ldo=128, scale=1.0, o=P, err_flag=None, stream=None)


def _status(lib, name, base, **change):
    return getattr(lib, name)(*{**base, **change}.values())


COMMON = [(dict(q=None), M.MOE_ERR_ARG), (dict(k=None), M.MOE_ERR_ARG), (dict(v=None), M.MOE_ERR_ARG),
          (dict(log_decay=None), M.MOE_ERR_ARG), (dict(Hs=0), M.MOE_ERR_ARG), (dict(r=0), M.MOE_ERR_ARG),
          (dict(Dk=0), M.MOE_ERR_ARG), (dict(Dk=136), M.MOE_ERR_UNSUPPORTED), (dict(Dv=256), M.MOE_ERR_UNSUPPORTED),
          (dict(Dk=60), M.MOE_ERR_ALIGN), (dict(Dv=4), M.MOE_ERR_ALIGN), (dict(ldq=120), M.MOE_ERR_ARG),
          (dict(ldk=132), M.MOE_ERR_ALIGN), (dict(q=P + 8), M.MOE_ERR_ALIGN), (dict(v=P + 2), M.MOE_ERR_ALIGN)]


@pytest.mark.parametrize("change,want", COMMON + [
    (dict(o=None), M.MOE_ERR_ARG), (dict(o=P + 4), M.MOE_ERR_ALIGN), (dict(N=-1), M.MOE_ERR_ARG),
    (dict(T=-1), M.MOE_ERR_ARG), (dict(cu_seqlens=None, T=9), M.MOE_ERR_ARG),
    (dict(cu_seqlens=None, max_seqlen=3), M.MOE_ERR_ARG), (dict(state_in=P + 4), M.MOE_ERR_ALIGN),
    (dict(state_out=P + 4), M.MOE_ERR_ALIGN), (dict(N=0), M.MOE_OK)], ids=str)
def test_forward_refusals(lib, change, want):
    assert _status(lib, "moe_linattn_fwd", FWD, **change) == want


@pytest.mark.parametrize("change,want", COMMON + [
    (dict(dout=None), M.MOE_ERR_ARG), (dict(dq=None), M.MOE_ERR_ARG), (dict(dk=None), M.MOE_ERR_ARG),
    (dict(dv=None), M.MOE_ERR_ARG), (dict(lddo=64), M.MOE_ERR_ARG), (dict(lddv=120), M.MOE_ERR_ARG),
    (dict(dk=P + 8), M.MOE_ERR_ALIGN), (dict(d_state_out=P, d_state_in=P), M.MOE_ERR_ARG),
    (dict(N=0), M.MOE_OK)], ids=str)
def test_backward_refusals(lib, change, want):
    assert _status(lib, "moe_linattn_bwd", BWD, **change) == want


@pytest.mark.parametrize("name", ["state_in", "d_state_out"])
@pytest.mark.parametrize("behind", [0, 32, 65536 - 32, -32, 32 - 65536])
def test_backward_refuses_a_state_gradient_over_states_that_it_reads(lib, name, behind):
    """One recurrence of the call reads these states while another writes d_state_in."""
    assert 65536 == BWD["N"] * BWD["Hs"] * BWD["Dk"] * BWD["Dv"] * 4
    at = 1 << 20
    change = {name: at, "d_state_in": at + behind}
    assert _status(lib, "moe_linattn_bwd", BWD, **change) == M.MOE_ERR_ARG


@pytest.mark.parametrize("behind", [32, 65536 - 32, -32, 32 - 65536])
def test_forward_refuses_states_that_overlap_in_part(lib, behind):
    at = 1 << 20
    assert _status(lib, "moe_linattn_fwd", FWD, state_in=at, state_out=at + behind) == M.MOE_ERR_ARG


@pytest.mark.parametrize("change,want", COMMON + [
    (dict(state=None), M.MOE_ERR_ARG), (dict(o=None), M.MOE_ERR_ARG), (dict(B=5), M.MOE_ERR_ARG),
    (dict(B=-1), M.MOE_ERR_ARG), (dict(state=P + 8), M.MOE_ERR_ALIGN), (dict(B=0), M.MOE_OK)], ids=str)
def test_step_refusals(lib, change, want):
    assert _status(lib, "moe_linattn_step", STEP, **change) == want


def test_workspaces_are_asked_for(lib):
    """Where a call needs a workspace, none or a short one is refused."""
    for op, name, base in ((M.MOE_OP_LINATTN_FWD, "moe_linattn_fwd", FWD), (M.MOE_OP_LINATTN_BWD, "moe_linattn_bwd", BWD)):
        need = M.moe_workspace_size(op, T=65536, d=64, l=64, E=2, k=1, S=1)
        if need:
            big = dict(N=1, T=65536, max_seqlen=65536)
            assert _status(lib, name, base, **big, ws=None) == M.MOE_ERR_WORKSPACE
            assert _status(lib, name, base, **big, ws_bytes=need - 1) == M.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("by", [4, 16])
def test_workspaces_of_another_alignment(lib, by):
    """The states in them are read and written 32 bytes at a time."""
    big = dict(N=1, T=65536, max_seqlen=65536)
    for op, name, base in ((M.MOE_OP_LINATTN_FWD, "moe_linattn_fwd", FWD), (M.MOE_OP_LINATTN_BWD, "moe_linattn_bwd", BWD)):
        assert M.moe_workspace_size(op, T=65536, d=64, l=64, E=2, k=1, f=65536, S=1) > 0
        assert _status(lib, name, base, **big, ws=P + by) == M.MOE_ERR_ALIGN


def _tensor(**change):
    x = dict(p=P, g=P, m=P, v=P, m_scale=None, v_scale=None, master=None, n=5000, weight_decay=0.0,
             p_dtype=M.MOE_DTYPE_F32, g_dtype=M.MOE_DTYPE_F32)
    return M.AdamWTensor(*{**x, **change}.values())


def _plan(lib, tensors, bits=32, size=None):
    rows = (M.AdamWTensor * len(tensors))(*tensors)
    need = M.moe_workspace_size(M.MOE_OP_ADAMW_PLAN, T=len(tensors))
    buf = ctypes.create_string_buffer(need)
    chunks = ctypes.c_longlong()
    status = lib.moe_adamw_plan(rows, len(tensors), bits, buf, need if size is None else size, ctypes.byref(chunks))
    return status, chunks.value


@pytest.mark.parametrize("change,bits,want", [
    (dict(p=None), 32, M.MOE_ERR_ARG), (dict(g=None), 32, M.MOE_ERR_ARG), (dict(m=None), 32, M.MOE_ERR_ARG),
    (dict(v=None), 32, M.MOE_ERR_ARG), (dict(n=-1), 32, M.MOE_ERR_ARG), (dict(p_dtype=2), 32, M.MOE_ERR_ARG),
    (dict(g_dtype=-1), 32, M.MOE_ERR_ARG), (dict(master=P), 32, M.MOE_ERR_ARG), (dict(), 8, M.MOE_ERR_ARG),
    (dict(), 16, M.MOE_ERR_UNSUPPORTED), (dict(p=P + 2), 32, M.MOE_ERR_ALIGN), (dict(m=P + 1), 32, M.MOE_ERR_ALIGN),
    (dict(g=P + 1, g_dtype=M.MOE_DTYPE_BF16), 32, M.MOE_ERR_ALIGN)], ids=str)
def test_plan_refusals(lib, change, bits, want):
    assert _plan(lib, [_tensor(), _tensor(**change)], bits)[0] == want


def test_plan_counts_chunks(lib):
    many = [_tensor(n=0, p=None, g=None, m=None, v=None), _tensor(n=1), _tensor(n=2048), _tensor(n=2049), _tensor(p=P + 4, n=10)]
    assert _plan(lib, many) == (M.MOE_OK, 0 + 1 + 1 + 2 + 1)
    assert _plan(lib, [_tensor(m_scale=P, v_scale=P, m=P + 1)], 8) == (M.MOE_OK, 3)
    assert _plan(lib, many, size=64)[0] == M.MOE_ERR_WORKSPACE


ADAMW = dict(plan=P, n_tensors=1, chunks=1, state_bits=32, lr=1e-3, lr_dev=None, rate1=0.1, rate2=0.01, eps=1e-8,
             max_norm=1.0, seed=0, ctl=P, ws=P, ws_bytes=1 << 30, err_flag=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(plan=None), M.MOE_ERR_ARG), (dict(ctl=None), M.MOE_ERR_ARG), (dict(n_tensors=0), M.MOE_ERR_ARG),
    (dict(chunks=-1), M.MOE_ERR_ARG), (dict(state_bits=4), M.MOE_ERR_UNSUPPORTED), (dict(rate1=0.0), M.MOE_ERR_ARG),
    (dict(rate2=1.1), M.MOE_ERR_ARG), (dict(eps=-1.0), M.MOE_ERR_ARG), (dict(lr=float("nan")), M.MOE_ERR_ARG),
    (dict(max_norm=float("nan")), M.MOE_ERR_ARG), (dict(ws=None), M.MOE_ERR_WORKSPACE),
    (dict(ws_bytes=8), M.MOE_ERR_WORKSPACE), (dict(ctl=P + 4), M.MOE_ERR_ALIGN), (dict(plan=P + 8), M.MOE_ERR_ALIGN),
    (dict(chunks=0), M.MOE_OK), (dict(chunks=0, max_norm=0.0, ws=None, ws_bytes=0), M.MOE_OK)], ids=str)
def test_step_of_adamw_refusals(lib, change, want):
    assert _status(lib, "moe_adamw_step", ADAMW, **change) == want
