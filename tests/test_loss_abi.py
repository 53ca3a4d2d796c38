"""Host-side refusals of the training-loss entry points: every bad argument is
an error before anything reaches the device (no device here)."""

import ctypes

import pytest
import torch

import error_feedback_gradient_gb300 as efg
from test_abi import _header_defines, _i64, lib  # noqa: F401


def _p(mib, extra=0):
    return ctypes.c_void_p((mib << 20) + extra)


ROWS, V, K = 4, 1000, 8
X, VAL, IDX, CNT, TAIL, LOSS, STATS, GRAD, RG = (_p(i) for i in range(1, 10))


def _topk(lib, x=X, dt=0, rows=ROWS, v=V, stride=V, k=K, tau=1.0, val=VAL, idx=IDX, cnt=CNT,
          tail=TAIL):
    return lib.ef_logits_topk(x, dt, rows, v, stride, k, tau, val, idx, cnt, tail, None)


def _loss(lib, x=X, dt=0, rows=ROWS, v=V, stride=V, k=K, val=VAL, idx=IDX, cnt=CNT, tail=TAIL,
          tau=1.0, loss=LOSS, stats=STATS):
    return lib.ef_distill_loss(x, dt, rows, v, stride, k, val, idx, cnt, tail, tau, loss, stats,
                               None)


def _grad(lib, x=X, dt=0, rows=ROWS, v=V, stride=V, k=K, val=VAL, idx=IDX, cnt=CNT, tau=1.0,
          stats=STATS, rg=RG, grad=GRAD, gstride=V):
    return lib.ef_distill_grad(x, dt, rows, v, stride, k, val, idx, cnt, tau, stats, rg, grad,
                               gstride, None)


def _both(lib, x=X, dt=0, rows=ROWS, v=V, stride=V, k=K, val=VAL, idx=IDX, cnt=CNT, tail=TAIL,
          tau=1.0, rg=RG, loss=LOSS, grad=GRAD, gstride=V):
    return lib.ef_distill_loss_grad(x, dt, rows, v, stride, k, val, idx, cnt, tail, tau, rg,
                                    loss, grad, gstride, None)


@pytest.mark.parametrize("call", [_topk, _loss, _grad, _both])
def test_row_calls_refuse_bad_sizes(lib, call):  # noqa: F811
    d = _header_defines()
    assert call(lib, dt=3) == d["EF_ERR_ARG"]
    assert call(lib, rows=-1) == d["EF_ERR_SIZE"]
    assert call(lib, rows=1 << 31) == d["EF_ERR_SIZE"]
    assert call(lib, v=-1, stride=0) == d["EF_ERR_SIZE"]
    assert call(lib, v=(1 << 30) + 1, stride=1 << 31) == d["EF_ERR_SIZE"]
    assert call(lib, stride=V - 1) == d["EF_ERR_SIZE"]
    assert call(lib, k=-1) == d["EF_ERR_K"]
    assert call(lib, k=V + 1) == d["EF_ERR_K"]
    assert call(lib, v=5000, stride=5000, k=d["EF_MAX_ROW_PACKET"] + 1) == d["EF_ERR_K"]
    for tau in (0.0, -1.0, float("nan"), float("inf")):
        assert call(lib, tau=tau) == d["EF_ERR_ARG"]
    assert call(lib, rows=0) == d["EF_OK"]


@pytest.mark.parametrize("call", [_topk, _loss, _grad, _both])
def test_row_calls_refuse_bad_buffers(lib, call):  # noqa: F811
    d = _header_defines()
    for name in ("x", "val", "idx"):
        assert call(lib, **{name: None}) == d["EF_ERR_NULL"], name
    assert call(lib, x=_p(1, 2)) == d["EF_ERR_ALIGN"]
    assert call(lib, dt=1, x=_p(1, 1)) == d["EF_ERR_ALIGN"]
    for name, i in (("val", 2), ("idx", 3), ("cnt", 4)):
        assert call(lib, **{name: _p(i, 2)}) == d["EF_ERR_ALIGN"], name


def test_row_outputs_may_not_overlap(lib):  # noqa: F811
    d = _header_defines()
    assert _topk(lib, cnt=None) == d["EF_ERR_NULL"]
    assert _topk(lib, val=_p(1, 64)) == d["EF_ERR_ALIAS"]
    assert _topk(lib, idx=_p(2, 4 * ROWS * K - 4)) == d["EF_ERR_ALIAS"]
    assert _topk(lib, tail=_p(4)) == d["EF_ERR_ALIAS"]
    assert _loss(lib, loss=None) == d["EF_ERR_NULL"]
    assert _loss(lib, loss=_p(1, 4)) == d["EF_ERR_ALIAS"]
    assert _loss(lib, stats=LOSS) == d["EF_ERR_ALIAS"]
    assert _loss(lib, stats=_p(7, 2)) == d["EF_ERR_ALIGN"]
    assert _grad(lib, stats=None) == d["EF_ERR_NULL"]
    assert _grad(lib, grad=None) == d["EF_ERR_NULL"]
    assert _grad(lib, grad=_p(1, 4)) == d["EF_ERR_ALIAS"]          # shifted by one element
    assert _grad(lib, grad=X, gstride=V + 1) == d["EF_ERR_ALIAS"]  # same start, other stride
    assert _grad(lib, gstride=V - 1) == d["EF_ERR_SIZE"]
    assert _grad(lib, grad=_p(7)) == d["EF_ERR_ALIAS"]             # over the stats
    assert _both(lib, grad=_p(6)) == d["EF_ERR_ALIAS"]             # over the loss
    assert _both(lib, loss=_p(1, 8)) == d["EF_ERR_ALIAS"]
    assert _both(lib, loss=None) == d["EF_ERR_NULL"]
    assert _both(lib, rg=_p(9, 1)) == d["EF_ERR_ALIGN"]


T, E, KK = 16, 8, 2
Z, IDS, MASK, BL, BC, BT, SG, BG, WS = (_p(i) for i in range(20, 29))


def _ws_size(lib, t=T, e=E, k=KK, offs=(0, T)):
    out = ctypes.c_size_t(0)
    st = lib.ef_balance_workspace_size(t, e, k, len(offs) - 1, _i64(offs), ctypes.byref(out))
    return st, out.value


def _bloss(lib, z=Z, dt=0, t=T, e=E, stride=E, ids=IDS, k=KK, mask=MASK, nseg=1, offs=(0, T),
           alpha=1.0, beta=0.0, loss=BL, cnt=BC, tok=BT, ws=WS, wsb=1 << 20):
    return lib.ef_balance_loss(z, dt, t, e, stride, ids, k, mask, nseg, _i64(offs), alpha, beta,
                               loss, cnt, tok, ws, wsb, None)


def _bgrad(lib, z=Z, dt=0, t=T, e=E, stride=E, k=KK, mask=MASK, nseg=1, offs=(0, T), alpha=1.0,
           beta=0.0, cnt=BC, tok=BT, sg=SG, grad=BG, gstride=E):
    return lib.ef_balance_grad(z, dt, t, e, stride, k, mask, nseg, _i64(offs), alpha, beta, cnt,
                               tok, sg, grad, gstride, None)


def _bboth(lib, z=Z, dt=0, t=T, e=E, stride=E, ids=IDS, k=KK, mask=MASK, nseg=1, offs=(0, T),
           alpha=1.0, beta=0.0, sg=SG, loss=BL, cnt=BC, tok=BT, grad=BG, gstride=E, ws=WS,
           wsb=1 << 20):
    return lib.ef_balance_loss_grad(z, dt, t, e, stride, ids, k, mask, nseg, _i64(offs), alpha,
                                    beta, sg, loss, cnt, tok, grad, gstride, ws, wsb, None)


@pytest.mark.parametrize("call", [_bloss, _bgrad, _bboth])
def test_balance_refuses_bad_sizes(lib, call):  # noqa: F811
    d = _header_defines()
    assert call(lib, dt=-1) == d["EF_ERR_ARG"]
    assert call(lib, t=-1, offs=(0, -1)) == d["EF_ERR_SIZE"]
    assert call(lib, t=1 << 31, offs=(0, 1 << 31)) == d["EF_ERR_SIZE"]
    assert call(lib, e=0) == d["EF_ERR_SIZE"]
    assert call(lib, e=d["EF_MAX_EXPERTS"] + 1, stride=4096) == d["EF_ERR_SIZE"]
    assert call(lib, stride=E - 1) == d["EF_ERR_SIZE"]
    assert call(lib, k=0) == d["EF_ERR_K"]
    assert call(lib, k=d["EF_MAX_EXPERTS"] + 1) == d["EF_ERR_K"]
    assert call(lib, nseg=0) == d["EF_ERR_SEGMENTS"]
    assert call(lib, nseg=2, offs=(0, 9, T - 1)) == d["EF_ERR_SEGMENTS"]
    assert call(lib, nseg=3, offs=(0, 9, 8, T)) == d["EF_ERR_SEGMENTS"]
    assert call(lib, nseg=1, offs=(1, T)) == d["EF_ERR_SEGMENTS"]
    assert call(lib, alpha=float("nan")) == d["EF_ERR_ARG"]
    assert call(lib, beta=float("inf")) == d["EF_ERR_ARG"]


def test_balance_refuses_bad_buffers(lib):  # noqa: F811
    d = _header_defines()
    st, need = _ws_size(lib)
    assert st == d["EF_OK"] and need >= 256
    assert _ws_size(lib, e=0)[0] == d["EF_ERR_SIZE"]
    assert _ws_size(lib, offs=(0, T + 1))[0] == d["EF_ERR_SEGMENTS"]
    for call in (_bloss, _bboth):
        for name in ("z", "ids", "loss", "cnt", "tok"):
            assert call(lib, **{name: None}) == d["EF_ERR_NULL"], name
        assert call(lib, ws=None) == d["EF_ERR_WORKSPACE"]
        assert call(lib, ws=_p(28, 128)) == d["EF_ERR_WORKSPACE"]
        assert call(lib, wsb=need - 1) == d["EF_ERR_WORKSPACE"]
        assert call(lib, loss=_p(23, 1)) == d["EF_ERR_ALIGN"]
        assert call(lib, cnt=_p(20, 4)) == d["EF_ERR_ALIAS"]       # inside the logits
        assert call(lib, tok=BL) == d["EF_ERR_ALIAS"]
        assert call(lib, ws=_p(24)) == d["EF_ERR_ALIAS"]
    for call in (_bgrad, _bboth):
        assert call(lib, grad=None) == d["EF_ERR_NULL"]
        assert call(lib, gstride=E - 1) == d["EF_ERR_SIZE"]
        assert call(lib, grad=_p(20, 4)) == d["EF_ERR_ALIAS"]
        assert call(lib, grad=Z, gstride=E + 8) == d["EF_ERR_ALIAS"]
        assert call(lib, sg=_p(26, 2)) == d["EF_ERR_ALIGN"]
    assert _bgrad(lib, cnt=None) == d["EF_ERR_NULL"]
    assert _bgrad(lib, tok=None) == d["EF_ERR_NULL"]


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        efg.logits_topk(x, 2, 1.0, None, None, None)          # not on a GPU


def test_dtype_constants_match_header():
    d = _header_defines()
    assert (efg.DTYPE_F32, efg.DTYPE_BF16, efg.DTYPE_F16) == (
        d["EF_DTYPE_F32"], d["EF_DTYPE_BF16"], d["EF_DTYPE_F16"])
