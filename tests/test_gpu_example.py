"""examples/distill_step.py: teacher packets, both losses with their gradients,
and the compressed update together; and the gradients it uses against
PyTorch's own differentiation of the same losses."""

import importlib.util
import os

import pytest
import torch

import error_feedback_gradient_gb300 as efg

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    path = os.path.join(ROOT, "examples", "distill_step.py")
    spec = importlib.util.spec_from_file_location("distill_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_losses_fall_and_runs_repeat():
    ex = _example()
    a = ex.train(steps=30, tokens=256)
    assert a[-1][0] < 0.7 * a[0][0]
    b = ex.train(steps=3, tokens=256)
    assert b == ex.train(steps=3, tokens=256)


def test_gradients_are_pytorchs():
    ex = _example()
    torch.manual_seed(0)
    model = ex.Student(32, 8, 500, 3)
    x = torch.randn(64, 32, device="cuda")
    t = torch.randn(64, 500, device="cuda") * 2
    k, tau = 20, 1.5
    v, i = torch.empty(64, k, device="cuda"), torch.empty(64, k, dtype=torch.int32, device="cuda")
    c, tail = torch.empty(64, dtype=torch.int32, device="cuda"), torch.empty(64, device="cuda")
    efg.logits_topk(t, k, tau, v, i, c, tail)
    logits, z, ids = model(x)
    gl, gz = torch.empty_like(logits), torch.empty_like(z)
    loss = torch.empty(64, device="cuda")
    efg.distill_loss_grad(logits.detach(), v, i, tau, loss, gl, counts=c, tail=tail)
    bl, bc = torch.empty(1, device="cuda"), torch.empty(1, 8, dtype=torch.int32, device="cuda")
    bt = torch.empty(1, dtype=torch.int32, device="cuda")
    efg.balance_loss_grad(z.detach(), ids, [0, 64], 0.3, 0.1, bl, bc, bt, gz)
    got, = torch.autograd.grad([logits, z], [model.flat], [gl, gz])

    # the same in 64 bits, by differentiation
    model64 = ex.Student(32, 8, 500, 3)
    model64.flat = torch.nn.Parameter(model64.flat.detach().double())
    logits, z, _ = model64(x.double())
    p = torch.softmax(t.double() / tau, 1)
    keep = torch.zeros_like(p).scatter_(1, i.long(), 1.0)
    q = torch.softmax(logits / tau, 1)
    rest_p, rest_q = (p * (1 - keep)).sum(1), (q * (1 - keep)).sum(1)
    kl = (keep * p * (torch.log(p) - torch.log(q))).sum(1) + rest_p * torch.log(rest_p / rest_q)
    f = 8.0 * torch.bincount(ids.reshape(-1).long(), minlength=8).double() / (2 * 64)
    balance = 0.3 * (f * torch.softmax(z, 1).mean(0)).sum() + 0.1 * torch.logsumexp(
        z, 1).square().mean()
    want, = torch.autograd.grad(kl.sum() + balance, [model64.flat])
    # 32-bit products of up to 500 terms on top of the losses' own rounding
    assert float((got.double() - want).abs().max()) <= 1e-4 * float(want.abs().max())
    assert float((loss.double() - kl).abs().max()) <= 1e-4
    assert float(bl[0]) == pytest.approx(float(balance), rel=1e-5)
