"""ef_distill_loss, ef_distill_grad and ef_distill_loss_grad against the 64-bit
oracle, within the bounds of losscheck.py."""

import math

import numpy as np
import pytest
import torch

import error_feedback_gradient_gb300 as efg
from losscheck import ROUND, U, assert_within, delta, f64, largest
from oracle import loss_oracle as lo
from test_gpu_logits_topk import _gen, logits

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def packet(s, k, seed, tau=1.0, ragged=False, noise=1.0):
    """A teacher near the student: its top k, counts and tail."""
    rows, vocab = s.shape
    t = torch.nan_to_num(s.float(), nan=0.0, posinf=5.0, neginf=-9.0).clamp(-50, 50)
    t = t + noise * torch.randn(rows, vocab, generator=_gen(seed), device=DEV)
    idx = torch.topk(t, k, 1).indices.sort(1).values
    val = torch.gather(t, 1, idx).contiguous()
    rest = t.scatter(1, idx, -math.inf)
    counts = torch.full((rows,), k, dtype=torch.int32, device=DEV)
    if ragged:
        counts = torch.randint(0, k + 1, (rows,), generator=_gen(seed + 1), device=DEV,
                               dtype=torch.int32)
    return val, idx.to(torch.int32).contiguous(), counts, torch.logsumexp(rest / tau, 1)


def like(s, pad=0, shift=0):
    rows, vocab = s.shape
    flat = torch.full((shift + rows * (vocab + pad) + 8,), 3.0, dtype=s.dtype, device=DEV)
    return flat, flat[shift:shift + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]


def check(s, val, idx, counts, tail, tau=1.0, row_grad=None, gpad=0, gshift=0):
    """All three calls on one set of inputs."""
    rows, vocab = s.shape
    with np.errstate(all="ignore"):
        loss, stats, grad = lo.distill(
            f64(s), idx.cpu().numpy(), f64(val), None if counts is None else counts.cpu().numpy(),
            None if tail is None else f64(tail), tau,
            None if row_grad is None else f64(row_grad))
    x, v = f64(s), f64(val)
    span = 2 * max(largest(x), largest(v)) / tau
    dl = delta(vocab, span)
    with np.errstate(all="ignore"):
        # p and |log p/q| of every slot, and of the rest
        xs = (np.take_along_axis(x, np.clip(idx.cpu().numpy(), 0, vocab - 1), 1)
              - stats[:, :1]) / tau
        y = (v - stats[:, 3:4]) / tau
        used = np.arange(v.shape[1]) < (v.shape[1] if counts is None
                                        else counts.cpu().numpy()[:, None])
        p = np.where(used & (xs > -np.inf), np.exp(y - stats[:, 4:5]), 0.0)
        gap = stats[:, 4] - stats[:, 2]
        far = np.where(p > 0, p * np.abs(y - xs - gap[:, None]), 0.0).sum(1)
        if tail is not None:
            rest = f64(tail) - stats[:, 3] / tau - stats[:, 1]
            far = far + np.where(stats[:, 5] > 0, stats[:, 5] * np.abs(rest - gap), 0.0)
    reach = np.nan_to_num(far, nan=0.0, posinf=0.0)
    got_loss = torch.full((rows,), 3.0, device=DEV)
    got_stats = torch.full((rows, 6), 3.0, device=DEV)
    efg.distill_loss(s, val, idx, tau, got_loss, got_stats, counts=counts, tail=tail)
    assert_within(f64(got_loss), loss, dl * (2 + reach), "loss")
    mag = np.abs(np.nan_to_num(stats, nan=0, posinf=0, neginf=0))
    assert_within(f64(got_stats), stats, dl * (1 + np.array([0, 0, 0, 0, 0, 1]) * mag) + U * mag, "stats")

    w = np.ones(rows) if row_grad is None else f64(row_grad)
    half, least = ROUND[s.dtype]
    with np.errstate(all="ignore"):
        z = (x - stats[:, :1]) / tau
        p = np.abs(grad) * tau + np.abs(w[:, None]) * (
            2 * np.nan_to_num(np.exp(z - stats[:, 2:3])) +
            2 * stats[:, 5:] * np.nan_to_num(np.exp(np.minimum(z - stats[:, 1:2], 0.0))))
    p = np.nan_to_num(p, nan=0, posinf=0)
    bound = 2 * dl * p / tau + (half * np.abs(np.nan_to_num(grad)) + least) * (1 + 2 * dl)
    bound = bound + 2.0 ** -120 * np.abs(w[:, None])          # flushed exponentials
    stats_in = got_stats
    for what in ("grad", "loss_grad"):
        flat, g = like(s, gpad, gshift)
        if what == "grad":
            efg.distill_grad(s, val, idx, tau, stats_in, g, counts=counts, row_grad=row_grad)
        else:
            both = torch.full((rows,), 3.0, device=DEV)
            efg.distill_loss_grad(s, val, idx, tau, both, g, counts=counts, tail=tail,
                                  row_grad=row_grad)
            assert_within(f64(both), loss, dl * (2 + reach), "loss of loss_grad")
        assert_within(f64(g), grad, bound, what)
        # nothing but the rows' own elements was written
        keep = torch.ones_like(flat, dtype=torch.bool)
        keep[gshift:gshift + rows * (vocab + gpad)].view(rows, vocab + gpad)[:, :vocab] = False
        assert bool((flat[keep] == 3.0).all()), f"{what} wrote outside its rows"
    return got_loss, got_stats


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("with_tail", [False, True])
@pytest.mark.parametrize("rows,vocab,k", [
    (1, 1, 1), (3, 2, 1), (5, 7, 7), (4, 255, 10), (9, 1000, 10), (3, 1000, 999),
    (3, 4099, 64), (2, 8192, 0), (3, 30522, 64), (2, 30522, 1024), (1, 131071, 128),
    (2, 262147, 100), (1, 600011, 33)])
def test_sizes(dtype, with_tail, rows, vocab, k):
    s = logits(rows, vocab, vocab + k, dtype)
    val, idx, counts, tail = packet(s, k, 1, 1.5)
    rg = torch.rand(rows, generator=_gen(2), device=DEV) + 0.5
    check(s, val, idx, counts, tail if with_tail else None, 1.5, rg)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift,gpad,gshift", [
    (1, 0, 1, 0), (6, 0, 6, 0), (0, 1, 0, 1), (3, 5, 0, 0), (0, 0, 1, 3), (8, 8, 16, 0),
    (7, 2, 0, 2)])
def test_strides_and_alignment(dtype, pad, shift, gpad, gshift):
    s = logits(5, 3001, 3, dtype, pad, shift)
    val, idx, counts, tail = packet(s, 50, 4, 2.0, ragged=True)
    check(s, val, idx, counts, tail, 2.0, None, gpad, gshift)


@pytest.mark.parametrize("vocab", [1000, 30522, 262147])
def test_ragged_counts_and_empty_packets(vocab):
    s = logits(12, vocab, 5)
    val, idx, counts, tail = packet(s, 40, 6, ragged=True)
    counts[:4] = torch.tensor([0, 40, 41, -3], dtype=torch.int32)   # 41 reads as 40, -3 as 0
    check(s, val, idx, counts, None)
    check(s, val, idx, counts, tail)
    check(s, val, idx, None, tail)                                  # every slot in use


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("with_tail", [False, True])
def test_masked_positions(dtype, with_tail):
    low = torch.finfo(dtype).min
    s = logits(8, 2050, 7, dtype)
    val, idx, counts, tail = packet(s, 30, 8)
    s[0] = -math.inf                                                # nothing left
    s[1].scatter_(0, idx[1].long(), -math.inf)                      # the packet masked
    keep = torch.zeros(2050, dtype=torch.bool, device=DEV)
    keep[idx[2].long()] = True
    s[2, ~keep] = -math.inf                                         # all but the packet masked
    s[3, torch.rand(2050, generator=_gen(1), device=DEV) < 0.7] = -math.inf
    s[4] = low                                                      # the lowest everywhere
    s[5, ~keep] = low
    counts[6] = 0
    val[7, 3:9] = -math.inf                                         # a teacher's own masks
    check(s, val, idx, counts, tail if with_tail else None)


def test_teacher_with_nothing_and_infinite_tail():
    s = logits(3, 500, 9)
    val, idx, counts, tail = packet(s, 10, 10)
    val[0] = -math.inf                      # no mass in the packet, all in the tail
    tail[1] = -math.inf                     # no mass outside it
    val[2], tail[2] = -math.inf, -math.inf  # none at all: loss 0, gradient 0
    loss, _ = check(s, val, idx, counts, tail)
    assert float(loss[2]) == 0.0


@pytest.mark.parametrize("dtype", TYPES)
def test_far_apart_logits(dtype):
    """A packet that holds nearly all of the mass, and one that holds none."""
    s = logits(4, 3000, 11, dtype)
    val, idx, counts, tail = packet(s, 5, 12)
    s[0].scatter_add_(0, idx[0].long(), torch.full((5,), 200.0, dtype=dtype, device=DEV))
    s[1].scatter_add_(0, idx[1].long(), torch.full((5,), -200.0, dtype=dtype, device=DEV))
    val[2] += 200.0
    tail[3] += 150.0
    check(s, val, idx, counts, tail)


@pytest.mark.parametrize("vocab", [700, 30522, 262147])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_nan_and_infinite_logits_show(vocab, bad):
    s = logits(4, vocab, 13)
    val, idx, counts, tail = packet(s, 6, 14)
    off = next(v for v in range(vocab) if v not in set(idx[0].tolist()))
    s[0, off] = bad
    s[1, int(idx[1, 2])] = bad
    val[2, 0] = bad
    loss, grad = torch.zeros(4, device=DEV), torch.zeros_like(s)
    efg.distill_loss_grad(s, val, idx, 1.0, loss, grad, counts=counts, tail=tail)
    assert torch.isnan(loss[:3]).all() and not torch.isnan(loss[3])
    assert torch.isnan(grad[:3]).all() and not torch.isnan(grad[3]).any()


@pytest.mark.parametrize("vocab", [700, 30522, 262147])
def test_malformed_packets_are_nan_rows(vocab):
    s = logits(7, vocab, 15, torch.bfloat16)
    val, idx, counts, tail = packet(s, 8, 16)
    good = idx.clone()
    idx[0, 3] = idx[0, 2]                   # twice the same position
    idx[1, 4], idx[1, 5] = good[1, 5], good[1, 4]
    idx[2, 7] = vocab
    idx[3, 0] = -1
    idx[4, 6] = 2 ** 31 - 1
    idx[5, 2:] = -1
    counts[5] = 2                           # unused slots are never looked at
    loss, stats = torch.zeros(7, device=DEV), torch.zeros(7, 6, device=DEV)
    grad = torch.zeros_like(s)
    efg.distill_loss(s, val, idx, 1.0, loss, stats, counts=counts, tail=tail)
    assert torch.isnan(loss[:5]).all() and torch.isnan(stats[:5]).all()
    assert torch.isfinite(loss[5:]).all() and torch.isfinite(stats[5:]).all()
    efg.distill_grad(s, val, idx, 1.0, stats, grad, counts=counts)
    assert torch.isnan(grad[:5]).all() and torch.isfinite(grad[5:]).all()
    loss.zero_()
    grad.zero_()
    efg.distill_loss_grad(s, val, idx, 1.0, loss, grad, counts=counts, tail=tail)
    assert torch.isnan(loss[:5]).all() and torch.isfinite(loss[5:]).all()
    assert torch.isnan(grad[:5]).all() and torch.isfinite(grad[5:]).all()


def test_rows_of_weight_zero():
    s = logits(5, 900, 17)
    val, idx, counts, tail = packet(s, 6, 18)
    rg = torch.tensor([0.0, 1.0, -0.0, 2.0, 0.0], device=DEV)
    s[0, 4] = math.nan
    idx[4, 1] = -5
    loss, stats = torch.zeros(5, device=DEV), torch.zeros(5, 6, device=DEV)
    efg.distill_loss(s, val, idx, 1.0, loss, stats, counts=counts, tail=tail)
    for both in (False, True):
        g = torch.full_like(s, 3.0)
        if both:
            efg.distill_loss_grad(s, val, idx, 1.0, loss, g, counts=counts, tail=tail,
                                  row_grad=rg)
            assert torch.isnan(loss[[0, 4]]).all()
        else:
            efg.distill_grad(s, val, idx, 1.0, stats, g, counts=counts, row_grad=rg)
        bits = g[[0, 2, 4]].view(torch.int32)
        assert bool((bits == 0).all()) and bool((g[[1, 3]] != 0).any(1).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(6, 1001, ), (3, 30522), (2, 262147), (1, 600011)])
def test_gradient_over_the_logits(dtype, rows, vocab):
    s = logits(rows, vocab, 19, dtype, pad=3)
    val, idx, counts, tail = packet(s, 20, 20)
    loss, stats = torch.zeros(rows, device=DEV), torch.zeros(rows, 6, device=DEV)
    efg.distill_loss(s, val, idx, 1.0, loss, stats, counts=counts, tail=tail)
    _, want = like(s, 3)
    efg.distill_grad(s, val, idx, 1.0, stats, want, counts=counts)
    a, _ = like(s, 3)
    a = a[:rows * (vocab + 3)].view(rows, vocab + 3)[:, :vocab]
    a.copy_(s)
    efg.distill_grad(a, val, idx, 1.0, stats, a, counts=counts)
    assert torch.equal(a, want)
    _, both = like(s, 3)
    efg.distill_loss_grad(s, val, idx, 1.0, loss, both, counts=counts, tail=tail)
    a.copy_(s)
    efg.distill_loss_grad(a, val, idx, 1.0, loss, a, counts=counts, tail=tail)
    assert torch.equal(a, both)


def test_gradient_against_differences_of_the_loss():
    """Differences of the 64-bit loss around the 32-bit logits."""
    s = logits(1, 60, 21, scale=2.0)
    val, idx, counts, tail = packet(s, 7, 22, 1.3)
    g, loss = torch.zeros_like(s), torch.zeros(1, device=DEV)
    efg.distill_loss_grad(s, val, idx, 1.3, loss, g, counts=counts, tail=tail)
    x, h = f64(s)[0], 1e-5
    for v in range(60):
        hi, low = x.copy(), x.copy()
        hi[v] += h
        low[v] -= h
        a, b = (lo.distill_row(y, idx[0].cpu().numpy(), f64(val)[0], float(tail[0]), 1.3)[0]
                for y in (hi, low))
        # central differences: h^2 / 6 times the third derivative, rounding 1e-16 / h
        assert abs(float(g[0, v]) - (a - b) / (2 * h)) <= 2e-9 + 2 * delta(60, 10.0)


def test_teacher_packets_end_to_end():
    """A student that equals its teacher, through logits_topk: no loss, no
    gradient beyond rounding."""
    x = logits(16, 30522, 23)
    k, tau = 64, 2.0
    v, i = torch.empty(16, k, device=DEV), torch.empty(16, k, dtype=torch.int32, device=DEV)
    c, t = torch.empty(16, dtype=torch.int32, device=DEV), torch.empty(16, device=DEV)
    efg.logits_topk(x, k, tau, v, i, c, t)
    loss, g = torch.empty(16, device=DEV), torch.empty_like(x)
    efg.distill_loss_grad(x, v, i, tau, loss, g, counts=c, tail=t)
    dl = delta(30522, largest(f64(x)) / tau)
    assert float(loss.abs().max()) <= 4 * dl + 40 * U
    assert float(g.abs().max()) <= (4 * dl + 40 * U) / tau


def test_equal_calls_give_equal_bits():
    s = logits(300, 5003, 24, torch.bfloat16)
    val, idx, counts, tail = packet(s, 30, 25, ragged=True)
    outs = []
    for _ in range(3):
        loss, g = torch.empty(300, device=DEV), torch.empty_like(s)
        efg.distill_loss_grad(s, val, idx, 1.0, loss, g, counts=counts, tail=tail)
        outs.append((loss, g))
    for loss, g in outs[1:]:
        assert torch.equal(loss, outs[0][0]) and torch.equal(g, outs[0][1])


def test_offsets_beyond_32_bits():
    stride = (1 << 30) + 24
    flat = torch.empty(2 * stride + 1000, dtype=torch.bfloat16, device=DEV)
    s = flat.as_strided((3, 1000), (stride, 1))
    s.copy_(logits(3, 1000, 26))
    val, idx, counts, tail = packet(s, 10, 27)
    dense = s.contiguous()
    loss, want = torch.empty(3, device=DEV), torch.empty_like(dense)
    efg.distill_loss_grad(dense, val, idx, 1.0, loss, want, counts=counts, tail=tail)
    loss2 = torch.empty(3, device=DEV)
    efg.distill_loss_grad(s, val, idx, 1.0, loss2, s, counts=counts, tail=tail)
    assert_within(f64(loss2), f64(loss), 2 * delta(1000, 15.0) * 40, "loss")
    assert float((s.float() - want.float()).abs().max()) <= 2.0 ** -8


def test_no_rows():
    s = torch.zeros(0, 9, device=DEV)
    e = torch.zeros(0, 2, device=DEV)
    efg.distill_loss_grad(s, e, e.int(), 1.0, torch.zeros(0, device=DEV), torch.zeros_like(s))


def test_replays_from_a_cuda_graph():
    s = logits(8, 30522, 28, torch.bfloat16)
    val, idx, counts, tail = packet(s, 64, 29)
    loss, g = torch.empty(8, device=DEV), torch.empty_like(s)

    def step():
        efg.distill_loss_grad(s, val, idx, 1.0, loss, g, counts=counts, tail=tail)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    s.copy_(logits(8, 30522, 30, torch.bfloat16))
    graph.replay()
    got = (loss.clone(), g.clone())
    step()
    assert torch.equal(loss, got[0]) and torch.equal(g, got[1])


def test_argument_errors():
    s = logits(2, 100, 31)
    val, idx, counts, tail = packet(s, 4, 32)
    loss, g = torch.empty(2, device=DEV), torch.empty_like(s)
    with pytest.raises(efg.EFError):
        efg.distill_loss(s, val, idx, 0.0, loss)
    with pytest.raises(ValueError):
        efg.distill_loss(s, val, idx.long(), 1.0, loss)
    with pytest.raises(ValueError):
        efg.distill_loss(s, val, idx, 1.0, torch.empty(3, device=DEV))
    with pytest.raises(ValueError):
        efg.distill_loss(s.double(), val, idx, 1.0, loss)
    with pytest.raises(ValueError):
        efg.distill_loss(s.t(), val, idx, 1.0, loss)
    with pytest.raises(ValueError):
        efg.distill_loss_grad(s, val, idx, 1.0, loss, g.half())
    with pytest.raises(efg.EFError):                       # a part of the logits
        efg.distill_loss_grad(s[:, :50], val, idx, 1.0, loss,
                              s.view(-1)[10:110].view(2, 50))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab,k,tau", [
    (6, 200, 5, 1.0), (40, 2000, 64, 2.0), (7, 30522, 64, 2.0), (3, 131071, 1, 2.15),
    (320, 40000, 100, 1.0)])
def test_losses_near_zero_keep_their_digits(dtype, rows, vocab, k, tau):
    # a student that is the teacher: the loss is 0 but for the powers' errors, at
    # most 2^-22 of a term on either side of the packet, and those of six
    # logarithms between 1/2 and 2, a unit in the last place each
    x = torch.randn(rows, vocab, generator=torch.Generator(device="cuda").manual_seed(k),
                    device="cuda").to(dtype) * 2
    v, i = torch.empty(rows, k, device="cuda"), torch.empty(rows, k, dtype=torch.int32,
                                                            device="cuda")
    c, tail = torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows,
                                                                               device="cuda")
    efg.logits_topk(x, k, tau, v, i, c, tail)
    loss = torch.empty(rows, device="cuda")
    efg.distill_loss(x, v, i, tau, loss, counts=c, tail=tail)
    assert float(loss.abs().max()) <= 2 * 2.0 ** -22 + 6 * 2.0 ** -23
    grad, again = torch.empty_like(x), torch.empty(rows, device="cuda")
    efg.distill_loss_grad(x, v, i, tau, again, grad, counts=c, tail=tail)
    assert float(again.abs().max()) <= 2 * 2.0 ** -22 + 6 * 2.0 ** -23
