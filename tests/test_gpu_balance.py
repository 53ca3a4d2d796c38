"""ef_balance_loss, ef_balance_grad and ef_balance_loss_grad against the 64-bit
oracle: counts exactly, the rest within the bounds of losscheck.py."""

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


def route(z, k, seed, dropped=0.0):
    ids = torch.topk(torch.nan_to_num(z.float(), neginf=-99.0), min(k, z.shape[1]), 1).indices
    if k > z.shape[1]:
        ids = ids[:, torch.arange(k, device=DEV) % z.shape[1]]
    ids = ids.to(torch.int32).contiguous()
    if dropped:
        ids[torch.rand(ids.shape, generator=_gen(seed), device=DEV) < dropped] = -1
    return ids


def like(z, pad, shift):
    rows, n = z.shape
    flat = torch.full((shift + rows * (n + pad) + 8,), 3.0, dtype=z.dtype, device=DEV)
    return flat, flat[shift:shift + rows * (n + pad)].view(rows, n + pad)[:, :n]


def check(z, ids, offs, alpha=0.7, beta=0.3, mask=None, seg_grad=None, gpad=0, gshift=0):
    T, E = z.shape
    k, nseg = ids.shape[1], len(offs) - 1
    loss, counts, tokens, grad = lo.balance(
        f64(z), ids.cpu().numpy(), offs, alpha, beta,
        None if mask is None else mask.cpu().numpy(), None if seg_grad is None else f64(seg_grad))
    dl = delta(E, largest(f64(z)))
    longest = max([b - a for a, b in zip(offs, offs[1:])] + [1])
    # every term of the loss is positive (alpha, beta > 0): relative errors add up
    big = largest(f64(z)) + math.log(E)
    loss_bound = (2 * dl + (longest + 40) * U) * (np.abs(loss) + 2 * beta * big)
    ws = torch.full((efg.balance_workspace_size(T, E, k, offs),), 0xAB, dtype=torch.uint8,
                    device=DEV)
    outs = {}
    half, least = ROUND[z.dtype]
    w = np.ones(nseg) if seg_grad is None else f64(seg_grad)
    x = f64(z)
    with np.errstate(all="ignore"):
        m = np.max(x, 1, keepdims=True) if T else x
        p = np.nan_to_num(np.exp(x - m))
        p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    bound = np.zeros((T, E))
    for s in range(nseg):
        a, b = offs[s], offs[s + 1]
        if tokens[s]:
            f = E * counts[s] / (k * int(tokens[s]))
            terms = abs(alpha) * (f + p[a:b] @ f[:, None]) + 2 * abs(beta) * big
            bound[a:b] = 4 * dl * abs(w[s]) * p[a:b] * terms / int(tokens[s])
    bound = bound + half * np.abs(grad) * (1 + 4 * dl) + least + 2.0 ** -120
    for call in ("loss", "both"):
        o = (torch.full((nseg,), 3.0, device=DEV),
             torch.full((nseg, E), 3, dtype=torch.int32, device=DEV),
             torch.full((nseg,), 3, dtype=torch.int32, device=DEV))
        if call == "loss":
            efg.balance_loss(z, ids, offs, alpha, beta, *o, mask=mask, workspace=ws)
        else:
            flat, g = like(z, gpad, gshift)
            efg.balance_loss_grad(z, ids, offs, alpha, beta, *o, g, mask=mask,
                                  seg_grad=seg_grad, workspace=ws)
            outs["both"] = (flat, g)
        assert efg.workspace_status(ws) == 0
        assert np.array_equal(o[1].cpu().numpy(), counts), f"counts of {call}"
        assert np.array_equal(o[2].cpu().numpy(), tokens), f"tokens of {call}"
        assert_within(f64(o[0]), loss, loss_bound, f"loss of {call}")
    flat, g = like(z, gpad, gshift)
    efg.balance_grad(z, k, offs, alpha, beta, o[1], o[2], g, mask=mask, seg_grad=seg_grad)
    outs["grad"] = (flat, g)
    keep = torch.ones_like(flat, dtype=torch.bool)
    keep[gshift:gshift + T * (E + gpad)].view(T, E + gpad)[:, :E] = False
    for what, (flat, g) in outs.items():
        assert_within(f64(g), grad, bound, f"gradient of {what}")
        assert bool((flat[keep] == 3.0).all()), f"{what} wrote outside its rows"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k", [
    (1, 1, 1), (1, 8, 2), (5, 2, 2), (64, 8, 2), (33, 7, 3), (100, 60, 4), (257, 64, 6),
    (129, 160, 6), (300, 256, 8), (70, 384, 8), (50, 1000, 5), (31, 1024, 16)])
def test_sizes(dtype, T, E, k):
    z = logits(T, E, T + E, dtype, scale=1.5)
    check(z, route(z, k, 1), [0, T])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift,gpad,gshift", [
    (1, 0, 1, 0), (0, 1, 0, 1), (8, 8, 0, 0), (0, 0, 3, 5), (4, 4, 4, 4)])
@pytest.mark.parametrize("E", [8, 61, 128])
def test_strides_and_alignment(dtype, E, pad, shift, gpad, gshift):
    z = logits(90, E, 3, dtype, pad, shift, scale=1.5)
    check(z, route(z, 3, 2), [0, 40, 90], gpad=gpad, gshift=gshift)


@pytest.mark.parametrize("E", [8, 100, 512])
def test_segments_masks_and_dropped_ids(E):
    z = logits(500, E, 4, scale=1.5)
    offs = [0, 0, 1, 130, 130, 131, 400, 500, 500]
    mask = (torch.rand(500, generator=_gen(5), device=DEV) > 0.3).to(torch.uint8)
    mask[131:400] = 0                                   # a segment of padding alone
    ids = route(z, 4, 6, dropped=0.2)
    ids[7, 0], ids[8, 1] = E, 2 ** 31 - 1               # outside: count for no expert
    ids[9, 2] = -(2 ** 31)
    sg = torch.rand(8, generator=_gen(7), device=DEV) + 0.5
    check(z, ids, offs, mask=mask, seg_grad=sg)
    check(z, ids, offs, mask=mask * 255, seg_grad=None)
    check(z, ids, offs, mask=mask.bool(), seg_grad=sg)


def test_many_segments():
    z = logits(3000, 16, 8, scale=1.5)
    rng = np.random.default_rng(1)
    offs = [0] + sorted(rng.integers(0, 3001, 1299).tolist()) + [3000]
    check(z, route(z, 2, 9), offs, seg_grad=torch.rand(1300, generator=_gen(3), device=DEV))


@pytest.mark.parametrize("E,T", [(8, 40000), (64, 20011), (256, 9000)])
def test_long_segments(E, T):
    z = logits(T, E, 10, torch.bfloat16, scale=1.5)
    check(z, route(z, 2, 11), [0, T])
    check(z, route(z, 2, 11), [0, 5, T - 9, T])


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_experts(dtype):
    low = torch.finfo(dtype).min
    z = logits(40, 24, 12, dtype, scale=1.5)
    z[:, 5] = -math.inf
    z[3] = -math.inf                                    # nothing left
    z[4] = low
    z[5, 1:] = low
    z[6, 1:] = -math.inf
    ids = route(z, 3, 13)
    # the lowest value's square is beyond fp32: the log-sum-exp term stays out here
    check(z, ids, [0, 20, 40], beta=0.0)
    z[4], z[5] = 0.0, 0.0
    check(z, ids, [0, 20, 40])


def test_collapsed_router():
    z = torch.full((600, 32), -30.0, device=DEV)
    z[:, 3] = 40.0
    check(z, torch.full((600, 1), 3, dtype=torch.int32, device=DEV), [0, 600])


def test_more_ids_than_experts():
    z = logits(30, 4, 14)
    check(z, route(z, 9, 15), [0, 30])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("T", [50, 30000])
def test_nan_shows_in_its_segment(bad, T):
    z = logits(T, 16, 16)
    z[T - 3, 2] = bad
    ids = torch.zeros(T, 1, dtype=torch.int32, device=DEV)
    offs = [0, 20, T]
    loss, counts = torch.zeros(2, device=DEV), torch.zeros(2, 16, dtype=torch.int32, device=DEV)
    tokens, g = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros_like(z)
    efg.balance_loss_grad(z, ids, offs, 1.0, 0.0, loss, counts, tokens, g)
    assert math.isnan(float(loss[1])) and not math.isnan(float(loss[0]))
    assert torch.isnan(g[T - 3]).any() and not torch.isnan(g[:T - 3]).any()
    assert counts[:, 0].tolist() == [20, T - 20]


def test_gradient_over_the_logits():
    for E in (8, 61, 256):
        z = logits(700, E, 17, torch.bfloat16, scale=1.5)
        ids = route(z, 2, 18)
        outs = []
        for in_place in (False, True):
            a = z.clone()
            g = a if in_place else torch.empty_like(z)
            o = (torch.empty(1, device=DEV), torch.empty(1, E, dtype=torch.int32, device=DEV),
                 torch.empty(1, dtype=torch.int32, device=DEV))
            efg.balance_loss_grad(a, ids, [0, 700], 1.0, 0.1, *o, g)
            outs.append((g, *o))
        assert all(torch.equal(x, y) for x, y in zip(*outs))
        a = z.clone()
        efg.balance_grad(a, 2, [0, 700], 1.0, 0.1, outs[0][2], outs[0][3], a)
        assert torch.equal(a, outs[0][0])


def test_no_tokens():
    z = torch.zeros(0, 8, device=DEV)
    o = (torch.full((2,), 3.0, device=DEV), torch.full((2, 8), 3, dtype=torch.int32, device=DEV),
         torch.full((2,), 3, dtype=torch.int32, device=DEV))
    efg.balance_loss(z, torch.zeros(0, 2, dtype=torch.int32, device=DEV), [0, 0, 0], 1.0, 1.0, *o)
    assert o[0].tolist() == [0.0, 0.0] and not o[1].any() and not o[2].any()


def test_equal_calls_give_equal_bits():
    z = logits(20000, 64, 19, scale=1.5)
    ids = route(z, 4, 20)
    outs = []
    for _ in range(3):
        o = (torch.empty(2, device=DEV), torch.empty(2, 64, dtype=torch.int32, device=DEV),
             torch.empty(2, dtype=torch.int32, device=DEV), torch.empty_like(z))
        efg.balance_loss_grad(z, ids, [0, 9000, 20000], 1.0, 0.1, *o)
        outs.append(o)
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_offsets_beyond_32_bits():
    stride = (1 << 30) + 24
    flat = torch.empty(2 * stride + 64, dtype=torch.bfloat16, device=DEV)
    z = flat.as_strided((3, 64), (stride, 1))
    z.copy_(logits(3, 64, 21))
    check(z, route(z, 2, 22), [0, 3])


def test_gradient_against_differences_of_the_loss():
    z = logits(6, 5, 23, scale=1.0)
    ids = route(z, 2, 24)
    o = (torch.empty(1, device=DEV), torch.empty(1, 5, dtype=torch.int32, device=DEV),
         torch.empty(1, dtype=torch.int32, device=DEV), torch.empty_like(z))
    efg.balance_loss_grad(z, ids, [0, 6], 0.7, 0.3, *o)
    x, i, h = f64(z), ids.cpu().numpy(), 1e-5
    for t in range(6):
        for e in range(5):
            hi, low = x.copy(), x.copy()
            hi[t, e] += h
            low[t, e] -= h
            d = (lo.balance(hi, i, [0, 6], 0.7, 0.3)[0]
                 - lo.balance(low, i, [0, 6], 0.7, 0.3)[0])[0] / (2 * h)
            assert abs(float(o[3][t, e]) - d) <= 2e-9 + 10 * delta(5, 4.0)


def test_on_another_stream_and_in_a_graph():
    z = logits(5000, 64, 25, torch.bfloat16, scale=1.5)
    ids = route(z, 4, 26)
    offs = [0, 1000, 5000]
    ws = torch.empty(efg.balance_workspace_size(5000, 64, 4, offs), dtype=torch.uint8, device=DEV)
    o = (torch.empty(2, device=DEV), torch.empty(2, 64, dtype=torch.int32, device=DEV),
         torch.empty(2, dtype=torch.int32, device=DEV), torch.empty_like(z))

    def step():
        efg.balance_loss_grad(z, ids, offs, 1.0, 0.1, *o, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want = [t.clone() for t in o]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in o:
        t.fill_(3)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(o, want))
