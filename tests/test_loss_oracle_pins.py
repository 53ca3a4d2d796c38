"""The 64-bit definitions of the training losses, pinned by worked examples,
by finite differences, and by mistakes that must be noticed."""

import math

import numpy as np
import pytest

from oracle import loss_oracle as lo

NEG = -math.inf


def test_packet_of_a_worked_row():
    x = np.array([[1.0, 3.0, NEG, 3.0, -2.0], [NEG, 0.0, NEG, NEG, NEG], [NEG] * 5])
    v, i, c, tail = lo.logits_topk(x, 2, 1.0)
    assert i.tolist() == [[1, 3], [1, -1], [-1, -1]] and c.tolist() == [2, 1, 0]
    assert v.tolist() == [[3.0, 3.0], [0.0, 0.0], [0.0, 0.0]]
    assert tail[0] == pytest.approx(math.log(math.exp(1) + math.exp(-2)))
    assert tail[1] == NEG and tail[2] == NEG
    _, i, _, _ = lo.logits_topk(np.array([[0.0, math.nan, -0.0, 5.0]]), 3, 1.0)
    assert i.tolist() == [[0, 1, 3]]                  # NaN first, then 5, then the lower zero


def test_distill_of_a_worked_row():
    # student uniform over 4, teacher 3 : 1 over two of them, nothing elsewhere
    s, t = np.zeros(4), np.log([3.0, 1.0])
    loss, stats, g = lo.distill_row(s, [1, 2], t, None, 1.0)
    assert loss == pytest.approx(0.75 * math.log(3) + 0.25 * math.log(1))
    assert g == pytest.approx([0.25, -0.5, 0.0, 0.25])
    b = math.log(3)
    assert stats == pytest.approx((0.0, math.log(2), math.log(4), b, math.log(4) - b, 0.0))
    # the same with a tail of weight 4: p = 3/8, 1/8, 1/2
    loss, stats, g = lo.distill_row(s, [1, 2], t, math.log(4), 1.0)
    want = 3 / 8 * math.log(3 / 2) + 1 / 8 * math.log(1 / 2) + 1 / 2 * math.log(1)
    assert loss == pytest.approx(want) and stats[5] == pytest.approx(0.5)
    assert g == pytest.approx([0.0, 0.25 - 3 / 8, 0.25 - 1 / 8, 0.0])


def test_distill_rows_with_nothing_left():
    s = np.array([0.5, NEG, 1.0])
    for idx, t, tail, sv in [([], [], None, s), ([1], [2.0], None, s), ([0], [1.0], 0.3,
                                                                       np.full(3, NEG))]:
        loss, _, g = lo.distill_row(sv, idx, t, tail, 1.0)
        assert loss == 0.0 and not g.any()
    # no packet but a tail: teacher and student both put everything there
    loss, stats, g = lo.distill_row(s, [], [], 1.7, 1.0)
    assert loss == pytest.approx(0.0) and stats[5] == 1.0 and not g.any()
    # a packet over the whole row has no place for the tail
    loss, stats, _ = lo.distill_row(np.zeros(2), [0, 1], [0.0, 0.0], 9.0, 1.0)
    assert loss == pytest.approx(0.0) and stats[5] == 0.0


@pytest.mark.parametrize("tail", [None, 0.7])
@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_distill_gradient_is_the_loss_difference(tail, tau):
    rng = np.random.default_rng(3)
    s = rng.standard_normal(9) * 2
    s[4] = NEG
    idx, t = [0, 3, 4, 7], rng.standard_normal(4) * 2
    _, _, g = lo.distill_row(s, idx, t, tail, tau)
    h = 1e-6
    for v in range(9):
        if s[v] == NEG:
            assert g[v] == 0.0
            continue
        hi, low = s.copy(), s.copy()
        hi[v] += h
        low[v] -= h
        d = (lo.distill_row(hi, idx, t, tail, tau)[0]
             - lo.distill_row(low, idx, t, tail, tau)[0]) / (2 * h)
        assert g[v] == pytest.approx(d, abs=1e-8)
    assert g.sum() == pytest.approx(0.0, abs=1e-12)   # a shift of all logits changes nothing


def test_distill_ends_at_the_teacher():
    # a student equal to the teacher, seen through a packet and its tail
    rng = np.random.default_rng(4)
    x = rng.standard_normal((1, 40)) * 3
    v, i, c, tail = lo.logits_topk(x, 6, 1.7)
    loss, _, g = lo.distill(x, i, v, c, tail, 1.7)
    assert loss[0] == pytest.approx(0.0, abs=1e-14) and np.abs(g).max() < 1e-14
    wrong_tail = lo.distill(x, i, v, c, tail + 0.5, 1.7)
    assert wrong_tail[0][0] > 1e-4


def test_balance_of_a_worked_segment():
    # two tokens, two experts, uniform router, both sent to expert 0
    z = np.zeros((2, 2))
    ids = np.array([[0], [0]], np.int32)
    loss, c, n, g = lo.balance(z, ids, [0, 2], 1.0, 0.0)
    assert loss[0] == pytest.approx(2.0 * 0.5) and c.tolist() == [[2, 0]] and n.tolist() == [2]
    # f = (2, 0): dz = p (f - 1) / n
    assert g == pytest.approx(np.array([[0.25, -0.25]] * 2))
    loss, _, _, _ = lo.balance(z, ids, [0, 2], 0.0, 3.0)
    assert loss[0] == pytest.approx(3.0 * math.log(2) ** 2)


def test_balance_gradient_is_the_loss_difference():
    rng = np.random.default_rng(5)
    z = rng.standard_normal((7, 5))
    z[2, 1] = NEG
    z[5] = NEG
    ids = rng.integers(-1, 6, (7, 2)).astype(np.int32)
    mask = np.array([1, 1, 1, 0, 1, 1, 1], np.uint8)
    offs, weights = [0, 4, 4, 7], np.array([1.5, 2.0, -0.5])
    _, _, _, g = lo.balance(z, ids, offs, 0.3, 0.2, mask, weights)
    h = 1e-6
    for t in range(7):
        for e in range(5):
            if z[t, e] == NEG:
                assert g[t, e] == 0.0
                continue
            hi, low = z.copy(), z.copy()
            hi[t, e] += h
            low[t, e] -= h
            d = (lo.balance(hi, ids, offs, 0.3, 0.2, mask)[0]
                 - lo.balance(low, ids, offs, 0.3, 0.2, mask)[0]) / (2 * h)
            assert g[t, e] == pytest.approx(float(d @ weights), abs=1e-8)
    assert not g[3].any()
