"""ef_logits_topk against the 64-bit oracle: positions, values and counts
exactly, the tail within the bound of losscheck.py."""

import math

import numpy as np
import pytest
import torch

import error_feedback_gradient_gb300 as efg
from losscheck import U, assert_within, delta, f64, largest
from oracle import loss_oracle as lo

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def logits(rows, vocab, seed, dtype=torch.float32, pad=0, shift=0, scale=3.0):
    """[rows, vocab] in rows of vocab + pad elements, starting `shift` elements
    into an allocation."""
    flat = torch.zeros(shift + rows * (vocab + pad) + 8, dtype=dtype, device=DEV)
    x = flat[shift:shift + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]
    x.copy_(torch.randn(rows, vocab, generator=_gen(seed), device=DEV) * scale)
    return x


def run(x, k, tau=1.0, stream=None):
    rows = x.shape[0]
    out = (torch.full((rows, k), 7.0, device=DEV),
           torch.full((rows, k), 7, dtype=torch.int32, device=DEV),
           torch.full((rows,), 7, dtype=torch.int32, device=DEV),
           torch.full((rows,), 7.0, device=DEV))
    efg.logits_topk(x, k, tau, *out, stream=stream)
    return out


def check(x, k, tau=1.0):
    v, i, c, tail = run(x, k, tau)
    wv, wi, wc, wtail = lo.logits_topk(f64(x), k, tau)
    assert np.array_equal(c.cpu().numpy(), wc), "counts"
    assert np.array_equal(i.cpu().numpy(), wi), "indices"
    assert np.array_equal(f64(v), wv, equal_nan=True), "values"
    span = largest(f64(x)) / tau
    bound = delta(x.shape[1], span) + U * np.abs(np.nan_to_num(wtail, neginf=0.0))
    assert_within(f64(tail), wtail, bound, "tail")
    return v, i, c, tail


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab,k", [
    (1, 1, 1), (3, 2, 1), (5, 7, 7), (4, 255, 10), (9, 1000, 10), (2, 1000, 1000),
    (3, 4099, 64), (2, 8192, 0), (3, 30522, 64), (2, 30522, 1024), (1, 131071, 256),
    (2, 262147, 100), (1, 300007, 33)])
def test_packets(dtype, rows, vocab, k):
    check(logits(rows, vocab, 10 * vocab + k, dtype), k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(1, 0), (6, 0), (0, 1), (3, 5), (8, 8)])
def test_row_strides_and_alignment(dtype, pad, shift):
    check(logits(5, 3001, 3, dtype, pad, shift), 50, 2.0)


@pytest.mark.parametrize("tau", [0.25, 1.0, 7.5])
def test_temperatures(tau):
    check(logits(3, 5000, 4), 20, tau)


@pytest.mark.parametrize("dtype", TYPES)
def test_ties_go_to_the_lower_index(dtype):
    x = logits(4, 9001, 5, dtype)
    x[0] = 1.0                                          # all equal
    x[1] = torch.round(x[1].float() / 3).to(dtype)      # a few distinct values
    x[2] = 0.0
    x[2, ::2] = -0.0                                    # zeros of both signs tie
    x[3, 100:9000] = x[3].max()                         # a long run of the largest
    check(x, 100)


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_and_special_values(dtype):
    low = torch.finfo(dtype).min
    x = logits(8, 2050, 6, dtype)
    x[0] = -math.inf                                    # nothing left
    x[1, 5:] = -math.inf                                # fewer than k left
    x[2] = low                                          # the type's lowest everywhere
    x[3, 17:] = low
    x[4, torch.rand(2050, generator=_gen(1), device=DEV) < 0.7] = -math.inf
    x[5, 3] = math.nan
    x[6, [0, 2049]] = math.inf
    x[7, 1000] = torch.finfo(dtype).max                 # one entry far above the rest
    check(x, 12)


def test_values_sorted_either_way():
    x = torch.arange(20000, device=DEV, dtype=torch.float32).flip(0).view(2, 10000) / 500
    check(x.contiguous(), 64)
    check(x.flip(1).contiguous(), 64)


def test_large_values_side_by_side():
    # the largest entries all within one short stretch of the row
    x = logits(3, 40000, 8)
    x[:, 20000:21500] += 30.0
    check(x, 1000)


def test_k_zero_is_the_log_sum_exp():
    x = logits(6, 777, 9)
    counts = torch.full((6,), 9, dtype=torch.int32, device=DEV)
    tail = torch.empty(6, device=DEV)
    efg.logits_topk(x, 0, 1.0, None, None, counts, tail)
    assert counts.tolist() == [0] * 6
    assert_within(f64(tail), torch.logsumexp(x.double(), 1).cpu().numpy(),
                  delta(777, largest(f64(x))) + 20 * U, "tail")


def test_no_rows_and_no_vocabulary():
    run(torch.zeros(0, 5, device=DEV), 3)
    counts = torch.full((2,), 9, dtype=torch.int32, device=DEV)
    tail = torch.empty(2, device=DEV)
    efg.logits_topk(torch.zeros(2, 0, device=DEV), 0, 1.0, None, None, counts, tail)
    assert counts.tolist() == [0, 0] and tail.tolist() == [-math.inf] * 2


def test_tail_is_optional():
    x = logits(2, 900, 11)
    v, i, c, _ = run(x, 9)
    v2, i2, c2 = torch.empty_like(v), torch.empty_like(i), torch.empty_like(c)
    efg.logits_topk(x, 9, 1.0, v2, i2, c2)
    assert torch.equal(v, v2) and torch.equal(i, i2) and torch.equal(c, c2)


def test_many_rows_match_few():
    """The same rows one at a time and in a large batch: the packets agree
    (other sizes may take another kernel), equal calls agree bit for bit."""
    x = logits(700, 6000, 12, torch.bfloat16)
    big, again = run(x, 40), run(x, 40)
    assert all(torch.equal(a, b) for a, b in zip(big, again))
    for r in (0, 1, 699):
        one = run(x[r:r + 1], 40)
        assert torch.equal(one[0][0], big[0][r]) and torch.equal(one[1][0], big[1][r])
        assert abs(float(one[3][0] - big[3][r])) <= 2 * delta(6000, 15.0) + 40 * U


def test_offsets_beyond_32_bits():
    stride = (1 << 30) + 24
    flat = torch.empty(2 * stride + 1000, dtype=torch.bfloat16, device=DEV)
    x = flat.as_strided((3, 1000), (stride, 1))
    x.copy_(torch.randn(3, 1000, generator=_gen(3), device=DEV))
    check(x, 10)


def test_on_another_stream():
    x = logits(64, 30522, 13, torch.bfloat16)
    want = run(x, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = x * 2
        got = run(y, 64, 2.0)
    side.synchronize()
    assert torch.equal(got[1], want[1]) and torch.equal(got[0], want[0] * 2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab,k", [(70001, 64), (131071, 1024), (150000, 300), (70001, 400)])
def test_rows_in_several_chunks(dtype, vocab, k):
    # in any order, ascending (every chunk above all before it), descending, and
    # the largest few in the last chunk
    x = logits(5, vocab, k, dtype)
    x[1] = x[1].sort().values
    x[2] = x[2].sort(descending=True).values
    x[3, vocab - 2000:] += 20.0
    x[4, :vocab // 2] = -math.inf
    check(x, k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab,k", [(130, 70), (1000, 500), (4076, 310), (9000, 300), (70001, 80)])
def test_as_many_nan_as_the_packet_holds(dtype, vocab, k):
    x = logits(4, vocab, vocab + k, dtype)
    x[0] = math.nan
    x[1, torch.randperm(vocab, generator=_gen(3), device=DEV)[:k]] = math.nan
    x[2] = -math.inf
    x[2, ::3] = math.nan
    x[3, :k] = math.inf
    check(x, k)


@pytest.mark.parametrize("dtype,vocabs", [(torch.float32, range(960, 1040, 3)),
                                          (torch.float32, range(448, 520, 5)),
                                          (torch.bfloat16, range(960, 1040, 7)),
                                          (torch.float16, range(1980, 2060, 7))])
def test_candidates_lists_of_every_size(dtype, vocabs):
    # shared memory from a little below to a little above what a launch gets unasked
    for vocab in vocabs:
        for k in (60, 97, 130, 250):
            check(logits(2, vocab, vocab + k, dtype), k)
