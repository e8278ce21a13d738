"""Corners of the cache's operators: digits of the fixed-point products, bounds of a call's size, the order of
loads that a kernel's waits count on, and values at the ends."""
import pytest
import torch

import kv_reference as ref
from gpu_util import require_gpu
from test_kv import attend

gpu = pytest.mark.gpu
TYPES = list(ref.TYPES.values())


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("D,ps", [(64, 16), (128, 64), (192, 16), (256, 24)])
def test_a_token_with_large_values_leaves_the_others_their_digits(D, ps, dtype):
    """64 tokens of weight 1, one of which has 512 times the others' scale, and codes 0 in every other column.

    There the other tokens' sums come out to half a step of the fixed-point weights for each token, which is
    512 / 8355000 / 2 of the others' scale; the fp32 operations on the way (quotient, factor, products, sum,
    division) take 16 roundings at most; the output has its own."""
    require_gpu()
    n, big, step = 64, 7, 2.0 ** -10
    g = torch.Generator().manual_seed(D)
    pages = -(-n // ps)
    k = torch.randint(-127, 128, (pages, 1, ps, D), generator=g).to(torch.int8)
    v = torch.randint(90, 128, (pages, 1, ps, D), generator=g).to(torch.int8)
    v[big // ps, 0, big % ps, ::2] = 0
    ks, vs = torch.full((pages, 1, ps), 0.01), torch.full((pages, 1, ps), step)
    vs[big // ps, 0, big % ps] = 512 * step
    table, lengths = torch.arange(pages)[None], torch.tensor([n])
    o, lse = attend(torch.zeros(1, 2, D, dtype=dtype), (k, v, ks, vs), table, lengths)
    t = torch.arange(n)
    want = (v[t // ps, 0, t % ps].double() * vs[t // ps, 0, t % ps].double()[:, None]).mean(0)
    size = (v[t // ps, 0, t % ps].double().abs().sum(0) * 512 * step / ref.TOP[3] / 2) / n
    bound = size + 16 * ref.U32 * (want + size)
    bound = bound + ref.half_step(want + bound, dtype)
    assert bool(((o[0].double() - want).abs() <= bound)[:, ::2].all()), float(((o[0].double() - want).abs() / bound)[:, ::2].max())
    assert bool(((o[0].double() - want).abs() <= bound).all())


@gpu
@pytest.mark.parametrize("at", [40000.3125, 39999.6875, 40000.4375, 300000.3125, 3000000.25])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_query_values_are_rounded_to_the_nearest_step(at, sign):
    """A query whose largest value is 8355000 steps of 2^-22, by which the others come out as fractions of a step.

    The largest meets codes 0, so the score is the others' sum: off by half a step each, and 16 roundings of the
    fp32 operations behind it.  One token's log-sum-exp is its score."""
    require_gpu()
    D, step = 64, 2.0 ** -22
    q = torch.full((1, 1, D), sign * at * step)
    q[0, 0, 0] = ref.TOP[3] * step
    k = torch.full((1, 1, 16, D), 127, dtype=torch.int8)
    k[..., 0] = 0
    v, s = torch.zeros_like(k), torch.ones(1, 1, 16)
    _, lse = attend(q, (k, v, s, s), torch.zeros(1, 1), torch.tensor([1]), scale=1.0)
    want = sign * at * step * 127 * (D - 1)
    assert abs(float(lse) - want) <= 127 * (D - 1) * step / 2 + 16 * ref.U32 * abs(want)
