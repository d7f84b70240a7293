"""The decode step over the 8-bit cache where its numbers reach the ends of their range: scales that are not finite,
values near the largest bf16."""
import pytest
import torch

import token_level_dynamic_seq_b200 as logo
from tests import cache8_reference as ref
from tests.test_gpu_cache8 import fresh, ints
from tests.test_gpu_decode8 import TYPES, build, fill, go

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


# n tokens, length, window, the block (of 64) whose scale is bad, tokens that take the global branch
SCALE_CASES = [
    (2, 65, 40, 1, []),              # a new block begins with the second draft
    (3, 66, 200, 1, [0]),            # the same with tokens 1 and 2; token 0 global
    (3, 300, 171, 1, []),            # the block's last position (127) is token 0's first
    (3, 300, 171, 1, [2]),           # token 2 sees it through the global branch only
    (4, 322, 130, 2, []),            # the windows begin at 189 .. 192: the last token sees nothing of 128 .. 191
    (1, 129, 1, 1, []),              # one token that sees nothing of it
    (4, 400, 50, 6, [1]),            # inside every window
    (4, 400, 50, 0, [1, 3]),         # before every window
]


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_a_scale_that_is_not_finite_reaches_the_tokens_that_see_its_block(dtype, d, bad, which):
    for n, L, W, blk, chosen in SCALE_CASES:
        cache, model, gen = build(1, 2, 512, d, dtype, 64, [L], seed=L + n)
        q, gate = torch.randn(1, 4, n, d, generator=gen).bfloat16(), torch.full((1, n), -1.0)
        gate[0, chosen] = 1.0
        getattr(cache, which)[0, :, blk] = bad
        ws = logo.decode8_workspace(cache, 4, n)
        out, _ = logo.decode8(q.cuda(), cache, ints([L]), gate.cuda(), torch.zeros(1, device="cuda"), W, ws=ws)
        logo.check(ws)
        want, bound = ref.decode(q[0], model.values("k", 0), model.values("v", 0), gate[0], 0.0, W)
        got = out[0].double().cpu()
        for i in range(n):
            t = L - n + i
            first = 0 if i in chosen else max(0, t - W + 1)
            if first < 64 * (blk + 1) and t >= 64 * blk:
                # (an infinite key scale may be a weight of zero or one; a value's sum is infinite or NaN)
                if which == "v_scale" or bad != bad:
                    assert not torch.isfinite(got[:, i]).any(), (n, L, W, blk, i)
            else:
                assert ((got[:, i] - want[:, i]).abs() <= bound[:, i]).all(), (n, L, W, blk, i)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,Hq,n", [(128, 4, 1), (64, 4, 4), (128, 8, 3), (128, 8, 4), (64, 1, 20)])
def test_large_values_with_many_equal_weights(dtype, d, Hq, n):
    """Every score is zero, so each output is a mean of thousands of values of one sign, up to 3.3e38: their sum is far
    beyond fp32, their mean is not.  And near the least that a scale stands for (2^-100)."""
    L, W = 9000, 4096
    gen = torch.Generator().manual_seed(41)
    for size in (1e-30, 1e34, 1e36, 3.3e38, -3.3e38):
        cache, model = fresh(1, 1, L, d, dtype, 64), ref.Model(1, 1, d, dtype, 64)
        k = torch.randn(1, 1, L, d, generator=gen).bfloat16()
        v = ((torch.rand(1, 1, L, d, generator=gen) + 1) / 2 * size).bfloat16()
        fill(cache, model, k, v, [0, L], [L])
        for tau, gate in ((1.0, 0.0), (-9.0, -2.5)):      # local only; a share of 0.076 of the global mean
            go(cache, model, gen, Hq, n, W, [L], tau=tau, gate=torch.full((1, n), gate), qsize=0.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,n", [(128, 1), (64, 5), (128, 12)])
def test_small_values_beside_large_ones_of_no_weight(dtype, d, n):
    """Blocks of values of 3e38 whose scores are thousands below the others', first, last and between blocks of 1e-20:
    the small ones are the output."""
    L, W = 1000, 2000
    gen = torch.Generator().manual_seed(43)
    for first in (0, 5, 14):
        cache, model = fresh(1, 1, L, d, dtype, 64), ref.Model(1, 1, d, dtype, 64)
        k, v = torch.randn(1, 1, L, d, generator=gen) * 0.01, torch.randn(1, 1, L, d, generator=gen) * 1e-20
        k[..., 0] = 1.0
        k[0, 0, 64 * first:64 * (first + 1), 0] = -1.0
        v[0, 0, 64 * first:64 * (first + 1)] = 3e38
        fill(cache, model, k.bfloat16(), v.bfloat16(), [0, L], [L])
        q = torch.randn(1, 2, n, d, generator=gen)
        q[..., 0] = 2e4
        gate, ws = torch.ones(1, n), logo.decode8_workspace(cache, 2, n)
        for tau in (0.0, 2.0):
            out, _ = logo.decode8(q.bfloat16().cuda(), cache, ints([L]), gate.cuda(), torch.tensor([tau], device="cuda"), W,
                                  ws=ws)
            logo.check(ws)
            kk, vv = model.values("k", 0), model.values("v", 0)
            vv[:, 64 * first:64 * (first + 1)] = 0.0        # weights of e^-1000 and less
            want, bound = ref.decode(q[0].bfloat16(), kk, vv, gate[0], tau, W)
            assert ((out[0].double().cpu() - want).abs() <= bound).all(), (first, tau)
