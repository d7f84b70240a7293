"""The decode step over the 8-bit cache where its numbers reach the ends of their range: scales that are not finite."""
import pytest
import torch

import token_level_dynamic_seq_b200 as logo
from tests import cache8_reference as ref
from tests.test_gpu_cache8 import ints
from tests.test_gpu_decode8 import TYPES, build

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
