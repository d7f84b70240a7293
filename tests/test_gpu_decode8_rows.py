"""The decode step over the 8-bit cache by the number of query rows of a key/value head (each count of eights has its
kernel), NaN codes at every place of a row, and blocks with one large row; against the definition in 64 bits."""
import pytest
import torch

import token_level_dynamic_seq_b200 as logo
from tests import cache8_reference as ref
from tests.test_gpu_cache8 import fresh, ints
from tests.test_gpu_decode8 import TYPES, build, fill, go

pytestmark = pytest.mark.gpu

# query heads of a group, new tokens: 9 to 32 rows
ROWS = [(9, 1), (13, 1), (2, 7), (5, 3), (16, 1), (17, 1), (6, 3), (19, 1), (5, 4), (7, 3), (11, 2), (1, 23), (8, 3), (24, 1),
        (5, 5), (9, 3), (29, 1), (2, 15), (31, 1), (8, 4)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", ROWS)
def test_every_count_of_rows(dtype, d, G, n):
    lens = [1500, 1499, 700, 31, 1]
    cache, model, gen = build(5, 1, 1500, d, dtype, 64, lens, seed=100 * G + n)
    for W in (1, 130, 5000):
        go(cache, model, gen, G, n, W, lens)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", [(1, 2), (2, 4), (4, 5), (3, 8)])
def test_nan_codes_reach_the_tokens_and_columns_that_see_them(d, G, n):
    """e4m3 NaN values in every column of the drafts' own positions, of the windows' first positions and behind the first
    draft's global branch, one to a row: each makes that column NaN for the tokens that see the row."""
    L, W, block = 500, 70, 64
    gen = torch.Generator().manual_seed(61)
    k = torch.randn(1, 1, L, d, generator=gen).bfloat16()
    clean = torch.randn(1, 1, L, d, generator=gen).bfloat16()
    q = torch.randn(1, G, n, d, generator=gen).bfloat16()
    gate = torch.full((1, n), -1.0)
    gate[0, 1] = 1.0                              # the second draft is global
    tau, lens = torch.zeros(1, device="cuda"), ints([L])
    first = L - n - W + 1                         # token 0's first position
    places = [L - n + i for i in range(n)] + [first + i for i in range(n)] + [first - 1, 3]
    for shift in range(0, d, 5):
        v, seen = clean.clone(), torch.zeros(n, d, dtype=torch.bool)
        for j, pos in enumerate(places):
            col = (shift + 11 * j) % d
            v[0, 0, pos, col] = float("nan")
            for i in range(n):
                t = L - n + i
                seen[i, col] |= pos <= t and (i == 1 or pos > t - W)
        cache, model = fresh(1, 1, L, d, torch.float8_e4m3fn, block), ref.Model(1, 1, d, torch.float8_e4m3fn, block)
        fill(cache, model, k, v, [0, L], [L])
        ws = logo.decode8_workspace(cache, G, n)
        out, _ = logo.decode8(q.cuda(), cache, lens, gate.cuda(), tau, W, ws=ws)
        logo.check(ws)
        got = out[0].double().cpu()
        assert torch.equal(torch.isnan(got), seen.expand(G, n, d)), shift
        want, bound = ref.decode(q[0], model.values("k", 0), torch.nan_to_num(model.values("v", 0), 0.0), gate[0], 0.0, W)
        assert ((got - want).abs() <= bound)[~seen.expand(G, n, d)].all(), shift


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", [(4, 1), (8, 2), (8, 3), (8, 4)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [10.0, 100.0, 3000.0, 1e6])
def test_blocks_with_one_large_row(size, dtype, d, G, n):
    """One key and one value of each block `size` times the others, whose codes are then few or zero: the error goes with
    the values that the codes stand for, not with the largest of the block."""
    L, block = 900, 64
    gen = torch.Generator().manual_seed(67)
    cache, model = fresh(1, 1, L, d, dtype, block), ref.Model(1, 1, d, dtype, block)
    k, v = torch.randn(1, 1, L, d, generator=gen), torch.randn(1, 1, L, d, generator=gen)
    for x, at in ((k, 7), (v, 40)):
        x[0, 0, at::block] *= size
    v[0, 0, 40::block, 1::2] = 0.0                # (in half of the columns the others are all there is)
    fill(cache, model, k.bfloat16(), v.bfloat16(), [0, L], [L])
    for W, tau in ((200, 2.0), (50, 0.0), (5, 0.0)):
        go(cache, model, gen, G, n, W, [L], tau=tau, gate=torch.ones(1, n), qsize=size ** -0.5)
