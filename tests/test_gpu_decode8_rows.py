"""The decode step over the 8-bit cache by the number of query rows of a key/value head (each count of eights has its
kernel), NaN codes at every place of a row, and int8 blocks with one large row; against the definition in 64 bits."""
import math

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
@pytest.mark.parametrize("size", [100.0, 3000.0])
def test_int8_blocks_with_one_large_row(d, G, n, size):
    """One key and one value of each block `size` times the others, whose codes are then few or zero.

    The bound.  The kernel multiplies code + 128 and starts its sums at -128 times the other operand's sum, so that its
    rounding errors go with (255 + 128) where the codes may be zero: a score is off by (d / 16 + 3) 2^-22 scale ks 383
    sum |q| more (d / 16 additions, its start and its scaling), ks the largest scale of the blocks, and a mean of values
    by (64 / 16 + 3) 2^-22 383 vs."""
    L, block = 900, 64
    gen = torch.Generator().manual_seed(67)
    cache, model = fresh(1, 1, L, d, torch.int8, block), ref.Model(1, 1, d, torch.int8, block)
    k, v = torch.randn(1, 1, L, d, generator=gen), torch.randn(1, 1, L, d, generator=gen)
    for x, at in ((k, 7), (v, 40)):
        x[0, 0, at::block] *= size
    fill(cache, model, k.bfloat16(), v.bfloat16(), [0, L], [L])
    q = (torch.randn(1, G, n, d, generator=gen) / math.sqrt(size)).bfloat16()
    gate, ws = torch.ones(1, n), logo.decode8_workspace(cache, G, n)
    for W, tau in ((200, 2.0), (50, 0.0)):
        out, _ = logo.decode8(q.cuda(), cache, ints([L]), gate.cuda(), torch.tensor([tau], device="cuda"), W, ws=ws)
        logo.check(ws)
        kk, vv = model.values("k", 0), model.values("v", 0)
        want, bound = ref.decode(q[0], kk, vv, gate[0], tau, W)
        ks, vs = model.quantised("k", 0)[1].max().item(), model.quantised("v", 0)[1].max().item()
        es = (d / 16 + 3) * 2.0 ** -22 / math.sqrt(d) * ks * 383 * q[0].double().abs().sum(-1, keepdim=True)
        assert es.max() < 0.05
        extra = (2 if tau < 1 else 1) * (2.1 * es * vv.abs().amax() + 7 * 2.0 ** -22 * 383 * vs)
        assert ((out[0].double().cpu() - want).abs() <= bound + extra).all(), (W, tau)
