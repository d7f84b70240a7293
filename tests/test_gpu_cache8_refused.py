"""Rows that the 8-bit cache refuses: one fault to a case, on a known sequence; that sequence stays as it was, its new
length is its start, and the others of the batch are served."""
import pytest
import torch

import token_level_dynamic_seq_b200 as logo
from tests.cache8_reference import Model
from tests.test_gpu_cache8 import check, fresh, ints, randn, same, workspace

pytestmark = pytest.mark.gpu

B, HKV, D, LMAX, BLOCK, HELD, ROWS, LONGEST = 4, 2, 64, 200, 64, 50, 60, 30

# what is wrong, the sequence, packed offsets, starts
FAULTS = [
    ("offsets out of order", 3, [0, 10, 20, 30, 15], [50, 50, 50, 50]),
    ("offsets beyond the rows", 3, [0, 10, 20, 40, 61], [50, 50, 50, 50]),
    ("longer than stated", 0, [0, 31, 40, 50, 60], [50, 50, 50, 50]),
    ("a negative offset", 0, [-1, 10, 20, 30, 40], [50, 50, 50, 50]),
    ("a negative start", 1, [0, 10, 20, 30, 40], [50, -1, 50, 50]),
    ("behind the cache's end", 2, [0, 10, 20, 41, 60], [50, 50, 180, 50]),
]


def prepared(dtype):
    gen = torch.Generator().manual_seed(11)
    cache, model, ws = fresh(B, HKV, LMAX, D, dtype, BLOCK), Model(B, HKV, D, dtype, BLOCK), workspace()
    k, v = randn(gen, B, HKV, HELD, D), randn(gen, B, HKV, HELD, D)
    logo.cache8_append(cache, k.cuda(), v.cuda(), ints([0] * B), ws=ws)
    logo.check(ws)
    for b in range(B):
        model.append(b, 0, k[b], v[b])
    return gen, cache, model


def bits(cache, b):
    return [t[b].contiguous().view(torch.uint8).clone() for t in
            (cache.k, cache.v, cache.k_scale, cache.v_scale, cache.k_tail, cache.v_tail)]


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("fault", FAULTS, ids=lambda f: f[0].replace(" ", "_"))
def test_append(fault, dtype):
    _, bad, cu, starts = fault
    gen, cache, model = prepared(dtype)
    k, v = randn(gen, 1, HKV, ROWS, D), randn(gen, 1, HKV, ROWS, D)
    was, new, ws = bits(cache, bad), ints([-7] * B), workspace()
    logo.cache8_append(cache, k.cuda(), v.cuda(), ints(starts), ws=ws, cu_seqlens=ints(cu), max_seqlen=LONGEST, new_len=new)
    with pytest.raises(logo.LogoError) as e:
        logo.check(ws)
    assert e.value.status == 1
    lens = [HELD] * B
    for b in range(B):
        if b != bad:
            model.append(b, starts[b], k[0, :, cu[b]:cu[b + 1]], v[0, :, cu[b]:cu[b + 1]])
            lens[b] = starts[b] + cu[b + 1] - cu[b]
    assert new.tolist() == [starts[b] if b == bad else lens[b] for b in range(B)]
    assert all(torch.equal(x, y) for x, y in zip(was, bits(cache, bad)))
    check(cache, model, lens)


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("fault", FAULTS, ids=lambda f: f[0].replace(" ", "_"))
def test_read(fault, dtype):
    _, bad, cu, starts = fault
    gen, cache, model = prepared(dtype)
    starts = [s - HELD if s == HELD else s for s in starts]      # positions that were written
    out = tuple(torch.full((1, HKV, ROWS, D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    ws = workspace()
    logo.cache8_read(cache, ints(starts), ROWS, ws=ws, cu_seqlens=ints(cu), max_seqlen=LONGEST, out=out)
    with pytest.raises(logo.LogoError) as e:
        logo.check(ws)
    assert e.value.status == 1
    for x, got in zip("kv", out):
        want = torch.full((1, HKV, ROWS, D), 3.0, dtype=torch.bfloat16)
        for b in range(B):
            if b != bad:
                n = cu[b + 1] - cu[b]
                want[0, :, cu[b]:cu[b + 1]] = model.values(x, b)[:, starts[b]:starts[b] + n].float().bfloat16()
        assert same(got.cpu(), want)
