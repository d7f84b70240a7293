"""Rows taken back from the 8-bit cache by an append that brings none: what is left is quantised as if the rows taken
back had never been there."""
import pytest
import torch

import token_level_dynamic_seq_b200 as logo
from tests.cache8_reference import Model
from tests.test_gpu_cache8 import check, fresh, ints, randn, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("d,block", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("packed", [True, False])
def test_drafts_rejected_without_a_new_token(dtype, d, block, packed):
    """Drafts larger than what lies before them raise their block's scale; rejecting all of them brings it back."""
    gen = torch.Generator().manual_seed(block + d)
    B, Hkv = 5, 2
    lens = [block // 2, block - 2, block, 2 * block + 1, 3]
    cache, model, ws = fresh(B, Hkv, 5 * block, d, dtype, block), Model(B, Hkv, d, dtype, block), workspace()
    for b, n in enumerate(lens):
        k, v = randn(gen, Hkv, n, d), randn(gen, Hkv, n, d)
        one = logo.Cache8(*(t[b:b + 1] for t in (cache.k, cache.v, cache.k_scale, cache.v_scale, cache.k_tail, cache.v_tail)))
        logo.cache8_append(one, k[None].cuda(), v[None].cuda(), ints([0]), ws=ws)
        model.append(b, 0, k, v)
    check(cache, model, lens)
    k, v = randn(gen, B, Hkv, 4, d) * 50, randn(gen, B, Hkv, 4, d) * 50
    logo.cache8_append(cache, k.cuda(), v.cuda(), ints(lens), ws=ws)
    keep, new = [0, 1, 2, 0, 4], ints([-7] * B)
    now = [n + i for n, i in zip(lens, keep)]
    none = torch.empty(1 if packed else B, Hkv, 0, d, dtype=torch.bfloat16, device="cuda")
    logo.cache8_append(cache, none, none, ints(now), ws=ws, new_len=new,
                       **(dict(cu_seqlens=ints([0] * (B + 1)), max_seqlen=0) if packed else {}))
    logo.check(ws)
    assert new.tolist() == now
    for b in range(B):
        model.append(b, lens[b], k[b, :, :keep[b]], v[b, :, :keep[b]])
    check(cache, model, now)
