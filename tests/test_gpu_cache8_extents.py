"""The 8-bit cache's calls at the ends of their sizes: caches shorter than what a kernel copies at a time, and calls on a
second stream that are captured into a graph together with the current one's."""
import pytest
import torch

import token_level_dynamic_seq_b200 as logo
from tests import cache8_reference as ref
from tests.test_gpu_cache8 import check, fresh, ints, randn, workspace
from tests.test_gpu_decode8 import TYPES, build, go, verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lmax", [1, 2, 15, 31, 33, 63, 65])
def test_short_caches(dtype, d, Lmax):
    """Fewer positions than one stage of the decode (32 or 64) or one block of the scales."""
    lens = [Lmax, 1, 0, (Lmax + 1) // 2]
    cache, model, gen = build(4, 2, Lmax, d, dtype, 64 if Lmax % 2 else 128, lens, seed=Lmax)
    check(cache, model, lens)
    for n in (1, 3):
        for W in (1, Lmax, 100):
            go(cache, model, gen, 4, n, W, lens)


def test_a_step_captured_on_two_streams():
    """Append and decode of two layers, each layer on a stream of its own, captured into one graph and replayed: what the
    calls allocate in the capture is theirs."""
    B, Hkv, Hq, d, Lmax, W = 2, 2, 8, 128, 300, 60
    gen = torch.Generator().manual_seed(71)
    lens = [70, 131]
    made = [build(B, Hkv, Lmax, d, t, 64, lens, seed=72 + i) for i, t in enumerate(TYPES)]
    at, held = ints(lens), [ints([0] * B), ints([0] * B)]
    k, v, q = (torch.zeros(B, h, 1, d, dtype=torch.bfloat16, device="cuda") for h in (Hkv, Hkv, Hq))
    gate, tau = torch.zeros(B, 1, device="cuda"), torch.zeros(1, device="cuda")
    ws = [logo.decode8_workspace(m[0], Hq) for m in made]
    main, side, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    outs = [None, None]
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        for i, s in ((0, None), (1, side)):
            logo.cache8_append(made[i][0], k, v, at, ws=ws[i], new_len=held[i], stream=s)
            outs[i] = logo.decode8(q, made[i][0], held[i], gate, tau, W, ws=ws[i], stream=s)
        main.wait_stream(side)
        at.copy_(held[0])
    for _ in range(5):
        kh, vh = randn(gen, B, Hkv, 1, d), randn(gen, B, Hkv, 1, d)
        qh, gh = torch.randn(B, Hq, 1, d, generator=gen).bfloat16(), torch.randn(B, 1, generator=gen)
        for x, y in ((k, kh), (v, vh), (q, qh), (gate, gh)):
            x.copy_(y)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            for _, model, _ in made:
                model.append(b, lens[b], kh[b], vh[b])
        lens = [n + 1 for n in lens]
        for i, (cache, model, _) in enumerate(made):
            logo.check(ws[i])
            assert held[i].tolist() == lens
            verify(cache, model, qh, gh, 0.0, W, lens, *outs[i])


@pytest.mark.parametrize("dtype", TYPES)
def test_the_largest_batch_of_the_sums_either_way(dtype):
    """63 to 66 sequences: the lengths are added up by the joining kernel, or by the first one."""
    for B in (63, 64, 65, 66):
        lens = [(i * 61) % 400 for i in range(B)]
        cache, model, gen = build(B, 2, 400, 128, dtype, 64, lens, seed=B)
        go(cache, model, gen, 4, 2, 50, lens)
