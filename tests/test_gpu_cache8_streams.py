"""The 8-bit cache's calls on a stream that is not the current one: what they allocate is not memory that the current
stream's queued work still uses."""
import pytest
import torch

import token_level_dynamic_seq_b200 as logo
from tests import cache8_reference as ref
from tests.test_gpu_cache8 import fresh, ints
from tests.test_gpu_decode8 import fill

pytestmark = pytest.mark.gpu


def test_memory_freed_on_the_current_stream_is_not_written_on_another():
    """A tensor as large as the call's result is copied behind a long kernel and freed on the host; the call on a second
    stream, which does not wait for the copy, must not write over it."""
    B, Hkv, d, n, L = 2, 2, 128, 4, 900
    gen = torch.Generator().manual_seed(51)
    cache, model = fresh(B, Hkv, L, d, torch.int8, 64), ref.Model(B, Hkv, d, torch.int8, 64)
    k, v = (torch.randn(1, Hkv, B * L, d, generator=gen).bfloat16() for _ in "kv")
    fill(cache, model, k, v, [0, L, 2 * L], [L, L])
    q = torch.randn(B, 8, n, d, generator=gen).bfloat16().cuda()
    gate, tau, held = torch.ones(B, n, device="cuda"), torch.zeros(1, device="cuda"), ints([L] * B)
    at, side = ints([0] * B), torch.cuda.Stream()
    size = logo.load_library().logo_decode8_workspace_size(cache._ref, 8, n)
    for shape, dtype, call in (
            ((B, 8, n, d), torch.bfloat16, lambda: logo.decode8(q, cache, held, gate, tau, 100, stream=side)[0]),
            ((B, n), torch.int32, lambda: logo.decode8(q, cache, held, gate, tau, 100, stream=side)[1]),
            ((2, B, Hkv, L, d), torch.bfloat16, lambda: logo.cache8_read(cache, at, L, stream=side)[0]),
            ((size,), torch.uint8, lambda: logo.decode8_workspace(cache, 8, n, stream=side))):
        want = call()
        torch.cuda.synchronize()
        want = want.clone()
        x = torch.full(shape, 7, dtype=dtype, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        y = x.clone()
        was = x.untyped_storage().data_ptr()
        del x
        got = call()
        assert got.untyped_storage().data_ptr() != was
        side.synchronize()
        torch.cuda.synchronize()
        assert (y == 7).all()
        if dtype != torch.uint8:
            assert torch.equal(got, want)


def test_results_freed_while_the_current_stream_reads_them():
    """A result is read on the current stream behind a long kernel and freed; further calls on the second stream must not
    get its memory before it was read."""
    B, Hkv, d, L = 1, 2, 64, 500
    gen = torch.Generator().manual_seed(52)
    cache, model = fresh(B, Hkv, L, d, torch.float8_e4m3fn, 64), ref.Model(B, Hkv, d, torch.float8_e4m3fn, 64)
    k, v = (torch.randn(1, Hkv, L, d, generator=gen).bfloat16() for _ in "kv")
    fill(cache, model, k, v, [0, L], [L])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    starts = [ints([i]) for i in range(5)]
    torch.cuda.synchronize()
    want = logo.cache8_read(cache, starts[0], 400)[0].clone()
    first, second = logo.cache8_read(cache, starts[0], 400, stream=side)
    side.synchronize()
    torch.cuda._sleep(100_000_000)
    y = first.clone()
    del first, second
    for at in starts[1:]:
        logo.cache8_read(cache, at, 400, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
