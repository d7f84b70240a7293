"""Quantising into the 8-bit cache and reading it back, on the GPU, against the definition in 64 bits: codes, scales
and tails bit for bit, whatever the pieces in which the rows were appended."""
import pytest
import torch

import token_level_dynamic_seq_b200 as logo
from tests.cache8_reference import Model

pytestmark = pytest.mark.gpu

TYPES = [torch.float8_e4m3fn, torch.int8]


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def fresh(B, Hkv, Lmax, d, dtype, block):
    """A cache whose memory holds what must never be used: NaN everywhere (0x7f codes, NaN scales and tails)."""
    c = logo.cache8(B, Hkv, Lmax, d, "cuda", dtype=dtype, block=block)
    for t in (c.k, c.v):
        t.view(torch.uint8).fill_(0x7f)
    for t in (c.k_scale, c.v_scale, c.k_tail, c.v_tail):
        t.fill_(float("nan"))
    return c


def workspace():
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    ws.zero_()
    return ws


def randn(gen, *shape):
    x = torch.randn(*shape, generator=gen)
    return (x * torch.exp(2 * torch.randn(shape[:-1], generator=gen))[..., None]).bfloat16()   # rows of uneven size


def same(a, b):
    return torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32),
                       b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32))


def check(cache, model, lens, since=None):
    """Codes, scales, tails and values read back of the first lens[b] positions, exactly.  `since`: where the last
    append began; after going back, the tail holds no block before that."""
    B, block = cache.B, cache.block
    for x, codes, scales, tails in (("k", cache.k, cache.k_scale, cache.k_tail), ("v", cache.v, cache.v_scale, cache.v_tail)):
        for b in range(B):
            n = lens[b]
            assert model.length(b) == n
            if n == 0:
                continue
            want, ws = model.quantised(x, b)
            got = codes[b, :, :n].double().cpu()
            assert torch.equal(torch.nan_to_num(got, 1e9), torch.nan_to_num(want, 1e9)), (x, b)
            assert same(scales[b, :, :ws.shape[1]].cpu(), ws), (x, b)
            rows = model.rows[x][b]
            last = (n - 1) // block
            for j in range(max(last - 1, since[b] // block if since else 0), last + 1):
                part = rows[:, j * block:(j + 1) * block]
                assert same(tails[b, :, j % 2, :part.shape[1]].cpu().contiguous(), part.contiguous()), (x, b, j)
    ws = workspace()
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    k, v = logo.cache8_read(cache, ints([0] * B), cu[-1], ws=ws, cu_seqlens=ints(cu), max_seqlen=max(lens))
    logo.check(ws)
    for x, got in (("k", k), ("v", v)):
        for b in range(B):
            if lens[b]:
                c, s = model.quantised(x, b)
                want = (c.float() * s.repeat_interleave(block, 1)[:, :lens[b], None]).bfloat16()
                assert same(torch.nan_to_num(got[0, :, cu[b]:cu[b + 1]].cpu().contiguous(), 7.0), torch.nan_to_num(want, 7.0)), (x, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,Hkv,Lmax,d,block,n", [
    (1, 1, 1, 64, 64, 1), (2, 3, 200, 128, 64, 200), (3, 2, 129, 64, 64, 129), (2, 2, 257, 128, 128, 257),
    (1, 2, 640, 64, 128, 640), (2, 1, 64, 128, 64, 63), (1, 1, 128, 128, 128, 128), (1, 4, 1111, 128, 64, 1000),
])
def test_a_prompt_at_once(dtype, B, Hkv, Lmax, d, block, n):
    gen = torch.Generator().manual_seed(n + d)
    cache, model, ws = fresh(B, Hkv, Lmax, d, dtype, block), Model(B, Hkv, d, dtype, block), workspace()
    k, v = randn(gen, B, Hkv, n, d), randn(gen, B, Hkv, n, d)
    got = ints([-5] * B)
    logo.cache8_append(cache, k.cuda(), v.cuda(), ints([0] * B), ws=ws, new_len=got)
    logo.check(ws)
    assert got.tolist() == [n] * B
    for b in range(B):
        model.append(b, 0, k[b], v[b])
    check(cache, model, [n] * B)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_ragged_pieces_packed(dtype, block, d):
    """Packed appends of uneven pieces, empty ones among them, give what appending at once gives."""
    gen = torch.Generator().manual_seed(block + d)
    B, Hkv, Lmax = 5, 2, 700
    cache, model, ws = fresh(B, Hkv, Lmax, d, dtype, block), Model(B, Hkv, d, dtype, block), workspace()
    lens = [0] * B
    for piece in ([64, 1, 0, 130, 127], [1, 63, 200, 0, 1], [300, 64, 1, 62, 65], [0, 0, 0, 0, 0], [1, 1, 1, 1, 1],
                  [129, 191, 2, 128, 250], [200, 3, 7, 64, 256]):
        cu = [0]
        for n in piece:
            cu.append(cu[-1] + n)
        k, v = randn(gen, 1, Hkv, cu[-1], d), randn(gen, 1, Hkv, cu[-1], d)
        new_len = ints([0] * B)
        logo.cache8_append(cache, k.cuda(), v.cuda(), ints(lens), ws=ws, cu_seqlens=ints(cu), max_seqlen=max(piece),
                           new_len=new_len)
        for b in range(B):
            model.append(b, lens[b], k[0, :, cu[b]:cu[b + 1]], v[0, :, cu[b]:cu[b + 1]])
            lens[b] += piece[b]
        assert new_len.tolist() == lens
        logo.check(ws)
        check(cache, model, lens)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [64, 128])
def test_one_token_at_a_time_with_growing_rows(dtype, block):
    """Every token larger than the ones before it, so every append raises the block's scale; then smaller ones."""
    gen = torch.Generator().manual_seed(3)
    B, Hkv, d, Lmax = 2, 2, 128, 2 * block + 9
    cache, model, ws = fresh(B, Hkv, Lmax, d, dtype, block), Model(B, Hkv, d, dtype, block), workspace()
    at = ints([0] * B)
    for i in range(Lmax):
        f = 1.03 ** (i if i < block else block - i)
        k, v = (torch.randn(B, Hkv, 1, d, generator=gen) * f).bfloat16(), randn(gen, B, Hkv, 1, d)
        nxt = ints([0] * B)
        logo.cache8_append(cache, k.cuda(), v.cuda(), at, ws=ws, new_len=nxt)
        at = nxt
        for b in range(B):
            model.append(b, i, k[b], v[b])
        if i in (0, 1, 17, block - 1, block, block + 5, Lmax - 1):
            check(cache, model, [i + 1] * B)
    logo.check(ws)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [64, 128])
def test_taking_drafts_back(dtype, block):
    """Appending again where the latest append began or within it (in its last two blocks), or at a multiple of the
    block."""
    gen = torch.Generator().manual_seed(5)
    B, Hkv, d, Lmax = 3, 2, 64, 6 * block
    cache, model, ws = fresh(B, Hkv, Lmax, d, dtype, block), Model(B, Hkv, d, dtype, block), workspace()
    lens, before = [0, 0, 0], [0, 0, 0]
    r = torch.Generator().manual_seed(block)
    for step in range(30):
        starts = []
        for b in range(B):
            # the latest append taken back in part or whole, or an earlier multiple of the block, or neither
            low = max(before[b], ((lens[b] - 1) // block - 1) * block)
            back = int(torch.randint(low, lens[b] + 1, (1,), generator=r)) if lens[b] else 0
            far = int(torch.randint(0, lens[b] // block + 1, (1,), generator=r)) * block
            starts.append([back, back, lens[b], far][int(torch.randint(4, (1,), generator=r))])
        n = [1, 4, 5, block - 1, block, 2 * block + 3][int(torch.randint(6, (1,), generator=r))]
        starts = [s if s + n <= Lmax else 0 for s in starts]
        k, v = randn(gen, B, Hkv, n, d), randn(gen, B, Hkv, n, d)
        logo.cache8_append(cache, k.cuda(), v.cuda(), ints(starts), ws=ws)
        for b in range(B):
            model.append(b, starts[b], k[b], v[b])
            lens[b] = starts[b] + n
        before = starts
        check(cache, model, lens, since=starts)
    logo.check(ws)


@pytest.mark.parametrize("dtype", TYPES)
def test_extreme_values(dtype):
    """Zeros, the smallest and largest bf16, infinities and NaN: the scale is over the finite ones."""
    B, Hkv, d, block = 1, 1, 64, 64
    x = torch.zeros(8 * block, d)
    x[0] = 0.0                                            # a zero block
    x[block:2 * block] = 1e-40                            # subnormal: below the floor of 2^-100
    x[2 * block] = 3.3e38
    x[2 * block + 1] = -3.3e38
    x[3 * block] = float("inf")
    x[3 * block + 1, :3] = torch.tensor([float("-inf"), float("nan"), 2.5])
    x[4 * block:5 * block] = float("nan")                 # nothing finite
    x[5 * block, 0], x[5 * block, 1:] = 2.0 ** -100, 2.0 ** -110
    x[6 * block:7 * block] = -0.0
    x[7 * block:] = torch.arange(block * d).view(block, d).float() - 2000
    x = x.bfloat16()[None]
    cache, model, ws = fresh(B, Hkv, 8 * block, d, dtype, block), Model(B, Hkv, d, dtype, block), workspace()
    logo.cache8_append(cache, x[None].cuda(), -x[None].cuda(), ints([0]), ws=ws)
    logo.check(ws)
    model.append(0, 0, x, -x)
    check(cache, model, [8 * block])


@pytest.mark.parametrize("dtype", TYPES)
def test_every_bf16_significand_rounds_as_the_quotient(dtype):
    """All pairs of significands of x and the block's maximum, with ties: 128 blocks of 128 values and their negatives."""
    d, block = 128, 64
    sig = torch.arange(128, 256).float()
    rows = []
    for a in sig:
        part = torch.zeros(block, d)
        for e in range(14):
            part[2 * e] = sig * 2.0 ** -e * (sig * 2.0 ** -e <= a)
            part[2 * e + 1] = -part[2 * e]
        part[block - 1, 0] = a
        rows.append(part)
    x = torch.cat(rows).bfloat16()[None]
    cache, model, ws = fresh(1, 1, x.shape[1], d, dtype, block), Model(1, 1, d, dtype, block), workspace()
    logo.cache8_append(cache, x[None].cuda(), (x[None] * 2.0 ** 50).cuda(), ints([0]), ws=ws)
    logo.check(ws)
    model.append(0, 0, x, x * 2.0 ** 50)
    check(cache, model, [x.shape[1]])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,block", [(64, 64), (128, 128)])
def test_reading_ranges(dtype, d, block):
    """Fixed ranges from any position, and packed ones with an empty sequence; other rows are left as they were."""
    gen = torch.Generator().manual_seed(9)
    B, Hkv, Lmax = 3, 2, 500
    cache, model, ws = fresh(B, Hkv, Lmax, d, dtype, block), Model(B, Hkv, d, dtype, block), workspace()
    k, v = randn(gen, B, Hkv, Lmax, d), randn(gen, B, Hkv, Lmax, d)
    logo.cache8_append(cache, k.cuda(), v.cuda(), ints([0] * B), ws=ws)
    for b in range(B):
        model.append(b, 0, k[b], v[b])
    want = {x: [model.values(x, b).float().bfloat16() for b in range(B)] for x in "kv"}
    for starts, n in (([0, 1, 499], 1), ([63, 64, 65], 70), ([0, 250, 127], 250)):
        got = logo.cache8_read(cache, ints(starts), n, ws=ws)
        for x, y in zip("kv", got):
            for b in range(B):
                assert same(y[b].cpu().contiguous(), want[x][b][:, starts[b]:starts[b] + n].contiguous())
    out = tuple(torch.full((1, Hkv, 300, d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    logo.cache8_read(cache, ints([10, 499, 100]), 300, ws=ws, cu_seqlens=ints([0, 129, 129, 260]), max_seqlen=131, out=out)
    for x, y in zip("kv", out):
        assert same(y[0, :, :129].cpu().contiguous(), want[x][0][:, 10:139].contiguous())
        assert same(y[0, :, 129:260].cpu().contiguous(), want[x][2][:, 100:231].contiguous())
        assert (y[0, :, 260:] == 3.0).all()
    k0, v0 = logo.cache8_read(cache, ints([0] * B), 0, ws=ws)
    assert k0.shape == (B, Hkv, 0, d)
    logo.check(ws)


def test_rows_that_do_not_fit_are_reported_and_leave_the_sequence_alone():
    gen = torch.Generator().manual_seed(2)
    B, Hkv, d, Lmax, block = 4, 2, 64, 100, 64
    dtype = torch.int8
    cache, model, ws = fresh(B, Hkv, Lmax, d, dtype, block), Model(B, Hkv, d, dtype, block), workspace()
    k, v = randn(gen, B, Hkv, 50, d), randn(gen, B, Hkv, 50, d)
    logo.cache8_append(cache, k.cuda(), v.cuda(), ints([0] * B), ws=ws)
    for b in range(B):
        model.append(b, 0, k[b], v[b])
    logo.check(ws)
    new = ints([0] * B)
    logo.cache8_append(cache, k.cuda(), v.cuda(), ints([50, 51, -1, 2 ** 31 - 1]), ws=ws, new_len=new)
    with pytest.raises(logo.LogoError) as e:
        logo.check(ws)
    assert e.value.status == 1
    assert new.tolist() == [100, 51, -1, 2 ** 31 - 1]
    model.append(0, 50, k[0], v[0])
    check(cache, model, [100, 50, 50, 50])
    # packed offsets out of order, beyond the rows, longer than stated
    for cu in ([0, 20, 10, 10, 10], [0, 20, 20, 20, 51], [0, 31, 31, 31, 31], [-1, 0, 0, 0, 0]):
        ws = workspace()
        logo.cache8_append(cache, k[:1].cuda().contiguous(), v[:1].cuda().contiguous(), ints([100, 50, 50, 50]), ws=ws,
                           cu_seqlens=ints(cu), max_seqlen=30)
        with pytest.raises(logo.LogoError):
            logo.check(ws)
    ws = workspace()
    out = tuple(torch.full((B, Hkv, 40, d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    logo.cache8_read(cache, ints([0, -3, 61, 2 ** 31 - 5]), 40, ws=ws, out=out)
    with pytest.raises(logo.LogoError):
        logo.check(ws)
    for y in out:
        assert (y[1:] == 3.0).all() and (y[0] != 3.0).any()


def test_a_sequence_of_the_batch_alone_and_a_captured_append():
    """A view of one sequence's cache is a cache; an append captured into a graph follows its start array."""
    gen = torch.Generator().manual_seed(4)
    B, Hkv, d, Lmax, block, dtype = 3, 2, 128, 300, 64, torch.float8_e4m3fn
    cache, model, ws = fresh(B, Hkv, Lmax, d, dtype, block), Model(B, Hkv, d, dtype, block), workspace()
    k, v = randn(gen, 1, Hkv, 70, d), randn(gen, 1, Hkv, 70, d)
    parts = (cache.k, cache.v, cache.k_scale, cache.v_scale, cache.k_tail, cache.v_tail)
    logo.cache8_append(logo.Cache8(*(t[1:2] for t in parts)), k.cuda(), v.cuda(), ints([0]), ws=ws)
    model.append(1, 0, k[0], v[0])
    check(cache, model, [0, 70, 0])
    x, y = (torch.ones(B, Hkv, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    at, nxt = ints([0, 70, 0]), ints([0, 0, 0])
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        logo.cache8_append(cache, x, y, at, ws=ws, new_len=nxt)
        at.copy_(nxt)
    lens = [0, 70, 0]
    for _ in range(130):
        a, c = randn(gen, B, Hkv, 1, d), randn(gen, B, Hkv, 1, d)
        x.copy_(a)
        y.copy_(c)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            model.append(b, lens[b], a[b], c[b])
            lens[b] += 1
    logo.check(ws)
    assert at.tolist() == lens
    check(cache, model, lens)
