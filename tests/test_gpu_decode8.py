"""The decode step over the 8-bit cache on the GPU against the definition in 64 bits, on the values that the cache
stands for; each element within the bound that the reference derives."""
import pytest
import torch

import token_level_dynamic_seq_b200 as logo
from tests import cache8_reference as ref
from tests.test_gpu_cache8 import fresh, ints, workspace

pytestmark = pytest.mark.gpu

TYPES = [torch.float8_e4m3fn, torch.int8]


def build(B, Hkv, Lmax, d, dtype, block, lens, seed, size=1.0):
    """A cache with lens[b] rows a sequence (everything else NaN), its model, and the generator."""
    gen = torch.Generator().manual_seed(seed)
    cache, model = fresh(B, Hkv, Lmax, d, dtype, block), ref.Model(B, Hkv, d, dtype, block)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    k = torch.randn(1, Hkv, cu[-1], d, generator=gen).mul(size).bfloat16()
    v = torch.randn(1, Hkv, cu[-1], d, generator=gen).bfloat16()
    fill(cache, model, k, v, cu, lens)
    return cache, model, gen


def fill(cache, model, k, v, cu, lens):
    if cu[-1]:
        ws = workspace()
        logo.cache8_append(cache, k.cuda(), v.cuda(), ints([0] * cache.B), ws=ws, cu_seqlens=ints(cu), max_seqlen=max(lens))
        logo.check(ws)
    for b in range(cache.B):
        model.append(b, 0, k[0, :, cu[b]:cu[b + 1]], v[0, :, cu[b]:cu[b + 1]])


def verify(cache, model, q, gate, tau, W, lens, out, selected, scale=0.0):
    assert selected.cpu().tolist() == (gate > tau).int().tolist()
    for b in range(cache.B):
        if lens[b] == 0:
            assert (out[b].float() == 0).all()
            continue
        want, bound = ref.decode(q[b], model.values("k", b), model.values("v", b), gate[b], tau, W, scale)
        err = (out[b].double().cpu() - want).abs()
        assert torch.isfinite(out[b].float()).all()
        worst = (err / bound).max().item()
        assert worst <= 1.0, f"sequence {b} (length {lens[b]}): {worst:.2f} of the bound"


def go(cache, model, gen, Hq, n, W, lens, tau=0.0, scale=0.0, gate=None, qsize=1.0):
    q = torch.randn(cache.B, Hq, n, cache.d, generator=gen).mul(qsize).bfloat16()
    gate = torch.randn(cache.B, n, generator=gen) if gate is None else gate
    ws = logo.decode8_workspace(cache, Hq, n)
    out, sel = logo.decode8(q.cuda(), cache, ints(lens), gate.cuda(), torch.tensor([tau], device="cuda"), W, ws=ws,
                            scale=scale)
    logo.check(ws)
    verify(cache, model, q, gate, tau, W, lens, out, sel, scale)
    return out


CASES = [
    # B, Hq, Hkv, d, n, W, block, lengths
    (1, 1, 1, 64, 1, 1, 64, [1]),
    (8, 8, 2, 128, 1, 100, 64, [1, 5, 63, 64, 65, 999, 1000, 0]),
    (6, 4, 4, 64, 1, 1, 128, [1000, 7, 512, 513, 3, 600]),
    (5, 16, 2, 128, 1, 5000, 64, [1000, 1, 100, 768, 900]),
    (4, 6, 2, 128, 1, 256, 128, [700, 256, 257, 2]),           # three heads a group
    (3, 10, 2, 64, 1, 64, 64, [640, 129, 64]),                 # five
    (7, 8, 1, 128, 4, 50, 64, [1000, 1, 2, 4, 5, 66, 511]),    # 32 rows, shorter than the drafts
    (4, 8, 2, 128, 2, 63, 64, [190, 64, 128, 127]),            # 8 rows
    (4, 8, 2, 64, 4, 130, 128, [777, 131, 3, 320]),            # 16 rows
    (3, 12, 4, 128, 5, 7, 64, [330, 200, 5]),                  # 15 rows
    (3, 3, 1, 64, 7, 1, 64, [129, 64, 6]),                     # 21 rows, window 1
    (2, 1, 1, 128, 32, 40, 64, [500, 33]),                     # 32 tokens, one head
    (70, 2, 2, 64, 1, 20, 64, [(i * 37) % 150 for i in range(70)]),  # more than two groups of 32 sequences
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", CASES)
def test_decode8_small_full(dtype, case):
    B, Hq, Hkv, d, n, W, block, lens = case
    cache, model, gen = build(B, Hkv, 1000, d, dtype, block, lens, seed=sum(lens) + n)
    go(cache, model, gen, Hq, n, W, lens)
    go(cache, model, gen, Hq, n, W, lens, tau=-100.0)      # every token global
    go(cache, model, gen, Hq, n, W, lens, tau=float("inf"))   # none


@pytest.mark.parametrize("seed", range(12))
def test_decode8_random_shapes(seed):
    r = torch.Generator().manual_seed(1000 + seed)
    pick = lambda *v: v[int(torch.randint(len(v), (1,), generator=r))]  # noqa: E731
    Hkv, G, d, block, dtype = pick(1, 2, 3, 8), pick(1, 2, 3, 4, 7, 8), pick(64, 128), pick(64, 128), pick(*TYPES)
    n = pick(1, 1, 2, 3, 4)
    Lmax = int(torch.randint(1, 3000, (1,), generator=r))
    B = int(torch.randint(1, 9, (1,), generator=r))
    lens = torch.randint(0, Lmax + 1, (B,), generator=r).tolist()
    W = int(torch.randint(1, 2000, (1,), generator=r))
    cache, model, gen = build(B, Hkv, Lmax, d, dtype, block, lens, seed)
    go(cache, model, gen, G * Hkv, n, W, lens)


@pytest.mark.parametrize("dtype", TYPES)
def test_long_caches(dtype):
    """32K positions, full, one short of full, and short ones beside them."""
    lens = [32768, 32767, 4096, 1, 20000]
    cache, model, gen = build(5, 1, 32768, 128, dtype, 64, lens, seed=1)
    gate = torch.tensor([[1.0], [-1.0], [0.5], [2.0], [0.1]])
    go(cache, model, gen, 4, 1, 4096, lens, gate=gate)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [1e-30, 1e30, 2e37])
def test_blocks_of_very_different_scales(dtype, size):
    """Values whose blocks differ by 60 orders of magnitude: the small ones count where the large ones are not seen.
    Keys and queries far from one with a scale that makes up for it."""
    B, Hkv, d, block, L = 2, 1, 64, 64, 320
    gen = torch.Generator().manual_seed(8)
    cache, model = fresh(B, Hkv, L, d, dtype, block), ref.Model(B, Hkv, d, dtype, block)
    k = torch.randn(1, Hkv, 2 * L, d, generator=gen) * 1e-12
    v = torch.randn(1, Hkv, 2 * L, d, generator=gen)
    v[:, :, :128] *= size
    v[:, :, L + 256:L + 300] *= size
    fill(cache, model, k.bfloat16(), v.bfloat16(), [0, L, 2 * L], [L, L])
    go(cache, model, gen, 2, 1, 100, [L, L], tau=10.0, scale=1e4 / 8, qsize=1e8)
    go(cache, model, gen, 2, 1, 100, [L, L], tau=-10.0, scale=1e4 / 8, qsize=1e8)


@pytest.mark.parametrize("n", [1, 2])
def test_more_sequences_than_a_cta_keeps_lengths_of(n):
    """1,300 sequences: the lengths of the last ones are read from memory again wherever they are needed."""
    lens = [(i * 53) % 97 for i in range(1300)]
    cache, model, gen = build(1300, 1, 97, 64, torch.int8, 64, lens, seed=4)
    go(cache, model, gen, 2, n, 40, lens)


def test_two_streams_with_a_workspace_each():
    """Two batches decoded at the same time on two streams give what each gives alone."""
    made = [build(2, 2, 3000, 128, t, 64, [3000, 1700], seed=30 + i) for i, t in enumerate(TYPES)]
    runs = []
    for cache, model, gen in made:
        q, gate = torch.randn(2, 8, 1, 128, generator=gen).bfloat16().cuda(), torch.randn(2, 1, generator=gen).cuda()
        runs.append((q, cache, ints([3000, 1700]), gate, torch.tensor([0.0], device="cuda"), 500,
                     logo.decode8_workspace(cache, 8)))
    alone = [logo.decode8(*r)[0] for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(20):
        outs = [logo.decode8(*r, stream=s)[0] for r, s in zip(runs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, outs):
            assert torch.equal(a, b)


def test_peaked_scores_and_long_tails_of_small_weights():
    """Scores up to several hundred, and a first key 20 above tens of thousands of others: their weights (2^-29 each)
    add up and are not lost."""
    cache, model, gen = build(2, 1, 2000, 64, torch.int8, 64, [2000, 1500], seed=3, size=12.0)
    go(cache, model, gen, 4, 1, 300, [2000, 1500], tau=-10.0, qsize=6.0)
    L, d = 30000, 64
    k = torch.zeros(1, 1, L, d)
    k[0, 0, 0, 0] = 160.0   # q.k / 8 = 20
    v = torch.ones(1, 1, L, d)
    v[0, 0, 0] = 0.0
    cache, model = fresh(1, 1, L, d, torch.int8, 64), ref.Model(1, 1, d, torch.int8, 64)
    fill(cache, model, k.bfloat16(), v.bfloat16(), [0, L], [L])
    q = torch.zeros(1, 1, 1, d)
    q[..., 0] = 1.0
    gate = torch.tensor([[0.0]])
    ws = logo.decode8_workspace(cache, 1)
    out, sel = logo.decode8(q.bfloat16().cuda(), cache, ints([L]), gate.cuda(), torch.tensor([-1.0], device="cuda"), 1, ws=ws)
    logo.check(ws)
    verify(cache, model, q.bfloat16(), gate, -1.0, 1, [L], out, sel)


@pytest.mark.parametrize("n", [1, 3])
def test_values_that_are_not_finite_stay_where_they_are_seen(n):
    """NaN keys and values before the window, and at a draft's position, reach only the tokens that see them."""
    B, Hkv, d, block, L, W = 1, 1, 64, 64, 300, 70
    gen = torch.Generator().manual_seed(6)
    k, v = torch.randn(1, Hkv, L, d, generator=gen).bfloat16(), torch.randn(1, Hkv, L, d, generator=gen).bfloat16()
    first = L - n - W + 1                    # token 0's first position
    k[0, 0, first - 1, 3] = float("nan")     # just before every window
    v[0, 0, first - 2] = float("nan")
    q = torch.randn(1, 2, n, d, generator=gen).bfloat16()
    tau, gate = torch.tensor([0.0], device="cuda"), torch.full((1, n), -1.0)

    def run(vv):
        cache, model = fresh(B, Hkv, L, d, torch.float8_e4m3fn, block), ref.Model(B, Hkv, d, torch.float8_e4m3fn, block)
        fill(cache, model, k, vv, [0, L], [L])
        ws = logo.decode8_workspace(cache, 2, n)
        out, _ = logo.decode8(q.cuda(), cache, ints([L]), gate.cuda(), tau, W, ws=ws)
        logo.check(ws)
        return out.float().cpu(), model

    out, model = run(v)
    clean = torch.nan_to_num(model.values("v", 0)[:, :], 0.0), torch.nan_to_num(model.values("k", 0), 0.0)
    want, bound = ref.decode(q[0], clean[1], clean[0], gate[0], 0.0, W)
    assert ((out[0].double() - want).abs() <= bound).all()
    if n > 1:   # the last draft's value is NaN: only the last token sees it; and token 0's first: only token 0
        w = v.clone()
        w[0, 0, L - 1, 5] = float("nan")
        w[0, 0, first, 9] = float("nan")
        out, model = run(w)
        bad = torch.isnan(out[0])
        assert bad[:, n - 1, 5].all() and bad[:, 0, 9].all() and int(bad.sum()) == 2 * 2
        vals = torch.nan_to_num(model.values("v", 0), 0.0)
        want, bound = ref.decode(q[0], clean[1], vals, gate[0], 0.0, W)
        assert ((out[0].double() - want).abs() <= bound)[~bad].all()


@pytest.mark.parametrize("dtype", TYPES)
def test_queries_keys_and_scales_that_are_not_finite(dtype):
    """A NaN query makes its own row NaN and no other; a NaN scale, every row that sees the block; all keys NaN, all."""
    cache, model, gen = build(2, 1, 700, 64, dtype, 64, [700, 130], seed=9)
    lens, tau = [700, 130], 0.0
    q, gate = torch.randn(2, 3, 2, 64, generator=gen).bfloat16(), torch.full((2, 2), 1.0)
    q[0, 1, 0, 5] = float("nan")
    q[1, 2, 1, 0] = float("inf")
    ws = logo.decode8_workspace(cache, 3, 2)
    go_ = lambda g=gate, W=100: logo.decode8(q.cuda(), cache, ints(lens), g.cuda(), torch.tensor([tau], device="cuda"),  # noqa: E731
                                             W, ws=ws)[0].float().cpu()
    out = go_()
    bad = torch.isnan(out).any(-1)
    want = torch.zeros(2, 3, 2, dtype=torch.bool)
    want[0, 1, 0] = want[1, 2, 1] = True
    assert torch.equal(bad, want)
    for b in range(2):
        ref_out, bound = ref.decode(q[b], model.values("k", b), model.values("v", b), gate[b], tau, 100)
        ok = ~want[b]
        assert ((out[b].double() - ref_out).abs() <= bound)[ok].all()
    cache.k_scale[0, 0, 3] = float("nan")        # positions 192 .. 255 of sequence 0: behind the window of 100
    assert torch.isnan(go_()[0]).all()           # global rows see them
    quiet = torch.full((2, 2), -1.0)
    assert torch.equal(torch.isnan(go_(quiet)).any(-1), want)
    cache.k_scale[0] = float("nan")
    assert torch.isnan(go_(quiet)[0]).all() and torch.equal(torch.isnan(go_(quiet)[1]).any(-1), want[1])
    logo.check(ws)


def test_gates_thresholds_and_row_behind_short_sequences():
    cache, model, gen = build(4, 2, 300, 64, torch.int8, 64, [300, 300, 300, 1], seed=2)
    nan, inf = float("nan"), float("inf")
    gate = torch.tensor([[nan, 1.0], [inf, -inf], [0.0, -0.0], [0.7, 0.7]])
    lens = [300, 300, 300, 1]
    q = torch.randn(4, 4, 2, 64, generator=gen).bfloat16()
    ws = logo.decode8_workspace(cache, 4, 2)
    for tau in (0.0, -1.0, nan):
        out, sel = logo.decode8(q.cuda(), cache, ints(lens), gate.cuda(), torch.tensor([tau], device="cuda"), 33, ws=ws)
        logo.check(ws)
        g = torch.where(gate == inf, torch.tensor(1e4), gate)     # sigmoid 1
        verify(cache, model, q, torch.where(gate.isnan(), -inf, g) if tau == tau else torch.full_like(g, -inf),
               tau if tau == tau else 0.0, 33, lens, out, sel)
        assert (out[3, :, 0].float() == 0).all()                  # the first of two tokens of a length of one


def test_lengths_out_of_range_are_reported():
    cache, model, gen = build(4, 2, 64, 64, torch.float8_e4m3fn, 64, [64, 40, 64, 30], seed=1)
    q, gate = torch.randn(4, 4, 64, generator=gen).bfloat16(), torch.full((4, 1), 1.0)
    ws = logo.decode8_workspace(cache, 4)
    out, sel = logo.decode8(q.cuda(), cache, ints([64, 65, -1, 30]), gate.cuda(), torch.tensor([0.0], device="cuda"), 16, ws=ws)
    with pytest.raises(logo.LogoError) as e:
        logo.check(ws)
    assert e.value.status == 1
    assert (out[1:3].float() == 0).all()
    assert out.shape == q.shape
    for b in (0, 3):
        want, bound = ref.decode(q[b][:, None], model.values("k", b), model.values("v", b), gate[b], 0.0, 16)
        assert ((out[b].double().cpu() - want[:, 0]).abs() <= bound[:, 0]).all()


def test_the_same_bits_again_on_a_stream_and_in_a_graph():
    lens = [900, 64, 333]
    cache, model, gen = build(3, 2, 1000, 128, torch.float8_e4m3fn, 128, lens, seed=12)
    q, gate = torch.randn(3, 8, 1, 128, generator=gen).bfloat16().cuda(), torch.randn(3, 1, generator=gen).cuda()
    tau, cl = torch.tensor([0.0], device="cuda"), ints(lens)
    ws = logo.decode8_workspace(cache, 8)
    first, _ = logo.decode8(q, cache, cl, gate, tau, 100, ws=ws)
    again, _ = logo.decode8(q, cache, cl, gate, tau, 100)
    torch.cuda.synchronize()
    assert torch.equal(first, again)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side, _ = logo.decode8(q, cache, cl, gate, tau, 100, stream=side)
    side.synchronize()
    assert torch.equal(first, on_side)
    out, graph = torch.zeros_like(q), torch.cuda.CUDAGraph()
    sel = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    with torch.cuda.graph(graph):
        logo.decode8(q, cache, cl, gate, tau, 100, ws=ws, out=out, selected=sel)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out)
    cl.copy_(ints([500, 64, 1]))       # lengths are read on the device: the graph follows them
    graph.replay()
    fresh_out, _ = logo.decode8(q, cache, cl, gate, tau, 100, ws=logo.decode8_workspace(cache, 8))
    torch.cuda.synchronize()
    assert torch.equal(fresh_out, out)
    logo.check(ws)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_serving_loop(dtype):
    """Prompts appended packed, then steps of one token and of drafts that are partly rejected, the cache's state
    followed by the model; and the bf16 decode over the rows read back agrees."""
    B, Hq, Hkv, d, Lmax, W, block = 3, 8, 2, 128, 400, 90, 64
    lens = [130, 64, 1]
    cache, model, gen = build(B, Hkv, Lmax, d, dtype, block, lens, seed=20)
    ws = logo.decode8_workspace(cache, Hq, 4)
    tau = 0.2
    for step in range(40):
        n = 1 if step % 4 else 4
        k, v = (torch.randn(B, Hkv, n, d, generator=gen).bfloat16() for _ in range(2))
        held = ints([0] * B)
        logo.cache8_append(cache, k.cuda(), v.cuda(), ints(lens), ws=ws, new_len=held)
        for b in range(B):
            model.append(b, lens[b], k[b], v[b])
        q, gate = torch.randn(B, Hq, n, d, generator=gen).bfloat16(), torch.randn(B, n, generator=gen)
        out, sel = logo.decode8(q.cuda(), cache, held, gate.cuda(), torch.tensor([tau], device="cuda"), W, ws=ws)
        logo.check(ws)
        now = [L + n for L in lens]
        assert held.tolist() == now
        if step % 5 == 0 or n > 1:
            verify(cache, model, q, gate, tau, W, now, out, sel)
        if n == 1 and step % 10 == 1:
            kc, vc = logo.cache8_read(cache, ints([0] * B), max(now), ws=ws)
            kc, vc = (torch.nan_to_num(x, 0.0) for x in (kc, vc))   # rows behind the shorter sequences: never written
            plain, _ = logo.decode(q[:, :, 0].contiguous().cuda(), kc, vc, held, gate[:, 0].contiguous().cuda(),
                                   torch.tensor([tau], device="cuda"), W)
            diff = (plain.double() - out[:, :, 0].double()).norm() / plain.double().norm()
            # both outputs and the bf16 decode's P (2^-8) and rows read back (2^-8) are rounded: 4 roundings of 2^-8 at most
            assert diff.item() <= 4 * 2.0 ** -8
        lens = [L - (step + b) % 3 if n > 1 else L for b, L in enumerate(now)]   # up to two drafts rejected
        for b in range(B):
            for x in "kv":
                model.rows[x][b] = model.rows[x][b][:, :lens[b]]


@pytest.mark.parametrize("dtype", TYPES)
def test_scores_far_below_zero_and_rising(dtype):
    """Scores around -1e31 are a softmax like any other; and scores that rise from stage to stage by a little more or
    less than what a stage may exceed the ones before it."""
    B, d, L = 1, 64, 640
    gen = torch.Generator().manual_seed(17)
    cache, model = fresh(B, 1, L, d, dtype, 64), ref.Model(B, 1, d, dtype, 64)
    k = torch.zeros(1, 1, L, d)
    k[..., 0] = -1.0
    v = torch.randn(1, 1, L, d, generator=gen)
    fill(cache, model, k.bfloat16(), v.bfloat16(), [0, L], [L])
    q = torch.zeros(1, 2, 1, d)
    q[0, 0, 0, 0], q[0, 1, 0, 0] = 8e31, -8e31
    gate = torch.tensor([[1.0]])
    ws = logo.decode8_workspace(cache, 2)
    for tau in (0.0, 2.0):
        out, sel = logo.decode8(q.bfloat16().cuda(), cache, ints([L]), gate.cuda(), torch.tensor([tau], device="cuda"), 100,
                                ws=ws)
        logo.check(ws)
        # every score is the same, so the weights are: the mean of the values
        vals = model.values("v", 0)
        want = vals[:, -100:].mean(1) + (torch.sigmoid(torch.tensor(1.0)).item() * vals.mean(1) if tau < 1 else 0)
        assert (out[0, :, 0].double().cpu() - want).abs().max().item() <= 2.0 ** -8 * want.abs().max().item() + 2.0 ** -9
    for step in (0.5, 1.2, 1.4, 3.0):
        cache, model = fresh(B, 1, L, d, dtype, 64), ref.Model(B, 1, d, dtype, 64)
        k = torch.randn(1, 1, L, d, generator=gen) * 0.05
        k[0, 0, :, 0] += torch.arange(L) // 32 * step       # 8 q.k / 8 rises by `step` (log2: 1.44 step) every 32 positions
        fill(cache, model, k.bfloat16(), v.bfloat16(), [0, L], [L])
        q = torch.zeros(1, 2, 1, d)
        q[..., 0] = 8.0
        q[0, 1] *= -1
        go_gate = torch.tensor([[1.0]])
        out, sel = logo.decode8(q.bfloat16().cuda(), cache, ints([L]), go_gate.cuda(), torch.tensor([0.0], device="cuda"), 300,
                                ws=ws)
        logo.check(ws)
        verify(cache, model, q.bfloat16(), go_gate, 0.0, 300, [L], out, sel)


@pytest.mark.parametrize("dtype", TYPES)
def test_equal_scores_of_any_size(dtype):
    """Equal scores get equal weights where fp32 has no digits left behind the point: at 2^20 to 2^32 the reference
    that is taken off the scores is itself rounded by up to 2^8."""
    B, d, L, W = 1, 64, 640, 100
    gen = torch.Generator().manual_seed(23)
    cache, model = fresh(B, 1, L, d, dtype, 64), ref.Model(B, 1, d, dtype, 64)
    k = torch.zeros(1, 1, L, d)
    k[..., 0] = -1.0
    v = torch.randn(1, 1, L, d, generator=gen)
    fill(cache, model, k.bfloat16(), v.bfloat16(), [0, L], [L])
    ws = logo.decode8_workspace(cache, 2)
    vals = model.values("v", 0)
    want = vals[:, -W:].mean(1)
    # out is off by half a step of bf16 (2^-8 of it), and each P by 2^-11 of itself against the sum of unrounded P
    tol = 2.0 ** -8 * want.abs() + 1.01 * 2.0 ** -11 * vals[:, -W:].abs().mean(1) + 1e-5
    for e in range(20, 33):
        for x in (1.0, 1.375, 1.9375):
            q = torch.zeros(1, 2, 1, d)
            q[0, 0, 0, 0], q[0, 1, 0, 0] = 8 * x * 2.0 ** e, -8 * x * 2.0 ** e
            out, sel = logo.decode8(q.bfloat16().cuda(), cache, ints([L]), torch.ones(1, 1).cuda(),
                                    torch.tensor([2.0], device="cuda"), W, ws=ws)
            logo.check(ws)
            assert ((out[0, :, 0].double().cpu() - want).abs() <= tol).all(), (e, x)


@pytest.mark.parametrize("B", [3, 70])
def test_a_workspace_with_an_earlier_timeout(B):
    """The status word of an earlier call whose wait ran out is reported again, whatever else the workspace holds; set
    up anew, the workspace serves."""
    lens = [(i * 29) % 200 for i in range(B)]
    cache, model, gen = build(B, 2, 256, 128, TYPES[0], 64, lens, seed=29)
    q, gate = torch.randn(B, 4, 1, 128, generator=gen).bfloat16(), torch.randn(B, 1, generator=gen)
    tau = torch.zeros(1, device="cuda")
    ws = logo.decode8_workspace(cache, 4)
    ws.fill_(0x7f)
    ws[:256] = 0
    ws[0] = 1
    logo.decode8(q.cuda(), cache, ints(lens), gate.cuda(), tau, 50, ws=ws)
    with pytest.raises(logo.LogoError) as e:
        logo.check(ws)
    assert e.value.status == 5
    ws[:256] = 0
    out, sel = logo.decode8(q.cuda(), cache, ints(lens), gate.cuda(), tau, 50, ws=ws)
    logo.check(ws)
    verify(cache, model, q, gate, 0.0, 50, lens, out, sel)


@pytest.mark.parametrize("dtype", TYPES)
def test_the_largest_queries_and_values(dtype):
    """Queries near bf16's largest against the smallest keys a scale stands for: one key is 1e6 ahead of the others,
    so the output is its value, here up to 3e38.  Also a window beyond 32 bits: the whole cache."""
    B, d, L, at = 1, 64, 200, 77
    gen = torch.Generator().manual_seed(31)
    cache, model = fresh(B, 1, L, d, dtype, 64), ref.Model(B, 1, d, dtype, 64)
    k = torch.full((1, 1, L, d), -2.0 ** -100)
    k[0, 0, at] = 2.0 ** -100
    v = (torch.rand(1, 1, L, d, generator=gen) * 2 - 1).mul(3e38)
    fill(cache, model, k.bfloat16(), v.bfloat16(), [0, L], [L])
    q = torch.zeros(1, 2, 1, d)
    q[0, :, 0, 5] = 3e38
    ws = logo.decode8_workspace(cache, 2)
    for W in (L, 2 ** 40):
        out, sel = logo.decode8(q.bfloat16().cuda(), cache, ints([L]), torch.ones(1, 1).cuda(),
                                torch.tensor([2.0], device="cuda"), W, ws=ws)
        logo.check(ws)
        want = model.values("v", 0)[:, at]
        # the weight is one: half a step of bf16, and a few of fp32
        assert ((out[0, :, 0].double().cpu() - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want.abs()).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_offsets_beyond_32_bits(dtype):
    """Rows at positions around 2^26 of two heads with 64 codes each: 2^32 bytes into either slab and 2^33 in all."""
    s, L, W, d, Hkv = 2 ** 26 - 64, 300, 200, 64, 2
    gen = torch.Generator().manual_seed(37)
    cache, model = logo.cache8(1, Hkv, s + 400, d, "cuda", dtype=dtype, block=64), ref.Model(1, Hkv, d, dtype, 64)
    k, v = (torch.randn(1, Hkv, L, d, generator=gen).bfloat16() for _ in "kv")
    ws = logo.decode8_workspace(cache, 4, 2)
    held = torch.zeros(1, dtype=torch.int32, device="cuda")
    logo.cache8_append(cache, k.cuda(), v.cuda(), ints([s]), ws=ws, new_len=held)
    assert held.item() == s + L
    model.append(0, 0, k[0], v[0])
    q, gate = torch.randn(1, 4, 2, d, generator=gen).bfloat16(), torch.full((1, 2), -1.0)
    out, sel = logo.decode8(q.cuda(), cache, held, gate.cuda(), torch.zeros(1, device="cuda"), W, ws=ws)
    kb, vb = logo.cache8_read(cache, ints([s]), L, ws=ws)
    logo.check(ws)
    verify(cache, model, q, gate, 0.0, W, [L], out, sel)
    for x, got in (("k", kb), ("v", vb)):
        assert torch.equal(got[0].cpu(), model.values(x, 0).float().bfloat16())
