"""Operators over a key/value cache held in 8 bits, as they are measured.

Three operators around one cache (codes in e4m3 or int8, one fp32 scale for every block of tokens and
key/value head, K and V apart):

  append  quantises new tokens into the cache as it is written (one token a sequence, or a whole prompt,
          fixed or packed lengths) and then reads the blocks it touched back;
  read    reads a range of every sequence back as bf16;
  decode  one step of local-global attention over the cache: windowed attention for every new token, and
          exact attention over the whole prefix for tokens whose gate passes the threshold.

``own`` false: the plain forms, elementary torch operations in 32 bits (64 next to a rounding border).
``own`` true: the calls a user makes of the library.
"""
import math
import random

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
FLOOR = 2.0 ** -100  # a block's largest magnitude counts as at least this


# ------------------------------------------------------------------------------------------- cases

def listed():
    def decode(name, **kw):
        base = {"op": "decode", "B": 1, "Hq": 32, "Hkv": 8, "d": 128, "n": 1, "W": 4096, "type": "e4m3", "block": 64}
        return {"name": name, **base, **kw}

    def cache(name, op, **kw):
        base = {"op": op, "B": 1, "Hkv": 8, "d": 128, "type": "e4m3", "block": 64, "packed": False}
        return {"name": name, **base, **kw}

    return [
        # one short chat next to another, one of the two tokens global: latency is what counts
        decode("decode_c4k", B=2, Hq=8, W=512, Lmax=4096, lo=4000, hi=4096, sel=1),
        # a single user at 32K tokens of context, the token global
        decode("decode_c32k_one", Lmax=32768, lo=32768, hi=32768, sel=1),
        # the serving batch: 64 sequences with full 32K caches, a fifth of the tokens global
        decode("decode_c32k", B=64, Lmax=32768, lo=32768, hi=32768, sel=13),
        # a ragged batch in int8 with large scale blocks
        decode("decode_ragged_int8", B=32, Lmax=16384, lo=1, hi=16384, sel=8, type="int8", block=128),
        # verification of four drafted tokens a sequence
        decode("decode_draft", B=16, n=4, Lmax=32768, lo=8192, hi=32768, sel=4),
        # narrow heads, eight query heads a key/value head, three drafted tokens, odd lengths
        decode("decode_d64_int8", B=24, Hq=16, Hkv=2, d=64, n=3, W=512, Lmax=4099, lo=100, hi=4099, sel=5, type="int8"),
        # two long documents, one of the tokens global
        decode("decode_c128k", B=2, Lmax=131072, lo=120000, hi=131072, sel=1),
        # the cache write of a decode step of 64 sequences
        cache("append_step", "append", B=64, Lmax=4096, start_lo=100, start_hi=4000, lo=1, hi=1),
        # the cache write of a whole prompt
        cache("append_prompt", "append", Lmax=32768, start_lo=0, start_hi=0, lo=32768, hi=32768),
        # the packed prompts of eight sequences, int8
        cache("append_packed_int8", "append", B=8, Lmax=16384, start_lo=0, start_hi=0, lo=1024, hi=16384, packed=True,
              type="int8", block=128),
        # a short prefix read back for reuse
        cache("read_c4k_int8", "read", B=2, Lmax=4096, start_lo=0, start_hi=0, lo=4096, hi=4096, type="int8"),
        # ragged prefixes of eight sequences read back packed
        cache("read_packed", "read", B=8, Lmax=16384, start_lo=0, start_hi=0, lo=1024, hi=16384, packed=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["decode", "decode", "decode", "append", "append", "read"])
    t, block, d = rng.choice(["e4m3", "int8"]), rng.choice([64, 128]), rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if kind == "decode":
        G, n = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
        n = min(n, 32 // G)
        Lmax = log(64, 65536)
        B = min(log(1, 64), max(1, 64 * 8 * 32768 * 128 // (2 * Hkv * Lmax * d)))
        return {"op": "decode", "B": B, "Hq": G * Hkv, "Hkv": Hkv, "d": d, "n": n, "W": log(1, 8192), "type": t,
                "block": block, "Lmax": Lmax, "lo": rng.randint(1, Lmax), "hi": Lmax, "sel": rng.randint(0, B)}
    long = rng.random() < 0.6 or kind == "read"
    top = log(16, 16384) if long else rng.randint(1, 9)
    low = top if rng.random() < 0.5 else max(1, top // rng.randint(2, 8))
    B = min(log(1, 64), max(1, (1 << 18) // top))
    start = 0 if kind == "append" and long else log(1, 2000)
    return {"op": kind, "B": B, "Hkv": Hkv, "d": d, "type": t, "block": block, "packed": low != top,
            "Lmax": start + top + rng.randint(0, 300), "start_lo": start // 3, "start_hi": start, "lo": low, "hi": top}


def spread(case, lo, hi, salt):
    """The lengths of a case: whole numbers in [lo, hi], both ends among them where there is room."""
    r = random.Random("%s %s %s %s %s" % (case["B"], case["Lmax"], lo, hi, salt))
    got = [r.randint(lo, hi) for _ in range(case["B"])]
    if case["B"] > 1:
        got[0], got[-1] = lo, hi
    return got


def lengths(case):
    return spread(case, case["lo"], case["hi"], "len")


def starts(case):
    return spread(case, case["start_lo"], case["start_hi"], "start")


def chosen(case):
    """Whether each sequence's tokens take the global branch: `sel` of the B, spread evenly."""
    B, s = case["B"], case["sel"]
    return [(b + 1) * s // B > b * s // B for b in range(B)]


def work(case):
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    if case["op"] == "decode":
        n, Hq, W = case["n"], case["Hq"], case["W"]
        seen = [L if c else min(L, W + n - 1) for L, c in zip(lengths(case), chosen(case))]
        scales = sum(-(-s // case["block"]) for s in seen) * Hkv * 2 * 4
        return {"bytes": sum(seen) * Hkv * d * 2 + scales + B * Hq * n * d * 4 + B * n * 8,
                "flops": 4.0 * d * Hq * n * sum(seen)}
    rows = sum(lengths(case))
    if case["op"] == "read":
        return {"bytes": rows * Hkv * d * 2 * 3, "flops": 0}
    back = sum(s % case["block"] + L for s, L in zip(starts(case), lengths(case)))
    kept = sum(min(L, 2 * case["block"]) for L in lengths(case))
    return {"bytes": Hkv * d * 2 * (rows * 2 + rows + kept * 2 + back * 3), "flops": 0}


# ------------------------------------------------------------------------------------------- inputs

def whole(v, dev, t=torch.int32):
    return torch.tensor(v, dtype=t, device=dev)


def offsets(v, dev):
    return whole([sum(v[:i]) for i in range(len(v) + 1)], dev)


def tokens(gen, shape, keys, dev):
    """Rows as a model writes them: unit variance; keys with a few channels several times as strong as the rest."""
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)
    if keys:
        c = torch.exp(0.6 * torch.randn(shape[-1], generator=gen, device=dev))
        x *= c / c.square().mean().sqrt()
    return x.bfloat16()


def filled(x, valid, block, kind):
    """Codes and scales of a cache [B, H, L, d] whose rows where `valid` [B, L] is true were written."""
    B, H, L, d = x.shape
    nblk = -(-L // block)
    mag = torch.where(valid[:, None, :, None], x.abs(), 0).amax(-1).float()
    mag = torch.nn.functional.pad(mag, (0, nblk * block - L)).view(B, H, nblk, block).amax(-1)
    scale = mag.clamp_min(FLOOR) / QMAX[kind]
    per_row = mag.clamp_min(FLOOR).repeat_interleave(block, 2)[:, :, :L, None]
    codes = torch.empty(x.shape, dtype=DTYPE[kind], device=x.device)
    for b in range(B):
        y = (x[b].double() * QMAX[kind] / per_row[b]).clamp(-QMAX[kind], QMAX[kind])
        codes[b] = (y.round() if kind == "int8" else y.float()).to(DTYPE[kind])
    touched = torch.nn.functional.pad(valid, (0, nblk * block - L)).view(B, 1, nblk, block).any(-1)
    return codes, torch.where(touched, scale, 0).contiguous()


def tails(x, lens, block):
    """The last two blocks' rows in bf16, [B, H, 2, block, d], as writing `lens` [B] rows leaves them."""
    B, H, L, d = x.shape
    pos = torch.arange(2 * block, device=x.device)
    last = (lens - 1).clamp_min(0) // block
    slot, row = pos // block, pos % block
    blk = torch.where(last[:, None] % 2 == slot, last[:, None], last[:, None] - 1)
    at = blk * block + row
    ok = (at >= 0) & (at < lens[:, None])
    rows = x[torch.arange(B, device=x.device)[:, None], :, at.clamp(0, L - 1)]          # [B, 2 block, H, d]
    rows = torch.where(ok[:, :, None, None], rows, torch.zeros_like(rows))
    return rows.transpose(1, 2).reshape(B, H, 2, block, d).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    B, Hkv, d, Lmax, block, kind = (case[k] for k in ("B", "Hkv", "d", "Lmax", "block", "type"))
    held = lengths(case) if case["op"] == "decode" else starts(case)
    if case["op"] == "read":
        held = [a + b for a, b in zip(held, lengths(case))]
    s = {"case": case, "block": block, "kind": kind, "held": whole(held, dev)}
    valid = torch.arange(Lmax, device=dev) < s["held"][:, None]
    for name in ("k", "v"):
        x = tokens(gen, (B, Hkv, Lmax, d), name == "k", dev)
        s[name], s[name + "_scale"] = filled(x, valid, block, kind)
        s[name + "_tail"] = tails(x, s["held"].long(), block)
        del x
    if case["op"] == "decode":
        n, Hq = case["n"], case["Hq"]
        s["q"] = tokens(gen, (B, Hq, n, d), False, dev)
        far = torch.rand(B, n, generator=gen, device=dev) * 2 + 0.05   # distance of each gate logit from the threshold
        s["tau"] = torch.full((1,), 0.8416, device=dev)
        s["gate"] = torch.where(whole(chosen(case), dev, torch.bool)[:, None], s["tau"] + far, s["tau"] - far)
    else:
        n = lengths(case)
        s["start"] = whole(starts(case), dev)
        s["rows"], s["longest"] = sum(n), max(n)
        s["cu"] = offsets(n, dev) if case["packed"] else None
        if case["op"] == "append":
            shape = (1, Hkv, sum(n), d) if case["packed"] else (B, Hkv, n[0], d)
            s["new_k"], s["new_v"] = tokens(gen, shape, True, dev), tokens(gen, shape, False, dev)
            # what the blocks that the append touches hold afterwards: from their first row to the new end
            back = [a % block + b for a, b in zip(starts(case), n)]
            s["back_start"] = whole([a - a % block for a in starts(case)], dev)
            s["back_cu"], s["back_rows"], s["back_longest"] = offsets(back, dev), sum(back), max(back)
            s["kept_rows"] = sum(a + b - max(a, ((a + b - 1) // block - 1) * block) for a, b in zip(starts(case), n))
            s["new_cu"] = offsets(n, dev)
    if own:  # the handles that a serving loop keeps: the cache object and the workspace
        import token_level_dynamic_seq_b200 as logo
        s["cache"] = logo.Cache8(s["k"], s["v"], s["k_scale"], s["v_scale"], s["k_tail"], s["v_tail"])
        s["ws"] = logo.decode8_workspace(s["cache"], case.get("Hq", Hkv), case.get("n", 1) if case["op"] == "decode" else 1)
    return s


# ------------------------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        import token_level_dynamic_seq_b200 as logo
        c, ws = s["cache"], s["ws"]
        if op == "decode":
            return logo.decode8(s["q"], c, s["held"], s["gate"], s["tau"], s["case"]["W"], ws=ws)
        if op == "read":
            return logo.cache8_read(c, s["start"], s["rows"] if s["cu"] is not None else s["longest"], ws=ws,
                                    cu_seqlens=s["cu"], max_seqlen=s["longest"])
        logo.cache8_append(c, s["new_k"], s["new_v"], s["start"], ws=ws, cu_seqlens=s["cu"], max_seqlen=s["longest"])
        k, v = logo.cache8_read(c, s["back_start"], s["back_rows"], ws=ws, cu_seqlens=s["back_cu"],
                                max_seqlen=s["back_longest"])
        return k, v, c.k_scale, c.v_scale, c.k_tail, c.v_tail
    if op == "decode":
        return plain_decode(s)
    if op == "read":
        k, v = (plain_read(s, x, s["start"], s["cu"], s["rows"]) for x in ("k", "v"))
        if s["cu"] is None:
            k, v = (x.view(x.shape[1], s["case"]["B"], -1, x.shape[3]).transpose(0, 1).contiguous() for x in (k, v))
        return k, v
    plain_append(s, "k")
    plain_append(s, "v")
    k, v = (plain_read(s, x, s["back_start"], s["back_cu"], s["back_rows"]) for x in ("k", "v"))
    return k, v, s["k_scale"], s["v_scale"], s["k_tail"], s["v_tail"]


def values(s, name):
    """The whole cache's values in fp32."""
    L = s[name].shape[2]
    return s[name].float() * s[name + "_scale"].repeat_interleave(s["block"], 2)[:, :, :L, None]


def softmax_rows(x, allowed):
    """Softmax over the last axis of the places where `allowed`; zero for a row without any."""
    x = torch.where(allowed, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0, m))
    t = p.sum(-1, keepdim=True)
    return p / torch.where(t == 0, 1, t)


def plain_decode(s):
    case = s["case"]
    q = s["q"].float()
    B, Hq, n, d = q.shape
    Hkv, L = s["k"].shape[1], s["k"].shape[2]
    G = Hq // Hkv
    x = (q.view(B, Hkv, G * n, d) @ values(s, "k").transpose(2, 3) / math.sqrt(d)).view(B, Hkv, G, n, L)
    pos = torch.arange(L, device=q.device)
    at = (s["held"].long()[:, None] - n + torch.arange(n, device=q.device))[:, None, None, :, None]
    seen = pos <= at
    near = seen & (pos > at - case["W"])
    sel = (s["gate"] > s["tau"])
    share = torch.where(sel, torch.sigmoid(s["gate"]), 0)[:, None, None, :, None]
    p = softmax_rows(x, near) + share * softmax_rows(x, seen)
    out = (p.view(B, Hkv, G * n, L) @ values(s, "v")).view(B, Hq, n, d)
    return out.bfloat16(), sel.int()


def rows_of(start, cu, total, B, device):
    """Sequence and position of each row of a packed range."""
    cu = cu.long()
    seq = torch.repeat_interleave(torch.arange(B, device=device), cu[1:] - cu[:-1], output_size=total)
    return seq, start.long()[seq] + torch.arange(total, device=device) - cu[seq]


def plain_read(s, name, start, cu, total):
    B, block = s[name].shape[0], s["block"]
    if cu is None:
        total = B * s["longest"]
        cu = torch.arange(B + 1, device=start.device) * s["longest"]
    seq, pos = rows_of(start, cu, total, B, start.device)
    x = s[name][seq, :, pos].float() * s[name + "_scale"][seq, :, pos // block][:, :, None]
    return x.bfloat16().transpose(0, 1)[None].contiguous()


def plain_append(s, name):
    case, block, kind = s["case"], s["block"], s["kind"]
    B, H, _, d = s[name].shape
    nblk = s[name + "_scale"].shape[2]
    new = s["new_" + name].transpose(1, 2).reshape(-1, H, d)                                # [rows, H, d]
    start, cu = s["start"].long(), s["new_cu"].long()
    seq, pos = rows_of(s["back_start"], s["back_cu"], s["back_rows"], B, start.device)
    old = pos < start[seq]
    tail = s[name + "_tail"][seq, :, pos // block % 2, pos % block]
    x = torch.where(old[:, None, None], tail, new[(cu[seq] + pos - start[seq]).clamp_min(0)]).double()
    mag = torch.where(torch.isfinite(x), x.abs(), 0).amax(-1)
    key = (seq * nblk + pos // block)[:, None].expand(-1, H)
    top = torch.full((B * nblk, H), FLOOR, dtype=torch.float64, device=x.device).scatter_reduce(0, key, mag, "amax")
    y = (x * QMAX[kind] / top.gather(0, key)[:, :, None]).clamp(-QMAX[kind], QMAX[kind])
    s[name][seq, :, pos] = (y.nan_to_num(0).round() if kind == "int8" else y.float()).to(DTYPE[kind])
    s[name + "_scale"][seq, :, pos // block] = top.gather(0, key).float() / QMAX[kind]
    # the last two blocks' new rows in bf16
    end = start + cu[1:] - cu[:-1]
    low = torch.maximum(start, ((end - 1) // block - 1) * block)
    seq, pos = rows_of(low, torch.cat([cu[:1], (end - low).cumsum(0)]), s["kept_rows"], B, start.device)
    s[name + "_tail"][seq, :, pos // block % 2, pos % block] = new[cu[seq] + pos - start[seq]]


# ------------------------------------------------------------------------------------------- in 64 bits

def rounded(y, kind):
    """y rounded to the nearest value of the type, ties to even, from the formats' definition."""
    if kind == "int8":
        return torch.round(y)
    _, e = torch.frexp(y.abs())                       # |y| = m 2^e with m in [1/2, 1)
    step = torch.ldexp(torch.ones_like(y), (e - 1).clamp_min(-6) - 3)   # three bits behind the point, least exponent -6
    return torch.round(y / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    B, block, kind = case["B"], case["block"], case["type"]
    top = QMAX[kind]
    if case["op"] == "decode":
        n, W, Hq, Hkv, d = (case[k] for k in ("n", "W", "Hq", "Hkv", "d"))
        out = torch.zeros(B, Hq, n, d, dtype=torch.float64, device="cuda")
        for b, (L, c) in enumerate(zip(lengths(case), chosen(case))):
            lo = 0 if c else max(0, L - n + 1 - W)
            ks, vs = (s[x][b, :, lo:L].double() * s[x + "_scale"][b].double()[:, torch.arange(lo, L, device="cuda") // block, None]
                      for x in ("k", "v"))
            for i in range(n):
                t = L - n + i
                if t < 0:
                    continue
                for first, share in ((max(0, t - W + 1), None), (0, s["gate"][b, i].double())):
                    if share is not None and not c:
                        continue
                    x = torch.einsum("hgd,hld->hgl", s["q"][b, :, i].double().view(Hkv, -1, d), ks[:, first - lo:t + 1 - lo])
                    o = torch.einsum("hgl,hld->hgd", torch.softmax(x * d ** -0.5, -1), vs[:, first - lo:t + 1 - lo])
                    out[b, :, i] += o.reshape(Hq, d) * (1 if share is None else 1 / (1 + torch.exp(-share)))
        return out, torch.tensor([[int(c)] * n for c in chosen(case)], dtype=torch.int32)
    got = {"k": [], "v": []}
    if case["op"] == "read":
        for x in ("k", "v"):
            for b, (a, n) in enumerate(zip(starts(case), lengths(case))):
                at = torch.arange(a, a + n, device="cuda")
                got[x].append(s[x][b, :, at].double() * s[x + "_scale"][b][:, at // block, None].double())
        k, v = ((torch.cat(got[x], 1)[None] if case["packed"] else torch.stack(got[x])) for x in ("k", "v"))
        return k, v
    scales, kept = {}, {}
    for x in ("k", "v"):
        scales[x], kept[x] = s[x + "_scale"].double().clone(), s[x + "_tail"].double().clone()
        at = 0
        for b, (a, n) in enumerate(zip(starts(case), lengths(case))):
            new = s["new_" + x][0, :, at:at + n] if case["packed"] else s["new_" + x][b]
            at += n
            f = a // block
            rows = torch.cat([s[x + "_tail"][b, :, f % 2, :a % block], new], 1).double()     # from the block's start
            parts = []
            for j in range(0, rows.shape[1], block):
                part = rows[:, j:j + block]
                big = part.abs().amax((1, 2)).clamp_min(FLOOR)
                scales[x][b, :, f + j // block] = big / top
                parts.append(rounded(part * top / big[:, None, None], kind) * (big / top)[:, None, None])
            got[x].append(torch.cat(parts, 1))
            for p in range(max(a, ((a + n - 1) // block - 1) * block), a + n):
                kept[x][b, :, p // block % 2, p % block] = new[:, p - a].double()
    k, v = (torch.cat(got[x], 1)[None] for x in ("k", "v"))
    return k, v, scales["k"], scales["v"], kept["k"], kept["v"]
