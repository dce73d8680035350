"""The paged-cache operators' cases: block tables and slot maps, rotary embedding (into the
cache, and for training), and attention of new tokens over a paged cache.

own = False computes each operator from elementary torch operations in 32 bits (64 for the
rotary angles); own = True makes the calls of exact_attention_146_b200.  exact() is a separate
computation in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of a small server: a token for each of 16 requests
        dict(name="tables decode 16", op="reserve", R=16, new=1, ctx=4000, page=16, pad=0, lens=1),
        # a large batch that mixes decoding requests, idle ones and prompt chunks, in buffers with some room behind
        dict(name="tables mixed 1500", op="reserve", R=1500, new=200, ctx=8000, page=16, pad=37, lens=2),
        # a third of the requests of a batch finish and give their blocks back
        dict(name="tables release 301", op="release", R=301, new=0, ctx=16000, page=32, pad=0, lens=3),
        # the keys and values of one decoding step, some rows of the captured batch unused
        dict(name="rope decode 48", op="append", T=48, pad=5, Hq=32, Hkv=8, d=128, rot=128, axes=1, pairs=False, mixed=False,
             page=16, layout="nhd", dtype="bf16", far=120000),
        # a video prompt: time, height and width axes, odd token count, slices of one fused projection
        dict(name="rope video 5003", op="append", T=5003, pad=0, Hq=16, Hkv=16, d=80, rot=80, axes=3, pairs=False, mixed=True,
             page=32, layout="hnd", dtype="f16", far=4000),
        # a training step's queries and keys, and their gradients
        dict(name="rope train 16384", op="train", T=16384, Hq=32, Hkv=8, d=128, rot=128, axes=1, pairs=False, mixed=False,
             dtype="bf16", far=4096),
        # decoding for a handful of short requests: the smallest call, latency counts
        dict(name="attend decode 4x1000", op="attend", R=4, new=1, ctx=1000, Hq=32, Hkv=8, d=128, page=16, window=0, causal=True,
             layout="nhd", dtype="bf16", pad=0, lens=4),
        # decoding for a full batch of long requests, rows of the captured batch unused
        dict(name="attend decode 48x16k", op="attend", R=48, new=1, ctx=16000, Hq=32, Hkv=8, d=128, page=16, window=0, causal=True,
             layout="nhd", dtype="bf16", pad=3, lens=5),
        # prompt chunks beside long contexts
        dict(name="attend chunks 8x512", op="attend", R=8, new=512, ctx=8000, Hq=32, Hkv=8, d=128, page=64, window=0, causal=True,
             layout="nhd", dtype="bf16", pad=0, lens=6),
        # ragged prompts, some of a single token, no shared heads
        dict(name="attend ragged 37 d64", op="attend", R=37, new=300, ctx=2500, Hq=16, Hkv=16, d=64, page=32, window=0, causal=True,
             layout="hnd", dtype="f16", pad=0, lens=7),
        # local attention with wide heads
        dict(name="attend window 5 d256", op="attend", R=5, new=700, ctx=6000, Hq=12, Hkv=4, d=256, page=16, window=1000, causal=True,
             layout="nhd", dtype="bf16", pad=0, lens=8),
        # the last chunk of one long prompt: the largest call
        dict(name="attend prefill 4096", op="attend", R=1, new=4096, ctx=28672, Hq=32, Hkv=8, d=128, page=128, window=0, causal=True,
             layout="nhd", dtype="bf16", pad=0, lens=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["reserve", "release", "append", "train", "attend", "attend", "attend"])
    lens = rng.randrange(1, 1 << 20)
    page = rng.choice([16, 32, 48, 64, 128])
    if op in ("reserve", "release"):
        R = _log(rng, 1, 1500)
        new = 0 if op == "release" else _log(rng, 1, max(1, min(4096, 300000 // R)))
        return dict(op=op, R=R, new=new, ctx=_log(rng, 1, 16000), page=page, pad=rng.choice([0, 0, 29]), lens=lens)
    Hkv = rng.choice([1, 2, 4, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "f16"])
    layout = rng.choice(["nhd", "hnd"])
    if op in ("append", "train"):
        d = rng.choice([32, 64, 80, 96, 128, 192, 256])
        axes = rng.choice([1, 1, 2, 3])
        c = dict(op=op, T=_log(rng, 1, max(8, 16384 * 5120 // ((Hq + Hkv) * d * 2))), Hq=Hq, Hkv=Hkv, d=d,
                 rot=rng.choice([d, d // 2]), axes=axes, pairs=rng.random() < 0.3, mixed=rng.random() < 0.5, dtype=dtype,
                 far=_log(rng, 100, 1000000))
        return c if op == "train" else dict(c, pad=rng.choice([0, 0, 3]), page=page, layout=layout)
    R = _log(rng, 1, 64)
    new = rng.choice([1, 1, _log(rng, 2, 4096)])
    ctx = _log(rng, 1, 28000)
    d = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
    # no more than the largest listed case, in the plain form's padded scores and in gathered keys
    while R > 1 and (R * new * (ctx + new) * Hq * max(d, 128) > 128 * 4096 * 32768 * 16 or R * (ctx + new) * Hkv * d > 5e8):
        R = max(1, R // 2)
    while new * (ctx + new) * Hq * max(d, 128) > 128 * 4096 * 32768 * 24:
        new = max(1, new // 2)
    causal = rng.random() < 0.9
    window = _log(rng, 16, 4000) if causal and rng.random() < 0.25 else 0
    return dict(op=op, R=R, new=new, ctx=ctx, Hq=Hq, Hkv=Hkv, d=d, page=page, window=window, causal=causal, layout=layout,
                dtype=dtype, pad=rng.choice([0, 0, 5]), lens=lens)


def _lengths(c):
    """The case's lengths: (tokens held before, new tokens) of each request."""
    R, new, ctx = c["R"], c["new"], c["ctx"]
    if c["lens"] == 0:   # full lengths
        return [ctx] * R, [new] * R
    rng = random.Random(c["lens"])
    ctxs = [rng.randint(ctx // 4, ctx) if rng.random() < 0.9 else rng.randint(0, min(ctx, 40)) for _ in range(R)]
    if new <= 1:
        return ctxs, [new] * R
    news = [rng.choice([0, 1, 1, rng.randint(1, new), rng.randint(1, new), new]) for _ in range(R)]
    news[rng.randrange(R)] = new
    return ctxs, news


def _blocks(n, page):
    return -(-n // page)


def _sections(c):
    """Pairs of each axis: (time, height, width) get about (2, 1, 1) ... of the rot / 2 pairs."""
    n, a = c["rot"] // 2, c["axes"]
    side = n // (a + 1)
    return [n - side * (a - 1)] + [side] * (a - 1)


def _axis_of(c):
    """The axis of each rotary pair: whole sections, or axes in turn until each has its share."""
    left, got = _sections(c), []
    if not c["mixed"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    left = list(left)
    while any(left):
        for a in range(len(left)):
            if left[a]:
                got.append(a)
                left[a] -= 1
    return got


# ------------------------------------------------------------------------------- inputs

def _cache(c, blocks, g, fill):
    """k and v caches, logically [block, slot, head, d]; "hnd" keeps a head's slots together in memory."""
    dt = DTYPES[c["dtype"]]
    Hkv, d, page = c["Hkv"], c["d"], c["page"]

    def one():
        shape = (blocks, page, Hkv, d) if c["layout"] == "nhd" else (blocks, Hkv, page, d)
        t = torch.empty(shape, device=DEV, dtype=dt)
        t.normal_(generator=g) if fill else t.zero_()
        return t if c["layout"] == "nhd" else t.permute(0, 2, 1, 3)
    return one(), one()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("reserve", "release"):
        ctxs, news = _lengths(c)
        page, R = c["page"], c["R"]
        held = [_blocks(x, page) for x in ctxs]
        tot = [_blocks(x + n, page) for x, n in zip(ctxs, news)]
        most = max(max(tot), _blocks(c["ctx"] + c["new"], page))
        spare = sum(tot) - sum(held) + 17
        blocks = sum(held) + spare
        ids = torch.randperm(blocks, device=DEV, generator=g).to(torch.int32)
        table = torch.full((R, most), -1, dtype=torch.int32, device=DEV)
        h = torch.tensor(held, device=DEV)
        mine = torch.arange(most, device=DEV)[None] < h[:, None]
        table[mine] = ids[:sum(held)]
        stack = torch.zeros(blocks, dtype=torch.int32, device=DEV)   # blocks that are free: stack[:count]
        stack[:spare] = ids[sum(held):]
        s.update(ctx=_i32(ctxs), table=table, stack=stack, count=_i32([spare]), tokens=sum(news), room=sum(news) + c["pad"])
        if c["op"] == "reserve":
            s.update(new=_i32(news))
        else:
            s.update(done=(torch.rand(R, device=DEV, generator=g) < 0.34).to(torch.int32))
        if own:   # the output buffers that a serving loop keeps
            whole = dict(dtype=torch.int32, device=DEV)
            s["outs"] = dict(free_count_out=torch.empty(1, **whole))
            if c["op"] == "reserve":
                s["outs"].update(cu_seqlens=torch.empty(R + 1, **whole), seq_lens=torch.empty(R, **whole),
                                 positions=torch.empty(s["room"], **whole), slots=torch.empty(s["room"], dtype=torch.int64, device=DEV))
            else:
                s["outs"].update(lens_out=torch.empty(R, **whole))
        return s
    dt = DTYPES[c["dtype"]]
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    if c["op"] in ("append", "train"):
        T, axes = c["T"], c["axes"]
        fused = torch.empty(T, Hq + 2 * Hkv, d, device=DEV, dtype=dt).normal_(generator=g)
        s.update(q=fused[:, :Hq], k=fused[:, Hq:Hq + Hkv], v=fused[:, Hq + Hkv:])
        if axes == 1:   # text: consecutive positions that end at `far`
            pos = torch.arange(T, device=DEV)[None] + max(0, c["far"] - T)
        else:           # frames of patches: the first axis runs on, the others walk a grid
            side = max(1, int(math.sqrt(max(1, T // 8))))
            t = torch.arange(T, device=DEV)
            pos = torch.stack([t // (side * side) + c["far"] // 2, (t // side) % side + c["far"] // 3, t % side + c["far"] // 4][:axes])
        s["pos"] = pos.to(torch.int32).contiguous()
        if c["op"] == "append":
            page = c["page"]
            blocks = _blocks(T, page) + 3
            s["kc"], s["vc"] = _cache(c, blocks, g, False)
            order = torch.randperm(blocks, device=DEV, generator=g)
            t = torch.arange(T, device=DEV)
            slots = order[t // page] * page + t % page
            slots[T - c["pad"]:] = -1
            s["slots"] = slots
            s["q_out"] = torch.zeros(T, Hq, d, device=DEV, dtype=dt)
        else:
            s["dq"] = torch.empty(T, Hq, d, device=DEV, dtype=dt).normal_(generator=g)
            s["dk"] = torch.empty(T, Hkv, d, device=DEV, dtype=dt).normal_(generator=g)
        inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])
        s["inv"], s["axis"] = inv.to(DEV), torch.tensor(_axis_of(c), device=DEV)
        if own:
            import exact_attention_146_b200 as fa
            s["rope"] = fa.RopeTable(inv.tolist(), axis=_axis_of(c), interleaved=c["pairs"])
        return s
    # attention over a paged cache
    ctxs, news = _lengths(c)
    page, T = c["page"], sum(news) + c["pad"]
    lens = [x + n for x, n in zip(ctxs, news)]
    need = [_blocks(x, page) for x in lens]
    blocks = sum(need) + 2
    s["kc"], s["vc"] = _cache(c, blocks, g, True)
    ids = torch.randperm(blocks, device=DEV, generator=g).to(torch.int32)
    table = torch.zeros((c["R"], max(1, max(need))), dtype=torch.int32, device=DEV)
    table[torch.arange(table.shape[1], device=DEV)[None] < torch.tensor(need, device=DEV)[:, None]] = ids[:sum(need)]
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    s.update(table=table, cu=_i32(cu), lens=_i32(lens), most_new=max(news), most_len=max(lens), total=sum(news))
    s["q"] = torch.empty(T, Hq, d, device=DEV, dtype=dt).normal_(generator=g)
    s["out"] = torch.zeros(T, Hq, d, device=DEV, dtype=dt)
    s["lse"] = torch.zeros(Hq, T, device=DEV, dtype=torch.float32)
    if own:
        import exact_attention_146_b200 as fa
        s["work"] = torch.empty(fa.paged_workspace_bytes(Hq, Hkv, d), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------- the framework's calls

def _own(s):
    import exact_attention_146_b200 as fa
    c = s["case"]
    if c["op"] == "reserve":
        cu, lens, pos, slots, count = fa.fa_kv_reserve(s["ctx"], s["new"], s["table"], s["stack"], s["count"], page_size=c["page"],
                                                       **s["outs"])
        return [cu, lens, pos, slots, count, s["table"]]
    if c["op"] == "release":
        lens, count = fa.fa_kv_release(s["ctx"], s["done"], s["table"], s["stack"], s["count"], page_size=c["page"], **s["outs"])
        return [lens, count, s["stack"]]
    if c["op"] == "append":
        fa.fa_rope_append(s["q"], s["k"], s["v"], s["pos"], s["rope"], s["kc"], s["vc"], s["slots"], q_out=s["q_out"])
        return [s["q_out"], s["kc"], s["vc"]]
    if c["op"] == "train":
        q, k = fa.fa_rope(s["q"], s["pos"], s["rope"], k=s["k"])
        dq, dk = fa.fa_rope(s["dq"], s["pos"], s["rope"], k=s["dk"], inverse=True)
        return [q, k, dq, dk]
    out, lse = fa.fa_paged_fwd(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["lens"], max_new=s["most_new"], causal=c["causal"],
                               window=c["window"] or None, out=s["out"], lse=s["lse"], workspace=s["work"])
    return [out, lse]


# ------------------------------------------------------------------------------- the plain forms

def _plain_reserve(s):
    page, ctx, new = s["case"]["page"], s["ctx"].long(), s["new"].long()
    total = ctx + new
    held, want = (ctx + page - 1) // page, (total + page - 1) // page
    off = torch.cumsum(want - held, 0) - (want - held)
    col = torch.arange(s["table"].shape[1], device=DEV)[None]
    fresh = (col >= held[:, None]) & (col < want[:, None])
    nth = s["count"].long() - 1 - (off[:, None] + col - held[:, None])
    table = torch.where(fresh, s["stack"][nth.clamp(0, s["stack"].numel() - 1)], s["table"])
    ends = torch.cumsum(new, 0)
    cu = torch.cat([torch.zeros_like(ends[:1]), ends])
    req = torch.repeat_interleave(torch.arange(new.numel(), device=DEV), new, output_size=s["tokens"])
    pos = ctx[req] + torch.arange(s["tokens"], device=DEV) - cu[req]
    slots = table[req, pos // page].long() * page + pos % page
    count = s["count"] - (want - held).sum().to(torch.int32)
    behind = torch.zeros(s["room"] - s["tokens"], dtype=torch.long, device=DEV)   # rows behind the last token: position 0, no slot
    return [cu.int(), total.int(), torch.cat([pos, behind]).int(), torch.cat([slots, behind - 1]), count, table]


def _plain_release(s):
    page, held = s["case"]["page"], (s["ctx"].long() + s["case"]["page"] - 1) // s["case"]["page"]
    gone = s["done"] != 0
    n = torch.where(gone, held, 0)
    off = torch.cumsum(n, 0) - n
    col = torch.arange(s["table"].shape[1], device=DEV)[None]
    mine = col < n[:, None]
    at = torch.where(mine, s["count"].long() + off[:, None] + col, s["stack"].numel())
    stack = torch.cat([s["stack"], s["stack"][:1]])
    stack[at.reshape(-1)] = s["table"].reshape(-1)   # the last place takes what is not given back
    return [torch.where(gone, 0, s["ctx"]), s["count"] + n.sum().to(torch.int32), stack[:-1]]


def _rotate(x, cos, sin, pairs):
    """Rotates the first 2 * cos.shape[-1] values of each head by the angles, in 32 bits."""
    n = cos.shape[-1]
    x32 = x.float()
    a, b = (x32[..., 0:2 * n:2], x32[..., 1:2 * n:2]) if pairs else (x32[..., :n], x32[..., n:2 * n])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if pairs else torch.cat([ra, rb], -1)
    return torch.cat([turned, x32[..., 2 * n:]], -1).to(x.dtype)


def _cos_sin(s):
    angle = s["pos"].double().t()[:, s["axis"]] * s["inv"]   # [T, rot / 2], in 64 bits: far positions
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _plain_append(s):
    cos, sin = _cos_sin(s)
    pairs, page = s["case"]["pairs"], s["case"]["page"]
    n = s["q"].shape[0] - s["case"]["pad"]   # the rows behind have no slot
    block, at = s["slots"][:n] // page, s["slots"][:n] % page
    s["q_out"][:n] = _rotate(s["q"], cos, sin, pairs)[:n]
    s["kc"][block, at] = _rotate(s["k"], cos, sin, pairs)[:n]
    s["vc"][block, at] = s["v"][:n]
    return [s["q_out"], s["kc"], s["vc"]]


def _plain_train(s):
    cos, sin = _cos_sin(s)
    pairs = s["case"]["pairs"]
    return [_rotate(s["q"], cos, sin, pairs), _rotate(s["k"], cos, sin, pairs), _rotate(s["dq"], cos, -sin, pairs),
            _rotate(s["dk"], cos, -sin, pairs)]


def _plain_attend(s):
    c = s["case"]
    page, Hkv, d = c["page"], c["Hkv"], c["d"]
    rep, R, most, L = c["Hq"] // Hkv, c["R"], s["most_new"], s["most_len"]
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    j = torch.arange(L, device=DEV)
    i = torch.arange(most, device=DEV)
    block = s["table"].long()[:, j // page]                                    # [R, L]
    k = s["kc"][block, (j % page)[None]].float()                               # [R, L, Hkv, d]
    v = s["vc"][block, (j % page)[None]].float()
    there = i[None] < new[:, None]                                             # [R, most]
    row = torch.where(there, s["cu"][:-1].long()[:, None] + i[None], 0)
    q = s["q"][row].float().reshape(R, most, Hkv, rep, d).permute(0, 2, 3, 1, 4).reshape(R, Hkv, rep * most, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(d))          # [R, Hkv, rep * most, L]
    last = i[None] + (s["lens"].long() - new)[:, None]                         # the row's own position
    seen = (j[None] < s["lens"].long()[:, None])[:, None, :].expand(R, most, L)
    if c["causal"]:
        seen = seen & (j[None, None] <= last[..., None])
    if c["window"]:
        seen = seen & (j[None, None] > last[..., None] - c["window"])
    hidden = ~seen[:, None, None]                                              # [R, 1, 1, most, L]
    x.view(R, Hkv, rep, most, L).masked_fill_(hidden, float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total)).reshape(R, Hkv * rep, most)
    o = o.reshape(R, Hkv, rep, most, d).permute(0, 3, 1, 2, 4).reshape(R, most, Hkv * rep, d)
    # rows behind the last request stay as they are
    s["out"][:s["total"]] = o[there].to(s["out"].dtype)
    s["lse"][:, :s["total"]] = lse.permute(0, 2, 1)[there].t()
    return [s["out"], s["lse"]]


def run(state):
    if own:
        return _own(state)
    plain = {"reserve": _plain_reserve, "release": _plain_release, "append": _plain_append, "train": _plain_train, "attend": _plain_attend}
    return plain[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] in ("reserve", "release"):
        ctxs, news = _lengths(c)
        held = sum(_blocks(x, c["page"]) for x in ctxs)
        if c["op"] == "release":
            return {"bytes": 12 * c["R"] + 8 * held // 3, "flops": 0}
        fresh = sum(_blocks(x + n, c["page"]) for x, n in zip(ctxs, news)) - held
        return {"bytes": 16 * c["R"] + 12 * (sum(news) + c["pad"]) + 8 * fresh, "flops": 0}
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    if c["op"] == "append":
        n = c["T"] - c["pad"]
        return {"bytes": 4 * n * (Hq + 2 * Hkv) * d + n * (4 * c["axes"] + 8), "flops": 3 * n * (Hq + Hkv) * c["rot"]}
    if c["op"] == "train":
        return {"bytes": 8 * c["T"] * (Hq + Hkv) * d + 8 * c["T"] * c["axes"], "flops": 6 * c["T"] * (Hq + Hkv) * c["rot"]}
    ctxs, news = _lengths(c)
    pairs = keys = 0
    for x, n in zip(ctxs, news):
        if not n:
            continue
        w = c["window"] or 1 << 60
        if c["causal"]:
            pairs += sum(min(x + i + 1, w) for i in range(n))
            keys += min(x + n, w + n - 1)
        else:
            pairs += n * (x + n)
            keys += x + n
    T = sum(news)
    return {"bytes": 4 * keys * Hkv * d + 4 * T * Hq * d + 4 * T * Hq, "flops": 4 * pairs * Hq * d}


# ------------------------------------------------------------------------------- the definitions, in 64 bits

def _turn64(x, s, sign):
    """Multiplies each pair, as a complex number, by exp(sign * i * position * frequency)."""
    c = s["case"]
    n = c["rot"] // 2
    x64 = x.double().clone()
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if c["pairs"] else (slice(0, n), slice(n, 2 * n))
    where = s["pos"].double()[s["axis"]]                        # [rot / 2, T]
    turn = torch.polar(torch.ones_like(where), sign * where * s["inv"][:, None]).t()[:, None]
    z = torch.complex(x64[..., first], x64[..., second]) * turn
    x64[..., first], x64[..., second] = z.real, z.imag
    return x64


def exact(case, seed):
    c = case
    if c["op"] in ("reserve", "release"):
        return None
    s = prepare(case, seed)
    if c["op"] == "train":
        return [_turn64(s["q"], s, 1.0), _turn64(s["k"], s, 1.0), _turn64(s["dq"], s, -1.0), _turn64(s["dk"], s, -1.0)]
    if c["op"] == "append":
        q, kc, vc = s["q_out"].double(), s["kc"].double(), s["vc"].double()
        k = _turn64(s["k"], s, 1.0)
        real = s["slots"] >= 0
        q[real] = _turn64(s["q"], s, 1.0)[real]
        slots = s["slots"][real]
        kc[slots // c["page"], slots % c["page"]] = k[real]
        vc[slots // c["page"], slots % c["page"]] = s["v"].double()[real]
        return [q, kc, vc]
    out, lse = s["out"].double(), s["lse"].double()
    rep = c["Hq"] // c["Hkv"]
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].long()
    for r in range(c["R"]):
        lo, hi, L = cu[r], cu[r + 1], lens[r]
        if hi == lo:
            continue
        pages = table[r, :_blocks(L, c["page"])]
        k = s["kc"][pages].reshape(-1, c["Hkv"], c["d"])[:L]
        v = s["vc"][pages].reshape(-1, c["Hkv"], c["d"])[:L]
        at = torch.arange(L - (hi - lo), L, device=DEV)[:, None]
        key = torch.arange(L, device=DEV)[None]
        mask = torch.zeros(hi - lo, L, dtype=torch.float64, device=DEV)
        if c["causal"]:
            mask[key > at] = -math.inf
        if c["window"]:
            mask[key <= at - c["window"]] = -math.inf
        for h in range(c["Hq"]):
            a = s["q"][lo:hi, h].double() @ k[:, h // rep].double().t() / math.sqrt(c["d"]) + mask
            z = torch.logsumexp(a, -1)
            lse[h, lo:hi] = z
            out[lo:hi, h] = torch.exp(a - z[:, None]) @ v[:, h // rep].double()
    return [out, lse]
