"""Plain 64-bit references of the paged-cache operators, and the tolerances of their kernels."""
from __future__ import annotations

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative


def blocks_of(n, page):
    return -(-n // page)


def make_paged(lens, page, Hkv, d, dtype, layout, seed, spare=3, poison=True, device="cuda"):
    """Caches and a block table for requests of `lens` keys in shuffled blocks.  With poison, every slot
    that holds no key is NaN, and table entries past a request's blocks name no block."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    need = [blocks_of(n, page) for n in lens]
    total = sum(need) + spare
    shape = {"nhd": (total, page, Hkv, d), "hnd": (total, Hkv, page, d), "pair": (total, 2, page, Hkv, d)}[layout]

    def fill(shape):
        t = torch.empty(shape, device=device, dtype=torch.float32)
        return t.normal_(generator=g).to(dtype)
    if layout == "pair":      # k and v slices of one tensor
        both = fill(shape)
        k, v = both[:, 0], both[:, 1]
    else:
        k, v = fill(shape), fill(shape)
        if layout == "hnd":
            k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    ids = torch.randperm(total, device=device, generator=g).tolist()
    table = torch.full((max(1, len(lens)), max(1, max(need, default=0)) + 2), 1 << 30 if poison else 0, dtype=torch.int32, device=device)
    at = 0
    used = torch.zeros((total, page), dtype=torch.bool, device=device)
    for r, n in enumerate(need):
        if n:
            table[r, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32, device=device)
            slots = torch.arange(lens[r], device=device)
            used[table[r, :n].long()[slots // page], slots % page] = True
            at += n
    if poison:
        k[~used] = float("nan")
        v[~used] = float("nan")
    return k, v, table


def attend64(q, k, v, table, cu, lens, *, causal, window, scale):
    """(out, lse, tolerance of out, tolerance of lse), in 64 bits, of the rows of all requests (others 0).

    Tolerances, for the kernels' arithmetic (u: half a step of the type): S is an fp32 sum of d products
    scaled by a rounded constant, |dS| <= (d + 4) 2^-24 sum |q k| scale; the exponential is off by at most
    2^-13.5 relative (its polynomial form; the hardware form by less); so each weight p / l is off by at most
    2 (dS + 2^-13.5) relative; P is rounded to the type (u), the fp32 sums of O and l add n 2^-24, and O is
    rounded once at the end.  fp16 has subnormals below 2^-14: half a step there is 2^-25, for P per key
    (against l >= 2^-8, the sum of weights where the reference maximum may lag by 2^8) and for O once."""
    T, Hq, d = q.shape
    page, Hkv = k.shape[1], k.shape[2]
    rep = Hq // Hkv
    u = HALF[q.dtype]
    out = torch.zeros((T, Hq, d), dtype=torch.float64, device=q.device)
    lse = torch.zeros((Hq, T), dtype=torch.float64, device=q.device)
    t_out, t_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(len(lens)):
        lo, hi, L = cu[r], cu[r + 1], lens[r]
        n = hi - lo
        if n <= 0:
            continue
        j = torch.arange(L, device=q.device)
        blk = table[r].long()[j // page] if L else j
        kk = k[blk, j % page].double() if L else torch.zeros((0, Hkv, d), dtype=torch.float64, device=q.device)
        vv = v[blk, j % page].double() if L else kk
        i = torch.arange(n, device=q.device)[:, None] + L - n
        seen = torch.ones((n, L), dtype=torch.bool, device=q.device)
        if causal:
            seen = j[None] <= i
        if window:
            seen = seen & (j[None] > i - window)
        for h in range(Hq):
            qh = q[lo:hi, h].double()
            s = qh @ kk[:, h // rep].t() * scale
            size = (qh.abs() @ kk[:, h // rep].abs().t() * scale).masked_fill(~seen, 0.0)
            s = s.masked_fill(~seen, -math.inf)
            z = torch.logsumexp(s, -1) if L else torch.full((n,), -math.inf, dtype=torch.float64, device=q.device)
            p = torch.exp(s - torch.where(torch.isinf(z), 0.0, z)[:, None])
            o = p @ vv[:, h // rep]
            a = p @ vv[:, h // rep].abs()
            dS = (d + 4) * 2.0 ** -24 * (size.amax(-1) if L else torch.zeros(n, dtype=torch.float64, device=q.device))
            rel = 2 * (dS + 2.0 ** -13.5 + (L + 2) * 2.0 ** -24)[:, None]
            tiny = (L * 2.0 ** -17 * (vv.abs().amax() if L else 0.0) + 2.0 ** -25) if q.dtype == torch.float16 else 1e-30
            out[lo:hi, h], lse[h, lo:hi] = o, z
            t_out[lo:hi, h] = (u * (1 + rel) + rel) * a + u * o.abs() * 1.01 + tiny
            t_lse[h, lo:hi] = dS + 2.0 ** -13.5 + (L + 2) * 2.0 ** -24 + 2.0 ** -22 * torch.where(torch.isinf(z), 0.0, z.abs())
    return out, lse, t_out, t_lse


def rope64(x, positions, inv_freq, axis, interleaved, sign=1.0):
    """The turn of every pair in 64 bits, as complex numbers; [T, H, d]."""
    n = len(inv_freq)
    y = x.double().clone()
    if n == 0:
        return y
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    pos = positions.double()[torch.tensor(axis, device=x.device)]
    angle = pos * torch.tensor(inv_freq, dtype=torch.float64, device=x.device)[:, None] * sign
    turn = torch.polar(torch.ones_like(angle), angle).t()[:, None]
    z = torch.complex(y[..., a], y[..., b]) * turn
    y[..., a], y[..., b] = z.real, z.imag
    return y


def rope_tolerance(x, y64, n, interleaved):
    """The angle is rounded to 2^-25 of a turn, and sine and cosine of it to a few 2^-24: at most 2^-20 of
    |x1| + |x2| in all, then two fp32 products and a sum, and one rounding of the result."""
    u = HALF[x.dtype]
    size = x.double().abs().clone()
    if n:
        a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
        both = size[..., a] + size[..., b]
        size[..., a], size[..., b] = both, both
    return u * y64.abs() * 1.001 + 2.0 ** -20 * size + (2.0 ** -25 if x.dtype == torch.float16 else 0.0)


def reserve_plain(ctx, new, table, free, count, page, T, max_blocks):
    """fa_kv_reserve on lists; returns (cu, lens, positions, slots, count, table)."""
    table = [list(row) for row in table]
    cu, lens, pos, slots = [0], [], [], []
    for r, (c, n) in enumerate(zip(ctx, new)):
        for b in range(blocks_of(c, page), blocks_of(c + n, page)):
            count -= 1
            table[r][b] = free[count]
        for x in range(c, c + n):
            pos.append(x)
            slots.append(table[r][x // page] * page + x % page)
        cu.append(cu[-1] + n)
        lens.append(c + n)
    pad = T - len(pos)
    return cu, lens, pos + [0] * pad, slots + [-1] * pad, count, table
