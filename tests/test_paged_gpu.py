"""The paged-cache operators on the GPU against plain 64-bit references: block tables and slots, rotary
embedding, attention over the cache, and a serving loop that runs them together."""
import math
import random

import pytest

import exact_attention_146_b200 as fa
from tests import _paged

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built_library():
    from exact_attention_146_b200 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.device_status()
    yield


@pytest.fixture(autouse=True)
def status_is_clean():
    yield
    st, word = fa.device_status()
    assert st == fa.FA_OK, f"device status {st} ({word:#x})"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------- block tables

def pool(ctx, page, max_blocks, spare, seed):
    """A table of the requests' blocks and a stack of `spare` free ones."""
    rng = random.Random(seed)
    held = [_paged.blocks_of(c, page) for c in ctx]
    ids = list(range(sum(held) + spare))
    rng.shuffle(ids)
    table, at = [], 0
    for n in held:
        table.append(ids[at:at + n] + [-7] * (max_blocks - n))
        at += n
    return table, ids[at:] + [-9] * at, spare


@pytest.mark.parametrize("R,page,most,pad,stride", [(1, 16, 1, 0, 0), (1, 1, 5, 2, 0), (7, 16, 40, 3, 5), (33, 48, 300, 0, 0),
                                                    (256, 16, 1, 5, 0), (257, 5, 9, 0, 1), (1024, 16, 3, 1, 0),
                                                    (1025, 32, 2, 0, 0), (2600, 16, 100, 17, 0), (3, 128, 4096, 0, 0)])
def test_reserve_then_release(R, page, most, pad, stride):
    rng = random.Random(R * 31 + page)
    ctx = [rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, 5 * page)]) for _ in range(R)]
    new = [rng.choice([0, 1, most, rng.randint(0, most)]) for _ in range(R)]
    width = max(_paged.blocks_of(c + n, page) for c, n in zip(ctx, new)) + 1
    spare = sum(_paged.blocks_of(c + n, page) - _paged.blocks_of(c, page) for c, n in zip(ctx, new)) + 2
    table, free, count = pool(ctx, page, width, spare, R)
    T = sum(new) + pad
    whole = i32([row + [-5] * stride for row in table])
    tab = whole[:, :width]
    cu, lens, pos, slots, cnt = fa.fa_kv_reserve(i32(ctx), i32(new), tab, i32(free), i32([count]), page_size=page, num_tokens=T)
    ref = _paged.reserve_plain(ctx, new, table, free, count, page, T, width)
    assert cu.tolist() == ref[0] and lens.tolist() == ref[1] and pos.tolist() == ref[2] and slots.tolist() == ref[3]
    assert cnt.tolist() == [ref[4]] and tab.tolist() == ref[5]
    assert stride == 0 or bool((whole[:, width:] == -5).all())
    # in place, and back
    ctx_d, cnt_d, tab2 = i32(ctx), i32([count]), i32(table)
    fa.fa_kv_reserve(ctx_d, i32(new), tab2, i32(free), cnt_d, page_size=page, num_tokens=T, seq_lens=ctx_d, free_count_out=cnt_d)
    assert ctx_d.tolist() == ref[1] and cnt_d.tolist() == [ref[4]] and tab2.tolist() == ref[5]
    done = [rng.choice([0, 0, 1, 5]) for _ in range(R)]
    stack = i32(free)
    fa.fa_kv_release(ctx_d, i32(done), tab2, stack, cnt_d, page_size=page, lens_out=ctx_d, free_count_out=cnt_d)
    want, n = list(free), ref[4]
    for r in range(R):
        if done[r]:
            for b in range(_paged.blocks_of(ref[1][r], page)):
                want[n] = ref[5][r][b]
                n += 1
    assert cnt_d.tolist() == [n] and stack.tolist() == want and tab2.tolist() == ref[5]
    assert ctx_d.tolist() == [0 if f else x for f, x in zip(done, ref[1])]


def test_reserve_of_no_requests():
    cu, lens, pos, slots, cnt = fa.fa_kv_reserve(i32([]), i32([]), torch.zeros((0, 4), dtype=torch.int32, device="cuda"), i32([3, 4]),
                                                 i32([2]), page_size=16, num_tokens=5)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 5 and pos.tolist() == [0] * 5 and cnt.tolist() == [2]


@pytest.mark.parametrize("ctx,new,free,count,site", [
    ([3, -1], [1, 1], [0, 1, 2, 3, 4, 5], 6, 41),          # a negative length
    ([3, 20], [1, -2], [0, 1, 2, 3, 4, 5], 6, 41),
    ([3, 60], [1, 10], [0, 1, 2, 3, 4, 5], 6, 41),         # longer than its row of the table (4 x 16)
    ([3, 20], [5, 10], [0, 1, 2, 3, 4, 5], 6, 42),         # more tokens than rows
    ([0, 0], [4, 4], [0, 1, 2, 3, 4, 5], 1, 43),           # more blocks than are free
    ([0, 0], [4, 4], [0, 1, 2, 3, 4, 5], 9, 43),           # a count beyond the stack
])
def test_reserve_refuses_a_whole_step(ctx, new, free, count, site):
    table = i32([[7, 7, 7, 7]] * 2)
    cu, lens, pos, slots, cnt = fa.fa_kv_reserve(i32(ctx), i32(new), table, i32(free), i32([count]), page_size=16, num_tokens=12)
    st, word = fa.device_status()
    assert st == fa.FA_ERR_PAGED_RANGE and (word >> 8) & 0xFF == site
    assert cu.tolist() == [0, 0, 0] and lens.tolist() == ctx and slots.tolist() == [-1] * 12 and cnt.tolist() == [count]
    assert bool((table == 7).all())


def test_bad_block_ids_are_reported_and_get_no_slot():
    table = i32([[99, -1], [3, -1]])
    _, _, pos, slots, _ = fa.fa_kv_reserve(i32([3, 15]), i32([2, 3]), table, i32([0, -4]), i32([2]), page_size=16, num_tokens=5)
    st, word = fa.device_status()
    assert st == fa.FA_ERR_PAGED_RANGE and (word >> 8) & 0xFF in (44, 45)
    assert pos.tolist() == [3, 4, 15, 16, 17] and slots.tolist() == [-1, -1, -1, -1, -1]   # 2 blocks: ids 0 and 1 alone are right


def test_release_refuses_more_blocks_than_the_stack_holds():
    stack = i32([5, 6, 7, 8])
    lens, cnt = fa.fa_kv_release(i32([33, 4]), i32([1, 0]), i32([[0, 1, 2], [3, 0, 0]]), stack, i32([2]), page_size=16)
    st, word = fa.device_status()
    assert st == fa.FA_ERR_PAGED_RANGE and (word >> 8) & 0xFF == 43
    assert lens.tolist() == [33, 4] and cnt.tolist() == [2] and stack.tolist() == [5, 6, 7, 8]


# ------------------------------------------------------------------------------- rotary embedding

def spec(rot, axes):
    inv = [10000.0 ** (-2.0 * i / max(rot, 1)) for i in range(rot // 2)]
    return inv, [i % axes for i in range(rot // 2)]


ROPE = [(torch.bfloat16, 128, 128, 1, False, 1, 4, 2), (torch.float16, 128, 64, 2, True, 700, 3, 1),
        (torch.bfloat16, 80, 80, 3, False, 33, 16, 16), (torch.bfloat16, 80, 20, 3, True, 129, 5, 1),
        (torch.float16, 32, 32, 4, False, 1000, 1, 1), (torch.bfloat16, 64, 6, 1, False, 3, 2, 2),
        (torch.float16, 256, 256, 1, True, 601, 8, 1), (torch.bfloat16, 192, 96, 3, False, 64, 6, 2),
        (torch.bfloat16, 80, 40, 1, False, 700, 6, 2), (torch.float16, 80, 40, 2, True, 9, 3, 3),
        (torch.bfloat16, 96, 0, 1, False, 5, 2, 1), (torch.float16, 96, 96, 1, True, 2500, 2, 0)]


def close(got, want, tol):
    bad = (got.double() - want).abs() > tol
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, worst {float(((got.double() - want).abs() / tol).max()):.2f} of the tolerance"


@pytest.mark.parametrize("dtype,d,rot,axes,pairs,T,Hq,Hkv", ROPE)
def test_rope_and_its_gradient(dtype, d, rot, axes, pairs, T, Hq, Hkv):
    torch.manual_seed(T + d)
    inv, axis = spec(rot, axes)
    table = fa.RopeTable(inv, axis=axis, interleaved=pairs)
    fused = torch.randn(T, Hq + 2 * Hkv, d, device="cuda").to(dtype)
    q, k = fused[:, :Hq], (fused[:, Hq:Hq + Hkv] if Hkv else None)
    pos = torch.randint(0, 1 << 20, (axes, T), device="cuda", dtype=torch.int32)
    for inverse in (False, True):
        got = fa.fa_rope(q, pos, table, k=k, inverse=inverse)
        got = got if Hkv else (got,)
        for g, x in zip(got, (q, k)):
            want = _paged.rope64(x, pos, inv, axis, pairs, -1.0 if inverse else 1.0)
            close(g, want, _paged.rope_tolerance(x, want, rot // 2, pairs))
    # in place on the projection: the same bits; what lies between the rows stays
    again = fused.clone()
    fa.fa_rope(again[:, :Hq], pos, table, k=again[:, Hq:Hq + Hkv] if Hkv else None, q_out=again[:, :Hq],
               k_out=again[:, Hq:Hq + Hkv] if Hkv else None)
    fresh = fa.fa_rope(q, pos, table, k=k)
    fresh = fresh if Hkv else (fresh,)
    assert torch.equal(again[:, :Hq], fresh[0]) and (Hkv == 0 or torch.equal(again[:, Hq:Hq + Hkv], fresh[1]))
    assert torch.equal(again[:, Hq + Hkv:], fused[:, Hq + Hkv:])


def test_rope_gradient_against_differences():
    """f(x) = sum(g * rope(x)) is linear: (f(x + h e) - f(x - h e)) / 2h in 64 bits is the gradient."""
    torch.manual_seed(5)
    inv, axis = spec(16, 2)
    pos = torch.randint(0, 5000, (2, 3), device="cuda", dtype=torch.int32)
    for pairs in (False, True):
        x = torch.randn(3, 1, 32, device="cuda").to(torch.float16)
        g = torch.randn(3, 1, 32, device="cuda").to(torch.float16)
        got = fa.fa_rope(g, pos, fa.RopeTable(inv, axis=axis, interleaved=pairs), inverse=True)

        def f(y):
            return float((_paged.rope64(y, pos, inv, axis, pairs) * g.double()).sum())
        for t in range(3):
            for e in range(32):
                h = torch.zeros(3, 1, 32, dtype=torch.float64, device="cuda")
                h[t, 0, e] = 0.5
                diff = f(x.double() + h) - f(x.double() - h)
                size = float(g[t].double().abs().max())
                assert abs(float(got[t, 0, e]) - diff) <= 2.0 ** -11 * abs(diff) + 2.0 ** -19 * size + 2.0 ** -25


@pytest.mark.parametrize("shift", [0, 1, 3])
def test_rope_of_unaligned_rows(shift):
    """Rows that start off a 16-byte boundary take the path of single values: the same numbers."""
    torch.manual_seed(9)
    inv, axis = spec(64, 1)
    table = fa.RopeTable(inv, axis=axis)
    buf = torch.randn(9 * (3 * 64 + shift) + 8, device="cuda").to(torch.bfloat16)
    x = torch.as_strided(buf, (9, 3, 64), (3 * 64 + shift, 64, 1), shift)
    pos = torch.arange(9, device="cuda", dtype=torch.int32) * 1000
    want = _paged.rope64(x, pos[None], inv, axis, False)
    close(fa.fa_rope(x, pos, table), want, _paged.rope_tolerance(x, want, 32, False))


@pytest.mark.parametrize("dtype,d,rot,axes,pairs,T,Hq,Hkv", ROPE[:11])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "pair"])
def test_rope_append(dtype, d, rot, axes, pairs, T, Hq, Hkv, layout):
    torch.manual_seed(T + d + 1)
    inv, axis = spec(rot, axes)
    page = 16
    k_cache, v_cache, _ = _paged.make_paged([T], page, Hkv, d, dtype, layout, 3, poison=False)
    before = k_cache.clone(), v_cache.clone()
    fused = torch.randn(T, Hq + 2 * Hkv, d, device="cuda").to(dtype)
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    pos = torch.randint(0, 1 << 17, (axes, T), device="cuda", dtype=torch.int32)
    slots = torch.randperm(k_cache.shape[0] * page, device="cuda")[:T]
    slots[torch.rand(T, device="cuda") < 0.2] = -1
    q_out = torch.full((T, Hq, d), 7.0, device="cuda", dtype=dtype)
    fa.fa_rope_append(q, k, v, pos, fa.RopeTable(inv, axis=axis, interleaved=pairs), k_cache, v_cache, slots, q_out=q_out)
    real = slots >= 0
    assert bool((q_out[~real] == 7.0).all())
    want = _paged.rope64(q, pos, inv, axis, pairs)
    close(q_out[real], want[real], _paged.rope_tolerance(q, want, rot // 2, pairs)[real])
    at = slots[real] // page, slots[real] % page
    want = _paged.rope64(k, pos, inv, axis, pairs)
    close(k_cache[at], want[real], _paged.rope_tolerance(k, want, rot // 2, pairs)[real])
    assert torch.equal(v_cache[at], v[real])
    rest = torch.ones(k_cache.shape[:2], dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(k_cache[rest], before[0][rest]) and torch.equal(v_cache[rest], before[1][rest])


def test_rope_append_reports_a_slot_past_the_cache():
    k_cache, v_cache, _ = _paged.make_paged([16], 16, 1, 64, torch.bfloat16, "nhd", 4, poison=False)
    x = torch.randn(3, 1, 64, device="cuda").to(torch.bfloat16)
    slots = torch.tensor([0, 64 * 16, 1], device="cuda")
    fa.fa_rope_append(None, x, x, i32([0, 1, 2]), fa.RopeTable([1.0] * 32), k_cache, v_cache, slots)
    st, word = fa.device_status()
    assert st == fa.FA_ERR_PAGED_RANGE and (word >> 8) & 0xFF == 46 and word >> 16 == 1
    assert torch.equal(v_cache[0, 0], x[0]) and torch.equal(v_cache[0, 1], x[2])


# ------------------------------------------------------------------------------- attention over the cache

def attend(lens, news, *, Hq, Hkv, d, page, dtype=torch.bfloat16, layout="nhd", causal=True, window=None, scale=None, pad=0, seed=0,
           gap=0, max_new=None, workspace=None, sharp=1.0, poison=True):
    """Runs fa_paged_fwd and compares every row; rows of no request keep their canary."""
    k, v, table = _paged.make_paged(lens, page, Hkv, d, dtype, layout, seed + 1, poison=poison)
    T = sum(news) + pad
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = (torch.empty(T, Hq + gap, d, device="cuda").normal_(generator=g) * sharp).to(dtype)[:, :Hq]
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.full((T, Hq, d), 3.0, device="cuda", dtype=dtype)
    lse = torch.full((Hq, T), 3.0, device="cuda")
    kw = dict(max_new=max(news, default=0) if max_new is None else max_new, causal=causal, window=window, scale=scale, workspace=workspace)
    fa.fa_paged_fwd(q, k, v, table, i32(cu), i32(lens), out=out, lse=lse, **kw)
    st, word = fa.device_status()
    assert st == fa.FA_OK, f"device status {st} ({word:#x})"
    want, z, t_out, t_lse = _paged.attend64(q, k, v, table, cu, lens, causal=causal, window=window, scale=scale)
    n = sum(news)
    close(out[:n], want[:n], t_out[:n])
    none = torch.isinf(z[:, :n])
    assert torch.equal(torch.isinf(lse[:, :n]), none) and bool((lse[:, :n][none] < 0).all())
    close(torch.where(none, 0.0, lse[:, :n]), torch.where(none, 0.0, z[:, :n]), t_lse[:, :n])
    assert bool((out[n:] == 3.0).all()) and bool((lse[:, n:] == 3.0).all())
    again = torch.full_like(out, 3.0)
    fa.fa_paged_fwd(q, k, v, table, i32(cu), i32(lens), out=again, return_lse=False, **kw)
    assert torch.equal(out, again)   # the same bits, with or without the LSE
    return q, k, v, table, cu, out, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [32, 64, 80, 96, 128, 192, 256])
def test_decode_every_head_dim(d, dtype):
    attend([1, 16, 17, 300, 1037, 0, 129], [1, 1, 1, 1, 1, 0, 1], Hq=8, Hkv=2, d=d, page=16, dtype=dtype, pad=3, seed=d)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (8, 8), (6, 2), (16, 1), (32, 1), (10, 2), (24, 2), (40, 2), (14, 2)])
def test_decode_head_ratios(Hq, Hkv):
    attend([33, 250, 1, 77], [1, 1, 1, 1], Hq=Hq, Hkv=Hkv, d=64, page=32, seed=Hq)


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 48, 100, 256])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "pair"])
def test_pages_and_layouts(page, layout):
    attend([130, 1, 513, 255], [1, 1, 1, 0], Hq=4, Hkv=2, d=64, page=page, layout=layout, seed=page)
    attend([130, 40, 513, 255], [100, 1, 30, 0], Hq=4, Hkv=2, d=64, page=page, layout=layout, seed=page + 1)


@pytest.mark.parametrize("new", [2, 3, 4, 7, 8, 16, 17, 31])
def test_a_few_new_tokens(new):
    attend([new, 500, 129, 64 + new], [new, new, 1, new // 2], Hq=8, Hkv=2, d=128, page=16, seed=new)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [32, 64, 80, 96, 128, 192, 256])
def test_chunks_every_head_dim(d, dtype):
    attend([700, 1, 333, 0, 900, 257], [300, 1, 333, 0, 65, 256], Hq=4, Hkv=2, d=d, page=16, dtype=dtype, pad=5, seed=d, gap=2)


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (3, 1), (12, 4), (16, 1), (5, 1), (40, 1), (14, 2), (130, 1)])
def test_chunks_head_ratios(Hq, Hkv):
    attend([400, 90, 129], [150, 33, 1], Hq=Hq, Hkv=Hkv, d=64, page=16, seed=Hq)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 5, 16, 100, 128, 129, 5000])
def test_window(window, d):
    attend([1000, 40, 129, 2000], [260, 40, 1, 1], Hq=4, Hkv=2, d=d, page=16, window=window, seed=window)
    attend([1000, 40, 129, 2000], [1, 1, 1, 2], Hq=4, Hkv=2, d=d, page=16, window=window, seed=window)


@pytest.mark.parametrize("d", [80, 128, 256])
def test_no_mask(d):
    attend([1000, 40, 129], [260, 50, 1], Hq=4, Hkv=2, d=d, page=32, causal=False, seed=d)
    attend([1000, 40, 129], [1, 2, 1], Hq=4, Hkv=2, d=d, page=32, causal=False, seed=d)


@pytest.mark.parametrize("news,lens", [([5, 3], [3, 0]), ([300, 200], [40, 0]), ([1, 1], [0, 0]), ([140], [1])])
def test_rows_that_see_no_key(news, lens):
    """More new tokens than keys: the first rows see nothing (O = 0, LSE = -inf)."""
    attend(lens, news, Hq=4, Hkv=2, d=64, page=16, seed=7)
    attend(lens, news, Hq=4, Hkv=2, d=128, page=16, causal=False, seed=8)


@pytest.mark.parametrize("new", [1, 130])
def test_large_scores(new):
    """Scores of a few hundred: the running maximum moves and the old sums are rescaled."""
    attend([1500, 640], [new, 1], Hq=4, Hkv=1, d=128, page=16, sharp=25.0, seed=new)


@pytest.mark.parametrize("new,L", [(1, 40000), (200, 30000), (2000, 2000)])
def test_one_long_request(new, L):
    attend([L], [new], Hq=8, Hkv=1, d=128, page=64, layout="hnd", seed=L)


def test_many_requests():
    rng = random.Random(3)
    lens = [rng.randint(1, 60) for _ in range(1100)]
    attend(lens, [rng.choice([0, 1, 1]) for _ in lens], Hq=2, Hkv=1, d=64, page=16, seed=3)
    attend(lens[:300], [rng.randint(0, n) for n in lens[:300]], Hq=2, Hkv=1, d=64, page=16, seed=4)


def test_max_new_is_only_a_bound():
    for bound in (1, 4, 5, 70, 1000):
        attend([300, 41], [1, 1], Hq=8, Hkv=2, d=128, page=16, max_new=bound, seed=1)


def test_workspace_holds_anything():
    """No initial contents are needed, and the size given by the library is enough: a canary behind it stays."""
    need = fa.paged_workspace_bytes(8, 2, 128)
    buf = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")   # NaN everywhere
    for news in ([1, 1, 1], [700, 1, 90]):
        attend([5000, 41, 800], news, Hq=8, Hkv=2, d=128, page=16, workspace=buf[:need], seed=2)
        assert bool((buf[need:] == 255).all())


@pytest.mark.parametrize("news,max_new,lens,cu,site", [
    ([1, 1], 1, [20, -1], None, 41), ([1, 1], 1, [20, 5000], None, 41), ([3, 1], 2, [20, 9], None, 41),
    ([200, 1], 200, [220, -5], None, 41), ([1, 1], 1, [20, 9], [0, 1, 99], 41), ([1, 1], 1, [20, 9], [1, 0, 1], 41)])
def test_requests_out_of_range_are_left_out(news, max_new, lens, cu, site):
    """The others are right, the left out one's rows stay as they were, and the status word tells."""
    good = [n if 0 <= n <= 300 else 9 for n in lens]
    k, v, table = _paged.make_paged(good, 16, 1, 64, torch.bfloat16, "nhd", 1)
    T = sum(news)
    q = torch.randn(T, 2, 64, device="cuda").to(torch.bfloat16)
    at = cu or [0, news[0], T]
    out, lse = torch.full((T, 2, 64), 3.0, device="cuda", dtype=q.dtype), torch.full((2, T), 3.0, device="cuda")
    fa.fa_paged_fwd(q, k, v, table, i32(at), i32(lens), max_new=max_new, out=out, lse=lse)
    st, word = fa.device_status()
    assert st == fa.FA_ERR_PAGED_RANGE and (word >> 8) & 0xFF == site
    width = table.shape[1] * 16
    for r in range(2):
        lo, hi = at[r], at[r + 1]
        if not (0 <= lo <= hi <= T):
            continue
        if hi - lo > max_new or not 0 <= lens[r] <= width:
            assert bool((out[lo:hi] == 3.0).all()) and bool((lse[:, lo:hi] == 3.0).all())
        else:
            want, z, t_out, t_lse = _paged.attend64(q, k, v, table, [0] * r + [lo, hi], [0] * r + [lens[r]], causal=True, window=None,
                                                    scale=0.125)
            close(out[lo:hi], want[lo:hi], t_out[lo:hi])


@pytest.mark.parametrize("new", [1, 100])
def test_a_block_that_does_not_exist_reads_as_zeros(new):
    lens = [200]
    k, v, table = _paged.make_paged(lens, 16, 2, 64, torch.bfloat16, "nhd", 1)
    q = torch.randn(new, 4, 64, device="cuda").to(torch.bfloat16)
    bad = table.clone()
    bad[0, 3], bad[0, 7] = -1, k.shape[0]
    out, _ = fa.fa_paged_fwd(q, k, v, bad, i32([0, new]), i32(lens), max_new=new)
    st, word = fa.device_status()
    assert st == fa.FA_ERR_PAGED_RANGE and (word >> 8) & 0xFF == 45
    for b in (3, 7):
        k[table[0, b].item()], v[table[0, b].item()] = 0.0, 0.0
    want, _, t_out, _ = _paged.attend64(q, k, v, table, [0, new], lens, causal=True, window=None, scale=0.125)
    close(out, want, t_out)


def test_pages_outside_the_window_are_not_looked_up():
    """A serving loop may have given back the blocks that its window has left."""
    for new in (1, 90):
        lens = [1000]
        k, v, table = _paged.make_paged(lens, 16, 1, 64, torch.bfloat16, "nhd", 1)
        first = 1000 - new - 64 + 1
        gone = first // 16
        q = torch.randn(new, 2, 64, device="cuda").to(torch.bfloat16)
        want, _, t_out, _ = _paged.attend64(q, k, v, table, [0, new], lens, causal=True, window=64, scale=0.125)
        for b in range(gone):
            k[table[0, b].item()] = v[table[0, b].item()] = float("nan")
        table[0, :gone] = -1
        out, _ = fa.fa_paged_fwd(q, k, v, table, i32([0, new]), i32(lens), max_new=new, window=64)
        close(out, want, t_out)


@pytest.mark.parametrize("new", [1, 120])
def test_on_a_stream_of_its_own(new):
    s = torch.cuda.Stream()
    k, v, table = _paged.make_paged([400], 16, 1, 64, torch.bfloat16, "nhd", 1)
    q = torch.randn(new, 2, 64, device="cuda").to(torch.bfloat16)
    torch.cuda.synchronize()
    out, lse = fa.fa_paged_fwd(q, k, v, table, i32([0, new]), i32([400]), max_new=new)
    cu, ln = i32([0, new]), i32([400])
    torch.cuda.synchronize()
    out2, lse2 = fa.fa_paged_fwd(q, k, v, table, cu, ln, max_new=new, stream=s)
    s.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 elements: its last blocks are written and read."""
    page, Hkv, d = 16, 8, 128
    blocks = (1 << 32) // (page * Hkv * d) + 40
    k_cache = torch.empty((blocks, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    v_cache = torch.empty_like(k_cache)
    n = 70
    ids = torch.arange(blocks - 5, blocks, device="cuda")
    t = torch.arange(n, device="cuda")
    slots = ids[t // page] * page + t % page
    q, k, v = (torch.randn(n, h, d, device="cuda").to(torch.bfloat16) for h in (16, Hkv, Hkv))
    inv, axis = spec(d, 1)
    fa.fa_rope_append(None, k, v, t.int(), fa.RopeTable(inv), k_cache, v_cache, slots)
    want = _paged.rope64(k, t[None], inv, axis, False)
    close(k_cache[ids].reshape(-1, Hkv, d)[:n], want, _paged.rope_tolerance(k, want, d // 2, False))
    assert torch.equal(v_cache[ids].reshape(-1, Hkv, d)[:n], v)
    table = torch.full((1, 5), 0, dtype=torch.int32, device="cuda")
    table[0] = ids.int()
    v_cache[ids[-1], n % page:] = float("nan")   # behind the last key
    for new in (1, 60):
        out, _ = fa.fa_paged_fwd(q[:new], k_cache, v_cache, table, i32([0, new]), i32([n]), max_new=new)
        want, _, t_out, _ = _paged.attend64(q[:new], k_cache[ids], v_cache[ids], torch.arange(5, device="cuda")[None], [0, new], [n],
                                            causal=True, window=None, scale=d ** -0.5)
        close(out, want, t_out)


def test_strides_of_axes_of_one_entry():
    """One KV head, or one block, in a tensor whose stride there is anything."""
    base = torch.randn(4, 16, 3, 64, device="cuda").to(torch.bfloat16)
    k = torch.as_strided(base, (4, 16, 1, 64), (16 * 192, 192, 7, 1), 64)
    v = torch.as_strided(base, (4, 16, 1, 64), (16 * 192, 192, 7, 1), 128)
    table = i32([[2, 0, 3, 1]])
    for new in (1, 40):
        q = torch.randn(new, 2, 64, device="cuda").to(torch.bfloat16)
        out, _ = fa.fa_paged_fwd(q, k, v, table, i32([0, new]), i32([60]), max_new=new)
        want, _, t_out, _ = _paged.attend64(q, k, v, table, [0, new], [60], causal=True, window=None, scale=0.125)
        close(out, want, t_out)


def mixed_problem(seed, d=128):
    lens = [300, 1, 900, 64, 2000, 17]
    news = [1, 1, 300, 2, 70, 0]
    k, v, table = _paged.make_paged(lens, 16, 2, d, torch.bfloat16, "nhd", seed)
    q = torch.randn(sum(news), 8, d, device="cuda").to(torch.bfloat16)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    return (q, k, v, table, i32(cu), i32(lens)), dict(max_new=300)


def test_two_calls_at_once_and_one_after_the_other():
    """Calls on two streams, each with its own workspace, and calls in one stream that share one."""
    args, kw = zip(*(mixed_problem(s) for s in (1, 2)))
    alone = [fa.fa_paged_fwd(*a, **w) for a, w in zip(args, kw)]
    need = fa.paged_workspace_bytes(8, 2, 128)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(a[0]) for _ in range(20)] for a in args]
    torch.cuda.synchronize()
    for i in range(20):
        for x in range(2):
            fa.fa_paged_fwd(*args[x], **kw[x], out=outs[x][i], return_lse=False, workspace=ws[x], stream=streams[x])
    torch.cuda.synchronize()
    for x in range(2):
        assert all(torch.equal(o, alone[x][0]) for o in outs[x])
    for i in range(20):
        fa.fa_paged_fwd(*args[i % 2], **kw[i % 2], out=outs[i % 2][i], return_lse=False, workspace=ws[0])
    torch.cuda.synchronize()
    assert all(torch.equal(outs[i % 2][i], alone[i % 2][0]) for i in range(20))


def test_mixed_call_captured_and_replayed():
    """Chunks and decoding requests in one captured call, replayed on new values and new lengths."""
    args, kw = mixed_problem(3)
    q, k, v, table, cu, lens = args
    ws = torch.empty(fa.paged_workspace_bytes(8, 2, 128), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(8, q.shape[0], device="cuda")
    fa.fa_paged_fwd(*args, **kw, out=out, lse=lse, workspace=ws)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        fa.fa_paged_fwd(*args, **kw, out=out, lse=lse, workspace=ws)
    for shift in (0, 1, 40):
        q.normal_()
        lens.copy_(i32([300 - shift, 1, 900 - shift, 64 - shift, 2000 - shift, 17]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = fa.fa_paged_fwd(*args, **kw)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_the_same_block_twice():
    """Two requests that share their first blocks (a common prefix), and one that names a block twice."""
    k, v, table = _paged.make_paged([200], 16, 2, 64, torch.bfloat16, "nhd", 5)
    table = torch.cat([table, table, table])
    table[2, 3] = table[2, 1]
    lens, news = [200, 130, 200], [1, 60, 3]
    q = torch.randn(sum(news), 4, 64, device="cuda").to(torch.bfloat16)
    cu = [0, 1, 61, 64]
    out, _ = fa.fa_paged_fwd(q, k, v, table, i32(cu), i32(lens), max_new=60)
    want, _, t_out, _ = _paged.attend64(q, k, v, table, cu, lens, causal=True, window=None, scale=0.125)
    close(out, want, t_out)


# ------------------------------------------------------------------------------- together

def test_serving_loop_matches_dense_attention():
    """Prompts in chunks, decoding, finished requests, reused blocks: every step's attention against the
    whole sequences, rotated and attended in 64 bits."""
    torch.manual_seed(11)
    Hq, Hkv, d, page, R = 8, 2, 64, 16, 5
    inv, axis = spec(d, 1)
    table = fa.RopeTable(inv, axis=axis)
    kv = fa.PagedKV(R, 40, page, Hkv, d, max_blocks=20, layout="hnd")
    hist = [[] for _ in range(R)]
    steps = [[30, 0, 100, 7, 0], [1, 64, 50, 1, 0], [1, 1, 1, 1, 33], "2,3", [1, 1, 20, 0, 1], [1, 1, 1, 90, 1]]
    for step in steps:
        if step == "2,3":
            kv.release(i32([0, 0, 1, 1, 0]))
            hist[2], hist[3] = [], []
            continue
        T = sum(step) + 2
        q, k, v = (torch.randn(T, h, d, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
        kv.reserve(i32(step), T)
        q_rot = torch.full((T, Hq, d), 0.0, device="cuda", dtype=torch.bfloat16)
        kv.append(q, k, v, table, q_out=q_rot)
        out, lse = kv.attend(q_rot, max_new=max(step))
        at = 0
        for r, n in enumerate(step):
            if n:
                hist[r].append((k[at:at + n], v[at:at + n]))
                kk, vv = torch.cat([x[0] for x in hist[r]]), torch.cat([x[1] for x in hist[r]])
                L = kk.shape[0]
                kk = _paged.rope64(kk, torch.arange(L, device="cuda")[None], inv, axis, False).to(torch.bfloat16)
                qq = _paged.rope64(q[at:at + n], torch.arange(L - n, L, device="cuda")[None], inv, axis, False)
                # the kernel attends the rotated rows as rounded: the same rows here, but for ties
                assert (q_rot[at:at + n].double() - qq).abs().max() <= 2.0 ** -7 * 8
                one = torch.arange(blocks := -(-L // page), device="cuda", dtype=torch.int32)[None]
                pad = blocks * page - L
                kc = torch.cat([kk, kk.new_zeros(pad, Hkv, d)]).view(blocks, page, Hkv, d)
                vc = torch.cat([vv, vv.new_zeros(pad, Hkv, d)]).view(blocks, page, Hkv, d)
                got_k = kv.k_cache[kv.block_table[r, :blocks].long()].reshape(-1, Hkv, d)[:L]
                assert (got_k.double() - kk.double()).abs().max() <= 2.0 ** -7 * 8   # a step of the largest value
                want, z, t_out, t_lse = _paged.attend64(q_rot[at:at + n], kv.k_cache, kv.v_cache, kv.block_table[r:r + 1], [0, n], [L],
                                                        causal=True, window=None, scale=d ** -0.5)
                close(out[at:at + n], want, t_out)
                close(lse[:, at:at + n], z, t_lse)
                assert torch.equal(kv.v_cache[kv.block_table[r, :blocks].long()].reshape(-1, Hkv, d)[:L], vv)
                del one, kc, vc
            at += n
        assert kv.seq_lens.tolist() == [sum(x[0].shape[0] for x in h) for h in hist]
    held = sum(-(-n // page) for n in kv.seq_lens.tolist())
    assert kv.free_count.item() == 40 - held
    owned = [b for r in range(R) for b in kv.block_table[r, :-(-kv.seq_lens[r].item() // page)].tolist()]
    assert sorted(owned + kv.free_blocks[:40 - held].tolist()) == list(range(40))


def test_captured_decoding_steps():
    """One decoding step captured into a graph and replayed: the same bits as the steps run eagerly."""
    torch.manual_seed(12)
    Hq, Hkv, d, page, R = 8, 2, 128, 16, 6
    table = fa.RopeTable(spec(d, 1)[0])
    prompt = [3, 70, 0, 16, 200, 1]
    one = i32([1, 1, 0, 1, 1, 1])
    T = 8

    def start():
        torch.manual_seed(13)
        kv = fa.PagedKV(R, 64, page, Hkv, d, max_blocks=32)
        n = sum(prompt)
        k, v = (torch.randn(n, Hkv, d, device="cuda").to(torch.bfloat16) for _ in range(2))
        kv.reserve(i32(prompt), n)
        kv.append(None, k, v, table)
        return kv

    q, k, v = (torch.zeros(T, h, d, device="cuda", dtype=torch.bfloat16) for h in (Hq, Hkv, Hkv))
    ws = torch.empty(fa.paged_workspace_bytes(Hq, Hkv, d), dtype=torch.uint8, device="cuda")

    def step(kv, q_rot, out, lse):
        kv.reserve(one, T)
        kv.append(q, k, v, table, q_out=q_rot)
        kv.attend(q_rot, max_new=1, out=out, lse=lse, workspace=ws)

    def inputs(i):
        g = torch.Generator(device="cuda")
        g.manual_seed(100 + i)
        for x in (q, k, v):
            x.copy_(torch.empty(x.shape, device="cuda").normal_(generator=g))

    bufs = [(torch.zeros(T, Hq, d, device="cuda", dtype=torch.bfloat16), torch.zeros(T, Hq, d, device="cuda", dtype=torch.bfloat16),
             torch.zeros(Hq, T, device="cuda")) for _ in range(2)]
    eager, graphed = start(), start()
    eager_out = []
    for i in range(20):
        inputs(i)
        step(eager, *bufs[0])
        eager_out.append((bufs[0][1].clone(), bufs[0][2].clone()))
    side = torch.cuda.Stream()
    graphed.reserve(i32([0] * R), T)   # makes the step's buffers; takes nothing
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        step(graphed, *bufs[1])
    for i in range(20):
        inputs(i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs[1][1], eager_out[i][0]) and torch.equal(bufs[1][2], eager_out[i][1])
    assert graphed.seq_lens.tolist() == eager.seq_lens.tolist() == [p + 20 * o for p, o in zip(prompt, one.tolist())]


# ------------------------------------------------------------------------------- shared rows

@pytest.mark.parametrize("T", [1, 70, 3001])
def test_positions_shared_by_all_axes(T):
    """Text in a model of three axes: one row of positions, expanded.  Behind it lies something else."""
    torch.manual_seed(T)
    inv, axis = spec(64, 3)
    table = fa.RopeTable(inv, axis=axis)
    memory = torch.full((4 * T,), 77777, dtype=torch.int32, device="cuda")
    memory[:T] = torch.arange(T, device="cuda") + 1000
    shared = memory[:T][None].expand(3, T)
    q, k, v = (torch.randn(T, h, 64, device="cuda").to(torch.bfloat16) for h in (4, 2, 2))
    got = fa.fa_rope(q, shared, table, k=k)
    for g, x in zip(got, (q, k)):
        want = _paged.rope64(x, shared, inv, axis, False)
        close(g, want, _paged.rope_tolerance(x, want, 32, False))
    k_cache, v_cache, _ = _paged.make_paged([T], 16, 2, 64, torch.bfloat16, "nhd", 3, poison=False)
    q_out = fa.fa_rope_append(q, k, v, shared, table, k_cache, v_cache, torch.arange(T, device="cuda"))
    assert torch.equal(q_out, got[0]) and torch.equal(k_cache.reshape(-1, 2, 64)[:T], got[1])


@pytest.mark.parametrize("new", [1, 90])
def test_a_table_shared_by_all_requests(new):
    """Samples of one prompt: one row of blocks, expanded; what only reads it takes it, what writes it does not."""
    k, v, table = _paged.make_paged([200], 16, 2, 64, torch.bfloat16, "nhd", 5)
    memory = torch.full((4, table.shape[1]), -3, dtype=torch.int32, device="cuda")
    memory[0] = table[0]
    shared = memory[:1].expand(3, -1)
    lens, news = [200, 150, 200], [new, 1, new]
    cu = [0, new, new + 1, 2 * new + 1]
    q = torch.randn(cu[-1], 4, 64, device="cuda").to(torch.bfloat16)
    out, lse = fa.fa_paged_fwd(q, k, v, shared, i32(cu), i32(lens), max_new=max(news))
    want, z, t_out, t_lse = _paged.attend64(q, k, v, table.expand(3, -1), cu, lens, causal=True, window=None, scale=0.125)
    close(out, want, t_out)
    close(lse, z, t_lse)
    stack = torch.full((40,), -9, dtype=torch.int32, device="cuda")
    left, count = fa.fa_kv_release(i32([33, 20, 5]), i32([1, 0, 1]), shared, stack, i32([2]), page_size=16)
    assert left.tolist() == [0, 20, 0] and count.tolist() == [6]
    assert stack[2:6].tolist() == memory[0, :3].tolist() + memory[0, :1].tolist() and bool((stack[6:] == -9).all())
    before = memory.clone()
    with pytest.raises(ValueError, match="overlap"):
        fa.fa_kv_reserve(i32([16, 16, 16]), i32([1, 1, 1]), shared, i32([0, 1, 2, 3]), i32([4]), page_size=16, num_tokens=3)
    assert torch.equal(memory, before)


# ------------------------------------------------------------------------------- steps of many tokens

def refused(ctx, new, table, stack, count, site, T, page, in_place):
    """The step is refused whole: reported, and nothing is taken."""
    before, ctx_d, count_d = table.clone(), i32(ctx), i32([count])
    kw = dict(seq_lens=ctx_d, free_count_out=count_d) if in_place else {}
    cu, lens, pos, slots, cnt = fa.fa_kv_reserve(ctx_d, i32(new), table, stack, count_d, page_size=page, num_tokens=T, **kw)
    st, word = fa.device_status()
    assert st == fa.FA_ERR_PAGED_RANGE and (word >> 8) & 0xFF == site
    assert not bool(cu.any()) and lens.tolist() == ctx and cnt.tolist() == [count]
    assert bool((slots == -1).all()) and not bool(pos.any()) and torch.equal(table, before)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("ctx,new,count,site", [
    ([3, -1], [9000, 9000], 6000, 41), ([3, 20], [15000, -2], 6000, 41), ([3, 39990], [9000, 9000], 6000, 41),
    ([3, 20], [15000, 10000], 6000, 42), ([3, 20], [30000, 1], 6000, 42),
    ([0, 0], [9000, 9000], 1000, 43), ([0, 0], [9000, 9000], 6001, 43), ([0, 0], [9000, 9000], -1, 43)])
def test_reserve_of_many_tokens_refuses_a_whole_step(ctx, new, count, site, in_place):
    table = torch.full((2, 2500), 7, dtype=torch.int32, device="cuda")
    refused(ctx, new, table, torch.arange(6000, dtype=torch.int32, device="cuda"), count, site, 20000, 16, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("R,ctx,new", [(1024, 0, 1 << 22), (1024, 5, 1 << 22), (1024, 0, (1 << 22) + 1), (2048, 0, 1 << 22), (512, 0, 1 << 23),
                                       (1025, 0, 1 << 22)])
def test_reserve_refuses_sums_beyond_32_bits(R, ctx, new, in_place):
    """The new tokens of many requests sum to a multiple of 2^32, or a little more: not a step of few tokens."""
    table = torch.full((R, 3), 7, dtype=torch.int32, device="cuda")
    refused([ctx] * R, [new] * R, table, torch.arange(8192, dtype=torch.int32, device="cuda"), 8192, 42, new, 1 << 22, in_place)


def test_reserve_of_millions_of_tokens():
    """A step large enough for the sums to be made apart, that fits: against the formulas on the GPU."""
    page, ctx, new = 128, [1000, 0, 77, 2_000_000], [1 << 21, 0, 5, (1 << 21) + 300]
    T = sum(new) + 9
    held, want = ([_paged.blocks_of(x, page) for x in xs] for xs in (ctx, [c + n for c, n in zip(ctx, new)]))
    width = max(want)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    ids = torch.randperm(sum(want) + 3, device="cuda", generator=g).int()
    table = torch.full((4, width), -7, dtype=torch.int32, device="cuda")
    at = 0
    for r in range(4):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    stack, count = torch.cat([ids[at:], torch.full((at,), -9, dtype=torch.int32, device="cuda")]), ids.numel() - at
    ref = table.clone()
    top = count
    for r in range(4):
        n = want[r] - held[r]
        ref[r, held[r]:want[r]] = stack[top - n:top].flip(0)
        top -= n
    cu, lens, pos, slots, cnt = fa.fa_kv_reserve(i32(ctx), i32(new), table, stack, i32([count]), page_size=page, num_tokens=T)
    assert torch.equal(table, ref) and cnt.tolist() == [top] and lens.tolist() == [c + n for c, n in zip(ctx, new)]
    starts = [sum(new[:r]) for r in range(5)]
    assert cu.tolist() == starts
    for r in range(4):
        x = torch.arange(ctx[r], ctx[r] + new[r], device="cuda")
        assert torch.equal(pos[starts[r]:starts[r + 1]].long(), x)
        assert torch.equal(slots[starts[r]:starts[r + 1]], ref[r].long()[x // page] * page + x % page)
    assert bool((slots[starts[4]:] == -1).all()) and not bool(pos[starts[4]:].any())


# ------------------------------------------------------------------------------- windows without a limit

@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 200, 1 << 30, 400])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_window_of_any_size_over_fewer_keys_than_tokens(d, window):
    """Positions below 0 less a window near 2^31: rows that see keys keep them."""
    attend([100, 300, 0, 7], [300, 300, 200, 20], Hq=4, Hkv=2, d=d, page=16, window=window, seed=d)
    attend([3, 300, 0, 1], [5, 1, 2, 1], Hq=4, Hkv=2, d=d, page=16, window=window, seed=d)


# ------------------------------------------------------------------------------- a step's rows

def test_rows_of_steps_kept_by_the_caller():
    """Two steps of different sizes, the first one's rows given: they outlive the second step; rows of the cache
    itself, captured with append and attend behind an eager reserve, stay where they are."""
    torch.manual_seed(21)
    table = fa.RopeTable(spec(64, 1)[0])
    kv = fa.PagedKV(2, 64, 16, 2, 64, max_blocks=32)
    mine = torch.full((70,), -5, dtype=torch.int32, device="cuda"), torch.full((70,), -5, dtype=torch.int64, device="cuda")
    got = kv.reserve(i32([40, 30]), 70, positions=mine[0], slots=mine[1])
    assert got[0] is mine[0] and got[1] is mine[1]
    kept = mine[1].clone()
    q, k, v = (torch.randn(70, h, 64, device="cuda").to(torch.bfloat16) for h in (4, 2, 2))
    kv.append(None, k, v, table)
    kv.reserve(i32([1, 1]), 5)
    assert torch.equal(mine[1], kept) and mine[0].tolist() == list(range(40)) + list(range(30))
    q5, k5, v5 = (torch.randn(5, h, 64, device="cuda").to(torch.bfloat16) for h in (4, 2, 2))
    out, q_rot = torch.zeros_like(q5), torch.zeros_like(q5)
    ws = torch.empty(fa.paged_workspace_bytes(4, 2, 64), dtype=torch.uint8, device="cuda")

    def rest():
        kv.append(q5, k5, v5, table, q_out=q_rot)
        kv.attend(q_rot, max_new=1, out=out, return_lse=False, workspace=ws)
    rest()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        rest()
    for n in (1, 300, 9, 64):   # steps of other sizes, with no tokens, between
        kv.reserve(i32([0, 0]), n)
    for x in (q5, k5, v5):
        x.normal_()
    kv.reserve(i32([1, 1]), 5)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone()
    lens = kv.seq_lens.tolist()
    assert lens == [42, 32]
    want, _, t_out, _ = _paged.attend64(q_rot, kv.k_cache, kv.v_cache, kv.block_table, [0, 1, 2], lens, causal=True, window=None, scale=0.125)
    close(got[:2], want[:2], t_out[:2])
    at = kv.slots[:2]
    assert torch.equal(kv.v_cache.reshape(-1, 2, 64)[at], v5[:2])


# ------------------------------------------------------------------------------- NaN

@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,news,bad", [
    ([9000], [1], [0]), ([9000], [3], [1]), ([9000, 40], [2, 1], [1, 2]), ([40, 17], [1, 1], [1]),    # few rows, cut or whole
    ([9000], [200], [0, 100, 199]), ([9000, 300, 20], [150, 130, 1], [3, 149, 170, 280]), ([40, 60], [40, 60], [5, 41])])
def test_a_row_of_nan_stays_nan(lens, news, bad, d):
    """q of NaN: O and LSE are NaN in that row, whether or not its unit is cut into pieces; the others are right."""
    k, v, table = _paged.make_paged(lens, 16, 2, d, torch.bfloat16, "nhd", d)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    q = torch.randn(cu[-1], 8, d, device="cuda").to(torch.bfloat16)
    clean = q.clone()
    q[bad] = float("nan")
    out, lse = fa.fa_paged_fwd(q, k, v, table, i32(cu), i32(lens), max_new=max(news))
    assert bool(out[bad].isnan().all()) and bool(lse[:, bad].isnan().all())
    rest = [t for t in range(cu[-1]) if t not in bad]
    want, z, t_out, t_lse = _paged.attend64(clean, k, v, table, cu, lens, causal=True, window=None, scale=d ** -0.5)
    close(out[rest], want[rest], t_out[rest])
    close(lse[:, rest], z[:, rest], t_lse[:, rest])


@pytest.mark.parametrize("new", [1, 200])
def test_one_nan_key_is_not_lost(new):
    """A key of NaN in the middle of a long request: every row that sees it is NaN (d = 128: each weight is an exponential)."""
    k, v, table = _paged.make_paged([9000], 16, 2, 128, torch.bfloat16, "nhd", 1)
    k[table[0, 100].item(), 3, 0] = float("nan")
    q = torch.randn(new, 8, 128, device="cuda").to(torch.bfloat16)
    out, lse = fa.fa_paged_fwd(q, k, v, table, i32([0, new]), i32([9000]), max_new=new)
    assert bool(out[:, :4].isnan().all()) and bool(lse[:4].isnan().all())
    assert not bool(out[:, 4:].isnan().any()) and not bool(lse[4:].isnan().any())


# ------------------------------------------------------------------------------- every key once

def counted(lens, news, *, Hq, Hkv, d, page, dtype, window=None, max_new=None):
    """q = 0: every visible key has the weight 1, so LSE = ln(visible keys), and with V one-hot (the column
    turns with every 8 keys and every head) O counts the keys of each column: a key left out, or taken
    twice, shows in a request of tens of thousands.

    Tolerances.  exp2(0) is 1 (its polynomial form, in the tile kernel at d = 32 and 64, is off by up to 2^-13.5),
    and sums of ones are exact.  A piece's LSE: log2f (1 ulp), two products with rounded factors, four steps
    of 2^-23 ln(keys) in all with the final sum m + logf.  The weights of up to `parts` pieces: __expf of
    an argument of at most 8 (12 ulp) of those LSEs, 2^-19 in all; their sum adds 2^-24 each.  A unit has no more
    pieces than CTAs of the tile kernel (148) or sqrt(8 steps) + 2 of the few-rows kernel, steps of 16
    keys at least.  O is rounded once more to its type."""
    k, v, table = _paged.make_paged(lens, page, Hkv, d, dtype, "nhd", 31)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    head = torch.arange(Hkv, device="cuda")
    want = torch.zeros(cu[-1], Hq, d, dtype=torch.float64, device="cuda")
    z = torch.zeros(Hq, cu[-1], dtype=torch.float64, device="cuda")
    seen = torch.ones(cu[-1], dtype=torch.float64, device="cuda")
    for r, L in enumerate(lens):
        j = torch.arange(L, device="cuda")
        hot = torch.nn.functional.one_hot((j[:, None] // 8 + 5 * head) % d, d)
        v[table[r].long()[j // page], j % page] = hot.to(dtype)
        upto = torch.cat([torch.zeros_like(hot[:1]), hot.cumsum(0)])              # [L + 1, Hkv, d]
        last = torch.arange(L - news[r], L, device="cuda")
        first = (last - window + 1).clamp(min=0) if window else torch.zeros_like(last)
        n = (last - first + 1).double()
        rows = slice(cu[r], cu[r + 1])
        want[rows] = ((upto[last + 1] - upto[first]).double() / n[:, None, None]).repeat_interleave(Hq // Hkv, 1)
        z[:, rows] = n.log()
        seen[rows] = n
    polynomial = 2.0 ** -13.5 if d in (32, 64) and (max(news) if max_new is None else max_new) * (Hq // Hkv) > 16 else 0.0
    parts = max(148, math.sqrt(8 * max(lens) / 16) + 2)
    rel = polynomial + 2.0 ** -19 + parts * 2.0 ** -24
    t_lse = rel + 4 * 2.0 ** -23 * z.abs()
    assert bool((t_lse < torch.log(seen / (seen - 1).clamp(min=0.5))).all())      # a key more or less is outside
    q = torch.zeros(cu[-1], Hq, d, device="cuda", dtype=dtype)
    out, lse = fa.fa_paged_fwd(q, k, v, table, i32(cu), i32(lens), max_new=max(news) if max_new is None else max_new, window=window)
    close(lse, z, t_lse)
    close(out, want, (_paged.HALF[dtype] + 2 * rel + 2.0 ** -21) * want + 2.0 ** -25)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,news,Hq,Hkv,d,page", [
    ([40000], [1], 8, 1, 128, 64), ([40000], [1], 8, 8, 64, 16), ([30000], [3], 8, 2, 256, 16), ([40000], [1], 12, 1, 128, 16),
    ([20000, 9000, 300, 1], [1, 1, 1, 1], 16, 4, 128, 16), ([25000, 70], [2, 2], 4, 2, 80, 100), ([40000], [1], 4, 1, 32, 3),
    ([30000], [200], 8, 1, 128, 64), ([20000], [130], 4, 4, 192, 16), ([9000, 40, 5000], [700, 1, 90], 8, 2, 128, 16),
    ([30000], [300], 4, 1, 256, 24), ([4000, 600], [140, 600], 4, 2, 64, 16), ([3000], [200], 3, 1, 32, 8),
    ([10000, 17], [40, 17], 6, 2, 96, 32), ([12000], [700], 2, 2, 80, 100), ([20000], [20], 40, 1, 128, 16)])
def test_every_key_once(lens, news, Hq, Hkv, d, page, dtype):
    counted(lens, news, Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype)


@pytest.mark.parametrize("window", [5, 100, 1000, 9000])
def test_every_key_of_a_window_once(window):
    counted([30000, 500], [1, 1], Hq=8, Hkv=2, d=128, page=16, dtype=torch.float16, window=window)
    counted([30000, 500, 20000], [300, 1, 7], Hq=8, Hkv=2, d=128, page=16, dtype=torch.float16, window=window)


def test_every_key_of_many_requests_once():
    rng = random.Random(41)
    lens = [rng.choice([1, 31, 32, 33, rng.randint(1, 9000)]) for _ in range(120)]
    for top in (1, 60):
        news = [min(n, rng.choice([1, 1, rng.randint(1, top)])) for n in lens]
        counted(lens, news, Hq=4, Hkv=2, d=128, page=16, dtype=torch.float16, max_new=top)


# ------------------------------------------------------------------------------- calls at the edges

@pytest.mark.parametrize("max_new", [1, 5, 200])
def test_a_step_without_tokens(max_new):
    """Every request idle: nothing is written, nothing is reported."""
    k, v, table = _paged.make_paged([300, 0, 20], 16, 2, 128, torch.bfloat16, "nhd", 2)
    q = torch.randn(7, 8, 128, device="cuda").to(torch.bfloat16)
    out, lse = torch.full_like(q, 3.0), torch.full((8, 7), 3.0, device="cuda")
    fa.fa_paged_fwd(q, k, v, table, i32([0, 0, 0, 0]), i32([300, 0, 20]), max_new=max_new, out=out, lse=lse)
    torch.cuda.synchronize()
    assert bool((out == 3.0).all()) and bool((lse == 3.0).all())


@pytest.mark.parametrize("news", [[1, 1], [1, 90]])
def test_a_table_without_blocks(news):
    """max_blocks = 0: requests of no keys alone; their rows see nothing."""
    k = torch.randn(4, 16, 2, 64, device="cuda").to(torch.bfloat16)
    q = torch.randn(sum(news), 4, 64, device="cuda").to(torch.bfloat16)
    table = torch.zeros((2, 0), dtype=torch.int32, device="cuda")
    out, lse = fa.fa_paged_fwd(q, k, k.clone(), table, i32([0, news[0], sum(news)]), i32([0, 0]), max_new=max(news))
    assert not bool(out.any()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("new", [1, 100])
def test_one_page_for_all(new):
    """A page longer than the request: a cache that is one array a request."""
    attend([30000, 17], [new, 1], Hq=4, Hkv=2, d=64, page=40000, seed=new)


def test_layers_that_share_tables():
    """Two layers over one set of tables: one reserve, one release, each its own keys and values."""
    torch.manual_seed(31)
    inv, axis = spec(64, 1)
    rope = fa.RopeTable(inv)
    first = fa.PagedKV(3, 20, 16, 2, 64, max_blocks=10)
    layers = [first, fa.PagedKV(3, 20, 16, 2, 64, tables=first, layout="hnd"), fa.PagedKV(3, 20, 16, 1, 128, tables=first, dtype=torch.float16)]
    kept = [[], [], []]
    lens = [0, 0, 0]
    for step in ([40, 0, 9], [1, 30, 1], [1, 1, 1]):
        T = sum(step)
        first.reserve(i32(step), T)
        lens = [a + b for a, b in zip(lens, step)]
        cu = [0, step[0], step[0] + step[1], T]
        for n, kv in enumerate(layers):
            dt = kv.k_cache.dtype
            q, k, v = (torch.randn(T, h, kv.d, device="cuda").to(dt) for h in (4, kv.Hkv, kv.Hkv))
            kept[n].append((step, v))
            table = rope if kv.d == 64 else fa.RopeTable(spec(128, 1)[0])
            rows = kv.append(q, k, v, table)
            out, lse = kv.attend(rows, max_new=max(step))
            want, z, t_out, t_lse = _paged.attend64(rows, kv.k_cache, kv.v_cache, first.block_table, cu, lens, causal=True, window=None,
                                                    scale=kv.d ** -0.5)
            close(out, want, t_out)
            close(lse, z, t_lse)
    for n, kv in enumerate(layers):   # each layer holds its own values, request by request
        for r in range(3):
            mine = torch.cat([v[sum(s[:r]):sum(s[:r + 1])] for s, v in kept[n]])
            pages = first.block_table[r, :_paged.blocks_of(lens[r], 16)].long()
            assert torch.equal(kv.v_cache[pages].reshape(-1, kv.Hkv, kv.d)[:lens[r]], mine)
    with pytest.raises(ValueError):
        layers[1].reserve(i32([1, 1, 1]), 3)
    with pytest.raises(ValueError):
        layers[1].release(i32([1, 0, 0]))
    first.release(i32([1, 1, 1]))
    assert first.free_count.item() == 20 and sorted(first.free_blocks.tolist()) == list(range(20))


@pytest.mark.parametrize("T", [500, 40000])
def test_reserve_and_release_captured(T):
    """Both updated in place in one graph, the many-token path among them: replays give what eager steps give."""
    page, R = 16, 37
    rng = random.Random(T)
    new = [rng.randint(0, T // R) for _ in range(R)]
    done = [rng.choice([0, 0, 1]) for _ in range(R)]

    def start():
        return dict(lens=torch.zeros(R, dtype=torch.int32, device="cuda"), table=torch.full((R, 4 * T // R // page + 8), -7, dtype=torch.int32, device="cuda"),
                    stack=torch.arange(5 * T // page, dtype=torch.int32, device="cuda"), count=i32([5 * T // page]),
                    cu=torch.zeros(R + 1, dtype=torch.int32, device="cuda"), pos=torch.zeros(T, dtype=torch.int32, device="cuda"),
                    slots=torch.zeros(T, dtype=torch.int64, device="cuda"))
    n, d = i32(new), i32(done)

    def step(s):
        fa.fa_kv_reserve(s["lens"], n, s["table"], s["stack"], s["count"], page_size=page, cu_seqlens=s["cu"], seq_lens=s["lens"], positions=s["pos"],
                         slots=s["slots"], free_count_out=s["count"])
        fa.fa_kv_release(s["lens"], d, s["table"], s["stack"], s["count"], page_size=page, lens_out=s["lens"], free_count_out=s["count"])
    eager, graphed = start(), start()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        step(graphed)
    for _ in range(3):
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(eager[x], graphed[x]) for x in eager)
    assert eager["lens"].tolist() == [0 if f else 3 * x for f, x in zip(done, new)]
