"""Argument checks of the paged-cache entry points, without a GPU: refusals come before any CUDA call
(fake pointers are never dereferenced), and the binding's own checks of shapes and types."""
import ctypes

import pytest

import exact_attention_146_b200 as fa
from exact_attention_146_b200 import build as fa_build
from exact_attention_146_b200 import paged

A = [(i + 1) << 33 for i in range(20)]   # arrays far apart
NO_DEVICE = (fa.FA_ERR_UNSUPPORTED_DEVICE, fa.FA_ERR_NOT_DEVICE_MEMORY)


@pytest.fixture(scope="module")
def L():
    fa_build.build()
    return fa.lib()


def reserve(L, ctx=A[0], new=A[1], R=4, table=A[2], stride=8, max_blocks=8, free=A[3], count=A[4], blocks=100, page=16, T=9, cu=A[5],
            lens=A[6], pos=A[7], slots=A[8], out=A[9]):
    return L.fa_kv_reserve(ctx, new, R, table, stride, max_blocks, free, count, blocks, page, T, cu, lens, pos, slots, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), 1), (dict(T=-1), 1), (dict(T=(1 << 30) + 1), 1), (dict(blocks=(1 << 30) + 1), 1), (dict(page=0), 1), (dict(blocks=-1), 1), (dict(max_blocks=-1), 1), (dict(stride=7), 1),
    (dict(max_blocks=1 << 28, stride=1 << 28), 1), (dict(cu=None), 1), (dict(count=None), 1), (dict(out=None), 1), (dict(ctx=None), 1),
    (dict(new=None), 1), (dict(lens=None), 1), (dict(table=None), 1), (dict(free=None), 1), (dict(pos=None), 1), (dict(slots=None), 1),
    (dict(slots=A[8] + 4), 3), (dict(pos=A[7] + 2), 3), (dict(ctx=A[0] + 1), 3), (dict(lens=A[1]), 8), (dict(lens=A[0] + 4), 8),
    (dict(pos=A[8] + 8), 8), (dict(cu=A[2] + 4 * 31), 8), (dict(out=A[3]), 8), (dict(table=A[3]), 8)])
def test_reserve_refusals(L, kw, code):
    assert reserve(L, **kw) == code


def test_reserve_accepts(L):
    assert reserve(L) in NO_DEVICE
    assert reserve(L, lens=A[0], out=A[4]) in NO_DEVICE                      # updated in place
    assert reserve(L, R=0, ctx=None, new=None, lens=None, table=None) in NO_DEVICE


def release(L, lens=A[0], done=A[1], R=4, table=A[2], stride=8, max_blocks=8, free=A[3], count=A[4], blocks=100, page=16, lens_out=A[5],
            out=A[6]):
    return L.fa_kv_release(lens, done, R, table, stride, max_blocks, free, count, blocks, page, lens_out, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), 1), (dict(page=0), 1), (dict(stride=7), 1), (dict(done=None), 1), (dict(lens_out=None), 1), (dict(count=None), 1),
    (dict(free=None), 1), (dict(free=A[3] + 2), 3), (dict(lens_out=A[1]), 8), (dict(free=A[2]), 8), (dict(out=A[0]), 8)])
def test_release_refusals(L, kw, code):
    assert release(L, **kw) == code


def test_release_accepts(L):
    assert release(L) in NO_DEVICE and release(L, lens_out=A[0], out=A[4]) in NO_DEVICE


def spec(rot=64, interleaved=0, axes=1, inv=None, axis=None):
    inv = [1.0] * (rot // 2) if inv is None else inv
    s = paged._RopeSpec(rot, interleaved, axes, (ctypes.c_double * max(1, len(inv)))(*inv), None)
    if axis is not None:
        s.axis = (ctypes.c_int * len(axis))(*axis)
    return s


def rope(L, q=A[0], qs=512, qo=A[1], qos=512, Hq=4, k=A[2], ks=512, ko=A[3], kos=256, Hkv=2, T=7, d=128, pos=A[4], ps=7, s=None, inverse=0):
    return L.fa_rope(q, qs, qo, qos, Hq, k, ks, ko, kos, Hkv, T, d, pos, ps, ctypes.byref(s) if s is not None else ctypes.byref(spec()),
                     inverse, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(Hq=-1), 1), (dict(d=48), 2), (dict(inverse=2), 1), (dict(qs=511), 1), (dict(kos=255), 1), (dict(ps=6), 1),
    (dict(q=None), 1), (dict(ko=None), 1), (dict(pos=None), 1), (dict(q=A[0] + 1), 3), (dict(pos=A[4] + 2), 3), (dict(qo=A[0] + 2), 8),
    (dict(qo=A[0], qos=520), 8), (dict(qo=A[2]), 8), (dict(ko=A[1]), 8), (dict(qo=A[4]), 8),
    (dict(s=spec(rot=63)), 1), (dict(s=spec(rot=130)), 1), (dict(s=spec(axes=0)), 1), (dict(s=spec(axes=5)), 1),
    (dict(s=spec(interleaved=2)), 1), (dict(s=spec(rot=4, inv=[1.0, float("nan")])), 1), (dict(s=spec(rot=4, axis=[0, 1])), 1),
    (dict(s=spec(rot=4, axis=[0, -1])), 1)])
def test_rope_refusals(L, kw, code):
    assert rope(L, **kw) == code


def test_rope_accepts(L):
    assert rope(L) in NO_DEVICE
    assert rope(L, qo=A[0], ko=A[2], kos=512) in NO_DEVICE                                   # in place
    fused = dict(q=A[0], qs=1024, k=A[0] + 1024, ks=1024)                                    # slices of one projection
    assert rope(L, **fused) in NO_DEVICE
    assert rope(L, **fused, qo=A[0], qos=1024, ko=A[0] + 1024, kos=1024) in NO_DEVICE
    assert rope(L, **fused, qo=A[0] + 512, qos=1024) == fa.FA_ERR_OVERLAP
    assert rope(L, T=0, q=None, k=None, qo=None, ko=None, pos=None) == fa.FA_OK
    assert rope(L, Hkv=0, k=None, ko=None) in NO_DEVICE


def cache(k=A[10], v=A[11], bs=16 * 2 * 128, ss=2 * 128, hs=128, n=50, page=16, Hkv=2, d=128):
    return paged._Cache(k, v, bs, ss, hs, n, page, Hkv, d)


def append(L, q=A[0], qs=512, qo=A[1], qos=512, Hq=4, k=A[2], ks=512, v=A[3], vs=512, T=7, pos=A[4], ps=7, s=None, c=None, slots=A[5]):
    return L.fa_rope_append(q, qs, qo, qos, Hq, k, ks, v, vs, T, pos, ps, ctypes.byref(s if s is not None else spec()),
                            ctypes.byref(c if c is not None else cache()), slots, None)


CACHES = [(dict(page=0), 1), (dict(n=-1), 1), (dict(Hkv=0), 1), (dict(d=72), 2), (dict(bs=16 * 2 * 128 - 8), 1), (dict(ss=2 * 128 + 4), 1),
          (dict(hs=120), 1), (dict(k=A[10] + 8), 3), (dict(v=A[10] + 256), 8), (dict(k=None), 1)]


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(Hq=-1), 1), (dict(ks=255), 1), (dict(vs=255), 1), (dict(slots=None), 1), (dict(slots=A[5] + 4), 3),
    (dict(k=None), 1), (dict(qo=A[10] + 512), 8), (dict(k=A[11]), 8), (dict(slots=A[10]), 8), (dict(qo=A[2]), 8), (dict(qo=A[0] + 4), 8),
    (dict(s=spec(rot=200)), 1)] + [(dict(c=cache(**kw)), code) for kw, code in CACHES])
def test_append_refusals(L, kw, code):
    assert append(L, **kw) == code


def test_append_accepts(L):
    assert append(L) in NO_DEVICE and append(L, qo=A[0]) in NO_DEVICE and append(L, Hq=0, q=None, qo=None) in NO_DEVICE
    # [block, head, slot, d]; k and v slices of one [block, 2, slot, head, d] or [block, slot, 2, head, d] array
    assert append(L, c=cache(ss=128, hs=16 * 128)) in NO_DEVICE
    n = 16 * 2 * 128
    assert append(L, c=cache(bs=2 * n, v=A[10] + 2 * n)) in NO_DEVICE
    assert append(L, c=cache(bs=2 * n, ss=4 * 128, v=A[10] + 4 * 128)) in NO_DEVICE
    assert append(L, c=cache(bs=2 * n - 2 * 128, ss=4 * 128, v=A[10] + 4 * 128)) == fa.FA_ERR_OVERLAP   # v's last row on the next block
    assert append(L, c=cache(bs=2 * n, v=A[10] + 2 * n - 256)) == fa.FA_ERR_OVERLAP
    # strides of axes of one entry mean nothing
    assert append(L, c=cache(Hkv=1, hs=3, bs=16 * 128, ss=128)) in NO_DEVICE and append(L, c=cache(n=1, bs=5)) in NO_DEVICE


def attend(L, q=A[0], qs=512, c=None, table=A[1], stride=8, max_blocks=8, cu=A[2], lens=A[3], R=4, T=9, Hq=4, max_new=3, scale=0.1, causal=1,
           window=0, out=A[4], lse=A[5], ws=A[6], ws_bytes=None):
    ws_bytes = fa.paged_workspace_bytes(4, 2, 128) if ws_bytes is None else ws_bytes
    return L.fa_paged_fwd(q, qs, ctypes.byref(c if c is not None else cache()), table, stride, max_blocks, cu, lens, R, T, Hq, max_new, scale,
                          causal, window, out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), 1), (dict(T=-1), 1), (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(max_new=-1), 1), (dict(qs=504), 1), (dict(qs=516), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(causal=2), 1), (dict(window=-1), 1), (dict(causal=0, window=4), 1),
    (dict(stride=7), 1), (dict(max_blocks=1 << 28, stride=1 << 28), 1), (dict(max_blocks=(1 << 27) - 1, stride=1 << 27), 1),
    (dict(q=None), 1), (dict(out=None), 1), (dict(cu=None), 1),
    (dict(lens=None), 1), (dict(table=None), 1), (dict(ws=None), 1), (dict(ws_bytes=1000), 1), (dict(ws=A[6] + 128), 3),
    (dict(q=A[0] + 8), 3), (dict(out=A[4] + 2), 3), (dict(lse=A[5] + 2), 3), (dict(out=A[0]), 8), (dict(lse=A[4]), 8), (dict(ws=A[10]), 8),
    (dict(out=A[11]), 8), (dict(lse=A[1]), 8)] + [(dict(c=cache(**kw)), code) for kw, code in CACHES if kw != dict(v=A[10] + 256)])
def test_attend_refusals(L, kw, code):
    assert attend(L, **kw) == code


def test_attend_accepts(L):
    assert attend(L) in NO_DEVICE and attend(L, lse=None) in NO_DEVICE and attend(L, causal=0) in NO_DEVICE
    assert attend(L, R=0, q=None, out=None) == fa.FA_OK and attend(L, T=0, q=None, out=None) == fa.FA_OK


def test_workspace_bytes(L):
    assert fa.paged_workspace_bytes(3, 2, 128) == 0 and fa.paged_workspace_bytes(4, 2, 100) == 0 and fa.paged_workspace_bytes(0, 1, 64) == 0
    assert all(fa.paged_workspace_bytes(8, 2, d) % 256 == 0 and fa.paged_workspace_bytes(8, 2, d) > 0 for d in fa.SUPPORTED_HEAD_DIMS)


def test_status_text(L):
    assert "out of range" in " ".join(fa.status_string(fa.FA_ERR_PAGED_RANGE).split())


def test_binding_checks():
    """Types, shapes and strides that the C entry points cannot see."""
    import torch
    with pytest.raises(ValueError):
        fa.RopeTable([1.0, 2.0], axis=[0])
    with pytest.raises(ValueError):
        fa.RopeTable([float("inf")])
    with pytest.raises(ValueError):
        fa.RopeTable([1.0], axis=[4])
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.fa_rope(x, torch.zeros(3, dtype=torch.int32), fa.RopeTable([1.0] * 32))          # not on a GPU
    with pytest.raises(ValueError):
        fa.fa_rope(x.float(), torch.zeros(3, dtype=torch.int32), fa.RopeTable([1.0] * 32))  # fp32
    with pytest.raises(ValueError):
        fa.fa_paged_fwd(x, x, x, None, None, None, max_new=1)
    with pytest.raises(ValueError):
        fa.fa_kv_release(torch.zeros(2), torch.zeros(2), None, None, None, page_size=16)
    with pytest.raises(ValueError):
        fa.PagedKV(1, 1, 16, 1, 64, layout="dnh", device="cpu")


class OnGpu:
    """A CPU tensor that says it is on a GPU: for the binding's look at types, shapes and strides."""
    is_cuda = True

    def __init__(self, t):
        self.t, self.dtype, self.shape = t, t.dtype, t.shape

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_expanded_positions_and_tables():
    """The stride that the tensor has is the one that is passed on: 0 for one row that all axes (or
    requests) share, and rows that overlap otherwise are refused."""
    import torch
    paged._init()
    table = fa.RopeTable([1.0, 0.5, 0.25], axis=[0, 1, 2])
    row = torch.arange(5, dtype=torch.int32)
    assert table._spec(OnGpu(row[None].expand(3, 5)), 5)[1:] == (row.data_ptr(), 0)
    assert table._spec(OnGpu(torch.zeros(3, 9, dtype=torch.int32)[:, :5]), 5)[2] == 9
    assert table._spec(OnGpu(row[:1][None].expand(3, 1)), 1)[2] == 0
    with pytest.raises(ValueError, match="overlap"):
        table._spec(OnGpu(torch.as_strided(torch.arange(16, dtype=torch.int32), (3, 5), (4, 1))), 5)
    blocks = torch.arange(8, dtype=torch.int32)
    shared = OnGpu(blocks[None].expand(4, 8))
    assert paged._table(shared, 4) == (blocks.data_ptr(), 0, 8)
    with pytest.raises(ValueError, match="overlap"):
        paged._table(shared, 4, written=True)
    for written in (False, True):
        with pytest.raises(ValueError, match="overlap"):
            paged._table(OnGpu(torch.as_strided(torch.arange(40, dtype=torch.int32), (4, 8), (7, 1))), 4, written)
        assert paged._table(OnGpu(torch.zeros(4, 12, dtype=torch.int32)[:, :8]), 4, written)[1:] == (12, 8)
        assert paged._table(OnGpu(blocks[None]), 1, written)[1:] == (8, 8)


def test_one_row_for_all(L):
    """A stride of 0 from axis to axis or row to row, where the array is only read."""
    assert rope(L, ps=0, s=spec(axes=3)) in NO_DEVICE and append(L, ps=0, s=spec(axes=3)) in NO_DEVICE
    assert attend(L, stride=0) in NO_DEVICE and release(L, stride=0) in NO_DEVICE
    assert reserve(L, stride=0) == fa.FA_ERR_INVALID_ARG
    assert rope(L, ps=-7) == attend(L, stride=-8) == release(L, stride=-8) == fa.FA_ERR_INVALID_ARG


def test_a_workspace_has_the_bytes_that_it_counts():
    """numel() of an expanded or strided tensor says more than there is memory behind its pointer, or skips some."""
    import torch
    paged._init()
    q, out = (OnGpu(torch.zeros(2, 4, 64, dtype=torch.bfloat16)) for _ in range(2))
    cache = OnGpu(torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16))
    ints = [OnGpu(torch.zeros(n, dtype=torch.int32)) for n in (2, 1)]
    table = OnGpu(torch.zeros(1, 3, dtype=torch.int32))
    need = fa.paged_workspace_bytes(4, 2, 64)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(need), torch.zeros(2 * need, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            fa.fa_paged_fwd(q, cache, cache, table, *ints, max_new=2, out=out, return_lse=False, workspace=OnGpu(ws), stream=0)
    with pytest.raises(ValueError, match="workspace"):
        fa.fa_paged_fwd(q, cache, cache, table, *ints, max_new=2, out=out, return_lse=False, workspace=torch.zeros(need, dtype=torch.uint8),
                        stream=0)


def test_a_cache_keeps_few_buffers(monkeypatch):
    """Steps of every size: what is kept grows with the largest step, not with the number of sizes, and a size
    has the same buffers each time."""
    import torch
    steps = []
    monkeypatch.setattr(paged, "fa_kv_reserve", lambda *a, **kw: steps.append((kw["num_tokens"], kw["positions"], kw["slots"])))
    kv = fa.PagedKV(2, 4, 16, 1, 64, device="cpu")
    at = {}
    for n in list(range(0, 3000)) + [7, 2999, 64, 65, 1]:
        pos, slots = kv.reserve(None, n)
        assert steps[-1] == (n, pos, slots) and kv.positions is pos and kv.slots is slots
        assert pos.shape == slots.shape == (n,) and pos.dtype == torch.int32 and slots.dtype == torch.int64
        assert n == 0 or at.setdefault(n, (pos.data_ptr(), slots.data_ptr())) == (pos.data_ptr(), slots.data_ptr())
    kept = sum(t.numel() for pair in kv._buffers.values() for t in pair)
    assert kept <= 2 * 4 * 2999
    mine = torch.zeros(5, dtype=torch.int32), torch.zeros(5, dtype=torch.int64)
    kept = dict(kv._buffers)
    assert kv.reserve(None, 5, positions=mine[0], slots=mine[1]) == mine and kv.positions is mine[0] and kv.slots is mine[1]
    pos, slots = kv.reserve(None, 5, slots=mine[1])
    assert slots is mine[1] and pos.data_ptr() == at[5][0] and kv._buffers == kept
    assert kv.reserve(None, 5)[1].data_ptr() == at[5][1]


def test_given_rows_of_the_wrong_size():
    import torch
    kv = fa.PagedKV(2, 4, 16, 1, 64, device="cpu")
    for name in ("seq_lens", "block_table", "free_blocks", "free_count", "cu_seqlens"):
        setattr(kv, name, OnGpu(getattr(kv, name)))
    rows = dict(positions=OnGpu(torch.zeros(6, dtype=torch.int32)), slots=OnGpu(torch.zeros(5, dtype=torch.int64)))
    with pytest.raises(ValueError, match="positions"):
        kv.reserve(OnGpu(torch.zeros(2, dtype=torch.int32)), 5, stream=0, **rows)
    assert kv.slots is None
