"""Host-side tests of the serving operators (no GPU): refusals of the C ABI and
of the binding before anything is launched, and the reference page layout."""
import ctypes

import numpy as np
import pytest
import torch

import ar_decoding_b200 as tidar
import kv4_ref
from ar_decoding_b200 import build

FAKE, MISALIGNED = 0x10000, 0x10008          # never dereferenced


@pytest.fixture(scope="module")
def L():
    build.build()
    return tidar.lib()


def _pool(**kw):
    return ctypes.byref(tidar.PagePool(**dict(dict(free_pages=FAKE, free_count=FAKE, capacity=4), **kw)))


def _tables(L, table=FAKE, ctx=FAKE, new=FAKE, pool=None, tout=FAKE, cout=FAKE, starts=FAKE, slots=FAKE, pos=FAKE, **kw):
    d = tidar.TablesDesc(**dict(dict(batch=2, page_size=64, num_pages=8, max_pages_per_seq=4, max_rows=64), **kw))
    return L.tidar_build_tables(ctypes.byref(d), table, ctx, new, pool or _pool(), tout, cout, starts, slots, pos, None)


def test_build_tables_refusals(L):
    assert L.tidar_build_tables(None, *[FAKE] * 3, _pool(), *[FAKE] * 5, None) == tidar.ERR_INVALID_ARG
    for kw in (dict(batch=-1), dict(max_rows=-1), dict(num_pages=0), dict(max_pages_per_seq=0), dict(page_size=0),
               dict(table=None), dict(ctx=None), dict(new=None), dict(tout=None), dict(cout=None), dict(starts=None),
               dict(slots=None), dict(slots=MISALIGNED), dict(pos=FAKE + 4), dict(pool=_pool(free_count=None)),
               dict(pool=_pool(capacity=-1)), dict(pool=_pool(free_pages=None))):
        assert _tables(L, **kw) == tidar.ERR_INVALID_ARG, kw
    for kw in (dict(page_size=48), dict(batch=65537), dict(max_pages_per_seq=1 << 25)):
        assert _tables(L, **kw) == tidar.ERR_UNSUPPORTED, kw
    assert _tables(L, batch=0, table=None) == tidar.OK


def _rows(L, fn, kp=FAKE, vp=FAKE, k=FAKE, v=FAKE, slots=FAKE, **kw):
    d = tidar.Kv4Desc(**dict(dict(rows=3, num_kv_heads=2, head_dim=128, page_size=64, num_pages=4, dtype=tidar.BF16), **kw))
    if fn == "append":
        return L.tidar_kv4_append(ctypes.byref(d), kp, vp, k, v, slots, None)
    return L.tidar_kv4_gather(ctypes.byref(d), kp, vp, slots, k, v, None)


@pytest.mark.parametrize("fn", ["append", "gather"])
def test_kv4_rows_refusals(L, fn):
    for kw in (dict(rows=-1), dict(num_kv_heads=0), dict(num_pages=0), dict(page_size=0), dict(kp=None), dict(vp=None),
               dict(k=None), dict(v=None), dict(slots=None), dict(kp=MISALIGNED), dict(k=MISALIGNED),
               dict(k_row_stride=255), dict(k_row_stride=260), dict(v_row_stride=128)):
        assert _rows(L, fn, **kw) == tidar.ERR_INVALID_ARG, kw
    for kw in (dict(head_dim=96), dict(page_size=8), dict(dtype=5)):
        assert _rows(L, fn, **kw) == tidar.ERR_UNSUPPORTED, kw
    assert _rows(L, fn, rows=0, k=None) == tidar.OK


def test_kv4_page_bytes(L):
    assert tidar.kv4_page_bytes(64, 128) == 4608 and tidar.kv4_page_bytes(16, 64) == 576
    assert L.tidar_kv4_page_bytes(64, 96) == 0 and L.tidar_kv4_page_bytes(8, 64) == 0
    with pytest.raises(ValueError):
        tidar.kv4_page_bytes(48, 128)


def _desc(**kw):
    return tidar.StepDesc(**dict(dict(batch=1, num_q_heads=4, num_kv_heads=2, head_dim=128, k=4, page_size=64,
                                      max_prefix_len=100, dtype=tidar.BF16, softmax_scale=0.0, path=0), **kw))


def _cache(**kw):
    return ctypes.byref(tidar.KVCacheDesc(**dict(dict(k_pages=FAKE, v_pages=FAKE, page_table=FAKE, seq_lens=FAKE,
                                                      num_pages=8, max_pages_per_seq=2), **kw)))


def _attn(L, d, c=None, q=FAKE, flags=3, lse=None, ws=None, wsb=0):
    return L.tidar_step_attn_kv4(ctypes.byref(d), c or _cache(), q, FAKE, FAKE, flags, FAKE, lse, ws, wsb, None)


def test_step_attn_kv4_refusals(L):
    for d in (_desc(num_q_heads=3), _desc(k=-1), _desc(path=9), _desc(max_prefix_len=1000)):
        assert _attn(L, d) == tidar.ERR_INVALID_ARG
    for d in (_desc(head_dim=96), _desc(k=17), _desc(page_size=48), _desc(dtype=7), _desc(path=tidar.PATH_PAIR),
              _desc(batch=32768, num_kv_heads=4, path=tidar.PATH_SIMT), _desc(path=tidar.PATH_DEC)):
        assert _attn(L, d) == tidar.ERR_UNSUPPORTED
    assert _attn(L, _desc(), q=None) == tidar.ERR_INVALID_ARG
    assert _attn(L, _desc(), q=MISALIGNED) == tidar.ERR_INVALID_ARG
    assert _attn(L, _desc(), flags=4) == tidar.ERR_INVALID_ARG
    assert _attn(L, _desc(), flags=0) == tidar.ERR_INVALID_ARG           # prefix only: lse is required
    assert _attn(L, _desc(), _cache(k_pages=MISALIGNED)) == tidar.ERR_INVALID_ARG
    assert _attn(L, _desc(batch=0)) == tidar.OK
    d = _desc(max_prefix_len=8192, num_q_heads=32, num_kv_heads=8, k=0, path=tidar.PATH_SIMT)
    c = _cache(max_pages_per_seq=129)
    need = L.tidar_step_attn_kv4_workspace_bytes(ctypes.byref(d))
    assert need > 0
    assert _attn(L, d, c, ws=FAKE, wsb=need - 1) == tidar.ERR_INVALID_ARG
    assert _attn(L, d, c, ws=FAKE + 16, wsb=need) == tidar.ERR_INVALID_ARG


def test_commit_kv4_refusals(L):
    d = ctypes.byref(_desc())
    assert L.tidar_commit_kv4(d, _cache(), None, FAKE, FAKE, None) == tidar.ERR_INVALID_ARG
    assert L.tidar_commit_kv4(ctypes.byref(_desc(k=20)), _cache(), FAKE, FAKE, FAKE, None) == tidar.ERR_UNSUPPORTED
    assert L.tidar_commit_kv4(d, None, FAKE, FAKE, FAKE, None) == tidar.ERR_INVALID_ARG


def test_linear_fused_refusals(L):
    def call(T=5, N=100, K=64, dt=tidar.BF16, x=FAKE, w=FAKE, b=None, act=0, r=None, y=FAKE):
        return L.tidar_linear_fused(T, N, K, dt, x, w, b, act, r, y, None)
    for kw in (dict(T=-1), dict(N=0), dict(K=0), dict(act=5), dict(act=-1), dict(x=None), dict(w=None), dict(y=None),
               dict(x=MISALIGNED), dict(b=MISALIGNED), dict(r=MISALIGNED), dict(y=MISALIGNED)):
        assert call(**kw) == tidar.ERR_INVALID_ARG, kw
    assert call(K=63) == tidar.ERR_UNSUPPORTED and call(dt=tidar.F32) == tidar.ERR_UNSUPPORTED
    assert call(T=0, x=None) == tidar.OK


def test_linear_fused_refuses_overlap_and_sizes_past_its_indices(L):
    x, w, b, r, y = (FAKE + (i << 24) for i in range(5))           # 16 MB apart
    def call(T=5, N=100, K=64, x=x, w=w, b=b, r=r, y=y):
        return L.tidar_linear_fused(T, N, K, tidar.BF16, x, w, b, 0, r, y, None)
    for kw in (dict(y=x), dict(y=w), dict(y=b), dict(y=r + 16), dict(y=r - 16), dict(y=x + 2 * 5 * 64 - 16),
               dict(y=w - 2 * 5 * 100 + 8), dict(y=w + 16 * 100)):
        assert call(**kw) == tidar.ERR_INVALID_ARG, kw
    for kw in (dict(T=2**30 + 1), dict(N=2**30 + 1), dict(K=2**30 + 8), dict(T=2**30, N=2**20)):
        assert call(**kw) == tidar.ERR_UNSUPPORTED, kw


def test_binding_refuses_host_tensors():
    i32, f = torch.int32, torch.bfloat16
    table, lens = torch.full((2, 4), -1, dtype=i32), torch.ones(2, dtype=i32)
    pool = dict(free_pages=torch.arange(8, dtype=i32), free_count=torch.tensor([8], dtype=i32))
    with pytest.raises(ValueError):
        tidar.build_tables(table, lens, lens, pool, page_size=64, num_pages=8, max_rows=64)
    cache = tidar.kv4_cache(4, 2, 64, 128, table, lens)
    rows, slots = torch.zeros(3, 2, 128, dtype=f), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        tidar.kv4_append(cache, rows, rows, slots)
    with pytest.raises(ValueError):
        tidar.kv4_gather(cache, slots, head_dim=128)
    q = torch.zeros(2, 1, 2, 128, dtype=f)
    with pytest.raises(ValueError):
        tidar.step_attn_kv4(q, q, q, cache, 0, max_prefix_len=8)
    with pytest.raises(ValueError):
        tidar.commit_kv4(cache, lens, 0, head_dim=128, max_prefix_len=8)
    with pytest.raises(ValueError):
        tidar.reserve(cache, pool, 0, max_prefix_len=8)
    with pytest.raises(ValueError):
        tidar.linear_fused(rows.reshape(-1, 64), torch.zeros(8, 64, dtype=f))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("is_key", [True, False])
def test_reference_page_roundtrip(D, is_key):
    rng = np.random.default_rng(D)
    x = rng.standard_normal((2, 16, D)).astype(np.float32)
    x[0, 3] = 0
    x[1, 2, 5] = np.inf
    pages = kv4_ref.pack(x, is_key)
    assert pages.shape == (2, tidar.kv4_page_bytes(16, D)) and pages.dtype == np.uint8
    got = kv4_ref.unpack(pages, 16, D, is_key)
    want = kv4_ref.values(x)
    np.testing.assert_array_equal(got, want)
    assert np.isnan(want[1, 2, :32]).all() and not np.isnan(want[1, 2, 32:]).any()
    fine = ~np.isnan(want)
    # a value is off by at most half a step, s <= max|x| / 7 (1 + 2^-5)
    top = np.abs(np.where(np.isinf(x), 0, x)).reshape(2, 16, D // 32, 32).max(-1).repeat(32, -1).reshape(x.shape)
    assert (np.abs(want - x)[fine] <= (top / 14 * (1 + 2.0 ** -5))[fine] + 1e-12).all()


def test_reference_layout_by_hand():
    # one row whose group 1 holds the code 1 at dim 8y + 2i + h = 13 (y 1, i 2, h 1) and 7 at dim 0
    x = np.zeros((16, 64))
    x[0, 32], x[0, 32 + 13] = 7.0, 1.0
    k, v = kv4_ref.pack(x, True).view(np.uint16), kv4_ref.pack(x, False).view(np.uint16)
    # n = 2: key units y 4 + 2G + h, value units y 4 + 2h + G
    assert k[2] == 7 and k[4 + 3] == 1 << 8 and np.count_nonzero(k[:16]) == 2
    assert v[1] == 7 and v[4 + 3] == 1 << 8 and np.count_nonzero(v[:16]) == 2
    assert k[16 * 16 + 1] == 0x3f80 and np.count_nonzero(k[16 * 16:]) == 1


@pytest.mark.parametrize("bad", [dict(page_table=(1, 4)), dict(page_table=(8,)), dict(page_table=(0, 4))])
def test_binding_refuses_tables_without_a_row_for_each_sequence(monkeypatch, bad):
    # A table with fewer rows than there are lengths would be read past its end.  Host
    # tensors stand in for device ones up to the library call, which is not reached.
    monkeypatch.setattr(tidar, "_dev", lambda *a, **kw: None)
    monkeypatch.setattr(tidar, "_away", lambda *a, **kw: False)
    monkeypatch.setattr(tidar, "lib", lambda: pytest.fail("the library was called"))
    shapes = dict(dict(page_table=(2, 4), seq_lens=(2,)), **bad)
    common = {n: torch.zeros(v, dtype=torch.int32) for n, v in shapes.items()}
    four = dict(common, **{n: torch.zeros(8, 2, 4608, dtype=torch.uint8) for n in ("k_pages", "v_pages")})
    wide = dict(common, **{n: torch.zeros(8, 2, 64, 128, dtype=torch.bfloat16) for n in ("k_pages", "v_pages")})
    pool = dict(free_pages=torch.arange(8, dtype=torch.int32), free_count=torch.tensor([8], dtype=torch.int32))
    count = torch.zeros(2, dtype=torch.int32)
    q, kv = torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 1, 2, 128, dtype=torch.bfloat16)
    for call in (lambda: tidar.commit_kv4(four, count, 0, head_dim=128, max_prefix_len=8),
                 lambda: tidar.reserve(four, pool, 0, max_prefix_len=8, head_dim=128),
                 lambda: tidar.reserve(wide, pool, 0, max_prefix_len=8),
                 lambda: tidar.commit(wide, count, 0, max_prefix_len=8),
                 lambda: tidar.step_attn(q, kv, kv, wide, 0, max_prefix_len=8),
                 lambda: tidar.step_attn_kv4(q, kv, kv, four, 0, max_prefix_len=8)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        tidar.step_attn(q, kv, kv, dict(wide, page_table=torch.zeros(2, 4, dtype=torch.int32), seq_lens=count[:1]), 0,
                        max_prefix_len=8)


def test_kv4_refuses_prefixes_past_its_indices(L):
    # a table this wide is a legal argument; the kernels count keys in 32 bits
    c = _cache(max_pages_per_seq=1 << 25)
    for k in (0, 4, 16):
        for path in range(4):
            d = _desc(k=k, max_prefix_len=(1 << 30) + 1, path=path)
            assert _attn(L, d, c, ws=FAKE, wsb=1 << 40) == tidar.ERR_UNSUPPORTED, (k, path)
            assert L.tidar_step_attn_kv4_plan(ctypes.byref(d), None, None, None) == tidar.ERR_UNSUPPORTED
            assert L.tidar_step_attn_kv4_workspace_bytes(ctypes.byref(d)) == 0
        d = _desc(k=k, max_prefix_len=(1 << 30) + 1)
        assert L.tidar_commit_kv4(ctypes.byref(d), c, FAKE, FAKE, FAKE, None) == tidar.ERR_UNSUPPORTED
    d = _desc(max_prefix_len=1 << 30, path=tidar.PATH_SIMT)
    assert L.tidar_step_attn_kv4_plan(ctypes.byref(d), None, None, None) == tidar.OK
