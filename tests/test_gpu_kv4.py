"""The 4-bit cache's store, read-back and commit against their definitions (the
codes, scales and values are exact: every comparison here is of equal bytes)."""
import numpy as np
import pytest
import torch

import ar_decoding_b200 as tidar
import kv4_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rows(seed, shape, dtype, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if kind == "ties":                          # quotients that fall on halves: scale 1 (top 7), codes k + 1/2
        x = torch.randint(-14, 15, shape, generator=g).float() / 2
        x[..., ::32] = 7.0
    elif kind == "wide":                        # magnitudes from 2^-130 to 2^127
        x = x * torch.exp2(torch.randint(-130, 128, (*shape[:-1], 1), generator=g).float())
    elif kind == "odd":
        x[..., 1] = float("nan")
        x[..., 33] = float("inf")
        if shape[-1] > 64:
            x[..., 64:96] = 0
            x[..., 96:] = -0.0
    return x.to(DT[dtype])


def cache_of(pages, H, ps, D, fill=0xA5):
    c = tidar.kv4_cache(pages, H, ps, D, torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                        torch.zeros(1, dtype=torch.int32, device="cuda"))
    c["k_pages"].fill_(fill)
    c["v_pages"].fill_(fill)
    return c


def expected(pages0, x, slots, ps, D, is_key):
    """Page bytes after the rows x [T][H][D] went to their slots."""
    want = pages0.copy()
    H = x.shape[1]
    one = np.zeros((H, 16, D))
    for t, s in enumerate(slots):
        if s < 0 or s >= want.shape[0] * ps:
            continue
        one[:, 0] = x[t]
        b = kv4_ref.pack(one, is_key)                    # [H][16-row page]
        page, r = s // ps, s % ps
        want[page, :, r * D // 2:(r + 1) * D // 2] = b[:, :D // 2]
        at = ps * D // 2
        want[page, :, at + r * D // 16:at + (r + 1) * D // 16] = b[:, 8 * D:8 * D + D // 16]
    return want


def same_bytes(got, want):
    # a NaN scale may be any NaN
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("kind", ["normal", "ties", "wide", "odd"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,D,ps", [(1, 1, 64, 16), (37, 2, 128, 16), (70, 3, 64, 32), (129, 8, 128, 64), (9, 1, 128, 128)])
def test_append_and_gather(T, H, D, ps, dtype, kind):
    k, v = rows(1, (T, H, D), dtype, kind), rows(2, (T, H, D), dtype, kind)
    pages = -(-T // ps) + 2
    r = np.random.default_rng(3)
    slots = r.permutation(pages * ps)[:T].astype(np.int64)
    if T > 4:
        slots[3], slots[4] = -1, -7
    c = cache_of(pages, H, ps, D)
    before = c["k_pages"].cpu().numpy()
    sl = torch.from_numpy(slots).cuda()
    tidar.kv4_append(c, k.cuda(), v.cuda(), sl)
    assert tidar.device_status() == (tidar.OK, 0)
    for name, x, is_key in (("k_pages", k, True), ("v_pages", v, False)):
        same_bytes(c[name].cpu().numpy(), expected(before, x.double().numpy(), slots, ps, D, is_key))
    for out_dt in DT.values():
        out = tuple(torch.full((T, H, D), 99.0, dtype=out_dt, device="cuda") for _ in range(2))
        tidar.kv4_gather(c, sl, out=out)
        for got, x in zip(out, (k, v)):
            want = np.where((slots < 0)[:, None, None], 99.0, kv4_ref.values(x.double().numpy()))
            np.testing.assert_array_equal(got.double().cpu().numpy(), want)
    assert tidar.device_status() == (tidar.OK, 0)


def test_slot_past_the_cache_is_reported_and_skipped():
    c = cache_of(2, 2, 16, 64)
    before = c["k_pages"].clone()
    k = rows(1, (3, 2, 64), "bf16").cuda()
    sl = torch.tensor([32, 1 << 40, -1], device="cuda")
    tidar.kv4_append(c, k, k, sl)
    assert tidar.device_status() == (tidar.ERR_DEVICE, tidar.DEVERR_BAD_PAGE)
    assert torch.equal(c["k_pages"], before)
    out = (torch.ones_like(k), torch.ones_like(k))
    tidar.kv4_gather(c, sl, out=out)
    assert tidar.device_status() == (tidar.ERR_DEVICE, tidar.DEVERR_BAD_PAGE)
    assert (out[0] == 1).all() and (out[1] == 1).all()


def test_strided_rows_of_a_projection():
    T, Hq, H, D = 21, 4, 2, 128
    qkv = rows(4, (T, Hq + 2 * H, D), "bf16").cuda()
    k, v = qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    sl = torch.arange(T, device="cuda")
    a, b = cache_of(2, H, 16, D), cache_of(2, H, 16, D)
    tidar.kv4_append(a, k, v, sl)
    tidar.kv4_append(b, k.contiguous(), v.contiguous(), sl)
    assert torch.equal(a["k_pages"], b["k_pages"]) and torch.equal(a["v_pages"], b["v_pages"])
    for bad in (k.transpose(0, 1), qkv[:, ::2], qkv[..., ::2]):
        with pytest.raises(ValueError):
            tidar.kv4_append(a, bad, bad, sl)
    with pytest.raises(tidar.TidarError):                     # rows not 16 bytes apart
        odd = torch.zeros(T * (H * D + 4), dtype=torch.bfloat16, device="cuda").as_strided((T, H, D), (H * D + 4, D, 1))
        tidar.kv4_append(a, odd, odd, sl)


def test_bad_shapes_are_refused():
    c = cache_of(2, 2, 16, 64)
    k, sl = rows(1, (3, 2, 64), "bf16").cuda(), torch.arange(3, device="cuda")
    for args in ((k, k[:2], sl), (k, k.float(), sl), (k, k, sl[:2]), (k, k, sl.int()), (k[:, :1], k[:, :1], sl),
                 (k.half(), k.half(), sl), (k[..., :32], k[..., :32], sl)):
        with pytest.raises(ValueError):
            tidar.kv4_append(c, *args)
    with pytest.raises(ValueError):
        tidar.kv4_gather(c, sl)
    tidar.kv4_append(c, k[:0], k[:0], sl[:0])
    assert tidar.kv4_gather(c, sl[:0], head_dim=64)[0].shape == (0, 2, 64)


def test_far_pages_pass_32_bit_offsets():
    # page bytes of the far page lie past 2^32
    ps, D, H = 128, 128, 8
    pages = (1 << 32) // (H * tidar.kv4_page_bytes(ps, D)) + 8
    c = cache_of(pages, H, ps, D, fill=0)
    k = rows(5, (2, H, D), "bf16").cuda()
    sl = torch.tensor([(pages - 1) * ps + 5, 7], device="cuda")
    tidar.kv4_append(c, k, k, sl)
    got = tidar.kv4_gather(c, sl, head_dim=D, dtype=torch.float32)
    want = kv4_ref.values(k.double().cpu().numpy())
    for g in got:
        np.testing.assert_array_equal(g.double().cpu().numpy(), want)
    assert int(c["k_pages"][pages - 1].count_nonzero()) > 0 and int(c["k_pages"][1:pages - 1].count_nonzero()) == 0


@pytest.mark.parametrize("k,ps,D,B", [(0, 16, 64, 1), (4, 64, 128, 3), (16, 16, 128, 5), (8, 32, 64, 40)])
def test_commit_zeroes_rejected_rows(k, ps, D, B):
    H, n = 2, max(k, 1)
    r = np.random.default_rng(k)
    P = r.integers(0, 3 * ps, B)
    need = -(-(P + n) // ps)
    table = np.full((B, int(need.max()) + 1), -1, dtype=np.int32)
    ids, at = r.permutation(int(need.sum()) + 1).astype(np.int32), 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    c = cache_of(len(ids), H, ps, D)
    c["page_table"], c["seq_lens"] = torch.from_numpy(table).cuda(), torch.from_numpy(P.astype(np.int32)).cuda()
    want = {m: c[m].cpu().numpy() for m in ("k_pages", "v_pages")}
    acc = r.integers(0, n + 1, B).astype(np.int32)
    wt, rel = table.copy(), []
    for b in range(B):
        for pos in range(P[b] + acc[b], P[b] + n):
            page, q = table[b, pos // ps], pos % ps
            for m in want.values():
                m[page, :, q * D // 2:(q + 1) * D // 2] = 0
                m[page, :, ps * D // 2 + q * D // 16:ps * D // 2 + (q + 1) * D // 16] = 0
        for e in range(-(-int(P[b] + acc[b]) // ps), -(-int(P[b] + n) // ps)):
            rel.append(int(table[b, e]))
            wt[b, e] = -1
    released, num = tidar.commit_kv4(c, torch.from_numpy(acc).cuda(), k, head_dim=D, max_prefix_len=int(P.max()) if P.max() else 1)
    assert tidar.device_status() == (tidar.OK, 0)
    for m in want:
        np.testing.assert_array_equal(c[m].cpu().numpy(), want[m])
    np.testing.assert_array_equal(c["page_table"].cpu().numpy(), wt)
    np.testing.assert_array_equal(c["seq_lens"].cpu().numpy(), P + acc)
    assert int(num) == len(rel) and released.cpu().numpy()[:len(rel)].tolist() == rel
    assert (released.cpu().numpy()[len(rel):] == -1).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_without_a_slot_are_zeros_where_the_call_allocates(D, dtype):
    c = tidar.kv4_cache(4, 3, 16, D, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                        torch.zeros(1, dtype=torch.int32, device="cuda"))
    rows = torch.randn(9, 3, D, device="cuda").to(dtype)
    tidar.kv4_append(c, rows, rows, torch.arange(9, device="cuda"))
    slots = torch.tensor([-1, 0, 5, -7, 8, -1], device="cuda")
    dirty = [torch.full((6, 3, D), float("nan"), device="cuda", dtype=dtype) for _ in range(4)]
    del dirty                                             # what the call is given to allocate
    k, v = tidar.kv4_gather(c, slots, head_dim=D, dtype=dtype)
    want = [torch.full_like(k, 3.0) for _ in range(2)]
    tidar.kv4_gather(c, slots, out=tuple(want))
    dead = slots < 0
    for got, ref in ((k, want[0]), (v, want[1])):
        assert (got[dead] == 0).all() and (ref[dead] == 3).all()
        assert torch.equal(got[~dead], ref[~dead])
    assert tidar.device_status() == (tidar.OK, 0)
