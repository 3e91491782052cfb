"""Step attention over the 4-bit cache against the 64-bit reference on the values
the cache stands for.

Tolerances.  bf16: every p is rounded once (2^-8 of itself at most) before it
meets V, the sum l is not, so the output moves by at most 2^-8 sum p|v| / l; the
result's own rounding adds 2^-8 |out|.  A score is a sum of D products in fp32
whose partial sums reach at most 143/7 of sum |q||k| (codes enter the matrix
product offset by 136 at most): D/16 + 8 roundings of 2^-23 of that, which is the lse's
error, and times sum p|v| the output's.  fp32: D + 8 roundings of 2^-23 of
sum |q||k|, and 2^-23 a step of sums over the keys.
"""
import numpy as np
import pytest
import torch

import ar_decoding_b200 as tidar
import kv4_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(seed, P, Hq, H, D, k, ps, dtype, q_scale=1.0, stale="random", extra=2):
    """A cache of quantised rows (rows past the prefix `stale`), step inputs, all on the GPU."""
    g = torch.Generator().manual_seed(seed)
    r = np.random.default_rng(seed)
    B, n, R = len(P), max(k, 1), (1 if k == 0 else k + k * k)
    need = [-(-(p + n) // ps) for p in P]
    ids = r.permutation(sum(need) + extra).astype(np.int32)
    table, at = np.full((B, max(need) + 1), -1, dtype=np.int32), 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    x = [torch.randn(len(ids), H, ps, D, generator=g).to(DT[dtype]).double().numpy() for _ in range(2)]
    if stale == "nan":
        for b in range(B):
            for pos in range(P[b], table.shape[1] * ps):
                if table[b, pos // ps] >= 0:
                    for m in x:
                        m[table[b, pos // ps], :, pos % ps] = np.nan
    pages = [kv4_ref.pack(m, key) for m, key in zip(x, (True, False))]
    if stale == "ff":                                  # bytes nobody wrote: codes -1, scales NaN
        used = np.zeros((len(ids), ps), dtype=bool)
        for b in range(B):
            for pos in range(P[b]):
                used[table[b, pos // ps], pos % ps] = True
        for m in pages:
            codes = m[..., :ps * D // 2].reshape(len(ids), H, ps, D // 2)
            codes[np.broadcast_to(~used[:, None], codes.shape[:3])] = 0xff
            sc = m[..., ps * D // 2:].reshape(len(ids), H, ps, D // 16)
            sc[np.broadcast_to(~used[:, None], sc.shape[:3])] = 0xff
    cache = dict(k_pages=torch.from_numpy(pages[0]).cuda(), v_pages=torch.from_numpy(pages[1]).cuda(),
                 page_table=torch.from_numpy(table).cuda(), seq_lens=torch.tensor(P, dtype=torch.int32).cuda())
    rnd = lambda *s: torch.randn(*s, generator=g).to(DT[dtype]).cuda()  # noqa: E731
    q = (torch.randn(B, R, Hq, D, generator=g) * q_scale).to(DT[dtype]).cuda()
    vals = [kv4_ref.unpack(m, ps, D, key) for m, key in zip(pages, (True, False))]      # [page][H][ps][D]
    pref = [[np.concatenate([v[i] for i in table[b, :-(-P[b] // ps)]], 1).transpose(1, 0, 2)[:P[b]] if P[b]
             else np.zeros((0, H, D)) for b in range(B)] for v in vals]
    return dict(cache=cache, q=q, k_blk=rnd(B, R, H, D), v_blk=rnd(B, R, H, D), pref=pref, table=table, P=P, k=k, ps=ps,
                D=D, dtype=dtype)


def compare(st, out, lse, step_keys=True, seqs=None):
    dt, D = st["dtype"], st["D"]
    q, kb, vb = (st[n].double().cpu().numpy() for n in ("q", "k_blk", "v_blk"))
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(len(st["P"])) if seqs is None else seqs:
        wo, wl, spread, mag = kv4_ref.attention(q[b], kb[b], vb[b], st["pref"][0][b], st["pref"][1][b], st["k"], step_keys)
        keys = st["P"][b] + q.shape[1]
        if dt == "bf16":
            s_err = (D / 16 + 8) * 2.0 ** -23 * mag * 143 / 7
            tol = 2.0 ** -8 * (np.abs(wo) + spread) + 2 * s_err * spread
        else:
            s_err = (D + 8) * 2.0 ** -23 * mag
            tol = (2 * s_err + 2.0 ** -23 * (keys + 64)) * spread
        l_tol = s_err + 2.0 ** -23 * (64 + np.where(np.isfinite(wl), np.abs(wl), 0)) * 4
        fine = np.isfinite(wl)
        assert (np.isneginf(l[b]) == np.isneginf(wl)).all()
        l_err = np.abs(l[b][fine] - wl[fine])
        assert (l_err <= np.broadcast_to(l_tol, wl.shape)[fine]).all(), l_err.max()
        assert (np.abs(o[b] - wo) <= tol + 1e-30).all(), (np.abs(o[b] - wo) / (tol + 1e-30)).max()


def run(st, path="auto", **kw):
    mp = kw.pop("max_prefix_len", max(max(st["P"]), 1))
    out, lse = tidar.step_attn_kv4(st["q"], st["k_blk"], st["v_blk"], st["cache"], st["k"], max_prefix_len=mp, path=path, **kw)
    assert tidar.device_status() == (tidar.OK, 0)
    return out, lse


def paths(k, G, D, dtype):
    """Every kernel family that takes the shape."""
    d = tidar.StepDesc(batch=1, num_q_heads=G, num_kv_heads=1, head_dim=D, k=k, page_size=64, max_prefix_len=64,
                       dtype=tidar.BF16 if dtype == "bf16" else tidar.F32, softmax_scale=0.0, path=0)
    got = ["simt"]
    for name in ("dec", "tc05"):
        d.path = tidar._PATHS[name]
        try:
            tidar.kv4_plan(d)
            got.append(name)
        except tidar.TidarError:
            pass
    return got


SHAPES = [  # P, Hq, H, D, k, ps, dtype
    ([0], 2, 2, 64, 0, 16, "f32"), ([0, 1, 63, 64, 65], 4, 2, 64, 4, 64, "f32"), ([256], 2, 2, 64, 4, 64, "f32"),
    ([17, 300], 2, 1, 128, 2, 32, "f32"),
    ([0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129], 4, 1, 128, 0, 16, "bf16"),
    ([200, 77, 0], 8, 2, 128, 0, 64, "bf16"), ([1000, 300], 16, 1, 128, 0, 128, "bf16"), ([333], 8, 8, 128, 0, 32, "bf16"),
    ([130, 5, 1], 12, 2, 128, 1, 64, "bf16"), ([500], 16, 2, 128, 1, 16, "bf16"),
    ([0, 1, 63, 64, 65, 128, 200], 8, 2, 128, 4, 64, "bf16"), ([300, 10], 4, 4, 128, 4, 16, "bf16"),
    ([900], 12, 2, 128, 8, 32, "bf16"), ([257, 640], 8, 2, 128, 16, 64, "bf16"), ([190], 16, 1, 128, 2, 128, "bf16"),
    ([77, 200], 4, 2, 64, 4, 64, "bf16"),
]


@pytest.mark.parametrize("P,Hq,H,D,k,ps,dtype", SHAPES, ids=lambda v: str(v).replace(" ", ""))
def test_every_path(P, Hq, H, D, k, ps, dtype):
    st = make(len(P) + k, P, Hq, H, D, k, ps, dtype, stale="ff")
    before = {n: st["cache"][n].clone() for n in ("k_pages", "v_pages")}
    for path in paths(k, Hq // H, D, dtype):
        compare(st, *run(st, path, append=False))
        for n in before:
            assert torch.equal(before[n], st["cache"][n])


@pytest.mark.parametrize("force", [0, 1])
@pytest.mark.parametrize("P,Hq,H,k,ps", [([8192], 32, 8, 0, 64), ([5000, 130, 0], 8, 2, 0, 16), ([4096], 16, 2, 1, 128),
                                         ([4100], 8, 1, 4, 64), ([3000, 64], 12, 2, 8, 32), ([8192], 8, 2, 16, 64)])
def test_splits_merge_both_ways(P, Hq, H, k, ps, force):
    st = make(7, P, Hq, H, 128, k, ps, "bf16", stale="nan")
    tidar.debug_set(tidar.DEBUG_FORCE_SPLIT_PARTIALS, force)
    try:
        for path in paths(k, Hq // H, 128, "bf16"):
            compare(st, *run(st, path, append=False))
    finally:
        tidar.debug_set(tidar.DEBUG_FORCE_SPLIT_PARTIALS, 0)


@pytest.mark.parametrize("q_scale", [0.0, 8.0, 60.0])
@pytest.mark.parametrize("k", [0, 4])
def test_flat_and_peaked_scores(k, q_scale):
    st = make(11, [700, 90], 8, 2, 128, k, 64, "bf16", q_scale=q_scale)
    for path in paths(k, 4, 128, "bf16"):
        compare(st, *run(st, path))


@pytest.mark.parametrize("k,ps,dtype,D", [(0, 16, "bf16", 128), (1, 64, "bf16", 128), (4, 64, "bf16", 128),
                                          (16, 16, "bf16", 128), (4, 32, "f32", 64), (8, 128, "bf16", 64)])
def test_append_stores_the_drafts(k, ps, dtype, D):
    st = make(13, [0, 15, 64, 130], 4, 2, D, k, ps, dtype, stale="ff")
    n = max(k, 1)
    base = {m: st["cache"][m].clone() for m in ("k_pages", "v_pages")}
    slots = np.array([[int(st["table"][b, pos // ps]) * ps + pos % ps for pos in range(p, p + n)] for b, p in enumerate(st["P"])])
    want = dict(k_pages=base["k_pages"].clone(), v_pages=base["v_pages"].clone())
    tidar.kv4_append(want, st["k_blk"][:, :n].reshape(-1, 2, D).contiguous(), st["v_blk"][:, :n].reshape(-1, 2, D).contiguous(),
                     torch.from_numpy(slots.reshape(-1)).cuda())
    for path in paths(k, 2, D, dtype):
        for m in base:
            st["cache"][m].copy_(base[m])
        compare(st, *run(st, path))
        for m in base:
            assert torch.equal(st["cache"][m], want[m]), (path, m)


def test_prefix_only_and_empty_slices():
    st = make(17, [0, 90, 200], 8, 2, 128, 4, 64, "bf16")
    for path in paths(4, 4, 128, "bf16"):
        out, lse = run(st, path, step_keys=False, append=False)
        assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
        compare(st, out, lse, step_keys=False)
    st = make(18, [0, 90], 8, 2, 128, 0, 64, "bf16")
    for path in paths(0, 4, 128, "bf16"):
        out, lse = run(st, path, step_keys=False, append=False)
        assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
        compare(st, out, lse, step_keys=False)


def test_agrees_with_the_bf16_cache_of_the_same_values():
    # the values are exact in bf16: step_attn on them differs by roundings of p and of the sums only
    for k in (0, 4):
        st = make(19, [300, 700], 8, 2, 128, k, 64, "bf16")
        c = st["cache"]
        pages = [torch.from_numpy(kv4_ref.unpack(c[m].cpu().numpy(), 64, 128, key)).to(torch.bfloat16).contiguous().cuda()
                 for m, key in (("k_pages", True), ("v_pages", False))]
        wide = dict(c, k_pages=pages[0], v_pages=pages[1])
        a = run(st, append=False)
        b = tidar.step_attn(st["q"], st["k_blk"], st["v_blk"], wide, k, max_prefix_len=700)
        compare(st, *a)
        compare(st, *b)


def test_nan_and_infinite_rows_reach_their_sequence_only():
    st = make(23, [100, 100], 4, 2, 128, 0, 64, "bf16")
    page = int(st["table"][1, 0])
    at = 64 * 64
    st["cache"]["k_pages"][page, 0, at + 8 * 5 + 1] = 0x7f          # scale of row 5, head 0: a NaN
    st["cache"]["k_pages"][page, 0, at + 8 * 5] = 0xc0
    for path in paths(0, 2, 128, "bf16"):
        out, lse = run(st, path, append=False)
        assert torch.isnan(out[1, :, :2]).all() and not torch.isnan(out[1, :, 2:]).any() and not torch.isnan(out[0]).any()
        compare(st, out, lse, seqs=[0])


@pytest.mark.parametrize("force", [0, 1])
@pytest.mark.parametrize("k", [0, 4])
def test_nan_survives_the_merge_of_splits(k, force):
    st = make(41, [4096, 4096], 8, 2, 128, k, 64, "bf16")
    page = int(st["table"][1, 20])
    st["cache"]["v_pages"][page, 1, 64 * 64 + 1] = 0x7f             # a value scale of row 0, head 1, first group: a NaN
    st["cache"]["v_pages"][page, 1, 64 * 64] = 0xc0
    page = int(st["table"][0, 40])
    st["cache"]["k_pages"][page, 0, 64 * 64 + 1] = 0x7f             # a key scale of head 0
    st["cache"]["k_pages"][page, 0, 64 * 64] = 0xc0
    tidar.debug_set(tidar.DEBUG_FORCE_SPLIT_PARTIALS, force)
    try:
        for path in paths(k, 4, 128, "bf16"):
            out, lse = run(st, path, append=False)
            nan = torch.isnan(out)
            assert nan[1, :, 4:, :32].all() and not nan[1, :, 4:, 32:].any() and not nan[1, :, :4].any(), path
            assert nan[0, :, :4].all() and torch.isnan(lse[0, :, :4]).all() and not nan[0, :, 4:].any(), path
            assert not torch.isnan(lse[1]).any() and not torch.isnan(lse[0, :, 4:]).any(), path
    finally:
        tidar.debug_set(tidar.DEBUG_FORCE_SPLIT_PARTIALS, 0)


def test_device_errors_skip_their_work():
    for k in (0, 4):
        for path in paths(k, 4, 128, "bf16"):
            st = make(29, [100, 100, 100], 8, 2, 128, k, 64, "bf16")
            st["cache"]["page_table"][1, 0] = -1
            st["cache"]["seq_lens"][2] = 101
            out, lse = tidar.step_attn_kv4(st["q"], st["k_blk"], st["v_blk"], st["cache"], k, max_prefix_len=100, path=path)
            status, bits = tidar.device_status()
            assert status == tidar.ERR_DEVICE and bits == tidar.DEVERR_BAD_PAGE | tidar.DEVERR_BAD_LEN, (path, bits)
            assert torch.isfinite(out).all()
            compare(st, out, lse, seqs=[0])
            assert torch.equal(st["cache"]["seq_lens"].cpu(), torch.tensor([100, 100, 101], dtype=torch.int32))


def test_bindings_checks():
    st = make(31, [10], 4, 2, 128, 0, 64, "bf16")
    c = st["cache"]
    call = lambda q=st["q"], kb=st["k_blk"], cache=c, **kw: tidar.step_attn_kv4(q, kb, st["v_blk"], cache, 0,  # noqa: E731
                                                                                 max_prefix_len=10, **kw)
    for bad in (dict(q=st["q"].float()), dict(kb=st["k_blk"][:, :, :1]), dict(cache=dict(c, k_pages=c["k_pages"][:, :1])),
                dict(cache=dict(c, k_pages=c["k_pages"].view(torch.int8))), dict(lse=torch.zeros(1, device="cuda")),
                dict(cache=dict(c, seq_lens=c["seq_lens"].repeat(2))), dict(out=st["q"][..., :64])):
        with pytest.raises(ValueError):
            call(**bad)
    assert call(want_lse=False)[1] is None


def test_captured_replayed_and_on_another_stream():
    for k in (0, 4):
        st = make(37, [900, 333], 8, 2, 128, k, 64, "bf16")
        want = run(st, append=False)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = run(st, append=False, stream=side)
        out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
        need = tidar.step_attn_kv4_workspace_bytes(tidar.step_attn_kv4_desc(st["q"], st["k_blk"], st["cache"], k, 900))
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tidar.step_attn_kv4(st["q"], st["k_blk"], st["v_blk"], st["cache"], k, max_prefix_len=900, append=False, out=out,
                                lse=lse, workspace=ws)
        g.replay()
        first = out.clone()
        st["q"].mul_(0.5)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, want[0]) and torch.equal(other[0], want[0])
        assert not torch.equal(out, first)
        compare(st, out, lse)


def test_wait_timeout_is_reported_and_recovered():
    # the dequantising warps fill no block, so the bounded waits run out; the next call is right
    st = make(77, [300], 8, 2, 128, 2, 64, "bf16")
    tidar.debug_set(tidar.DEBUG_STARVE_ATTENTION_LOADS, 1)
    try:
        tidar.step_attn_kv4(st["q"], st["k_blk"], st["v_blk"], st["cache"], 2, max_prefix_len=300, path="tc05")
    finally:
        tidar.debug_set(tidar.DEBUG_STARVE_ATTENTION_LOADS, 0)
    status, bits = tidar.device_status()
    assert status == tidar.ERR_TIMEOUT and bits & tidar.DEVERR_TIMEOUT
    compare(st, *run(st, path="tc05"))


@pytest.mark.parametrize("k", [0, 4])
@pytest.mark.parametrize("magnitude", [2.0 ** 126 * (1 - 2.0 ** -8), 2.0 ** 100, 2.0 ** -100, 2.0 ** -120])
def test_values_at_the_ends_of_the_range_are_exact(k, magnitude):
    # one key: the output is its value row as it is, on every path
    H, D, ps = 2, 128, 16
    g = torch.Generator().manual_seed(3)
    row = torch.randint(-7, 8, (1, H, D), generator=g).float() / 7
    row[..., ::32] = 1.0                                  # every group's maximum
    v = (row * magnitude).bfloat16().cuda()
    cache = tidar.kv4_cache(2, H, ps, D, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                            torch.ones(1, dtype=torch.int32, device="cuda"))
    tidar.kv4_append(cache, torch.zeros_like(v), v, torch.zeros(1, dtype=torch.int64, device="cuda"))
    want = tidar.kv4_gather(cache, torch.zeros(1, dtype=torch.int64, device="cuda"), head_dim=D)[1]
    ref = kv4_ref.unpack(kv4_ref.pack(v.double().cpu().numpy()[0, :, None], False), 1, D, False)[:, 0]
    assert (want.double().cpu().numpy()[0] == ref).all() and (want != 0).any()
    R = 1 if k == 0 else k + k * k
    q = torch.randn(1, R, 2 * H, D, generator=g).bfloat16().cuda()
    blk = torch.zeros(1, R, H, D, dtype=torch.bfloat16, device="cuda")
    for path in paths(k, 2, D, "bf16"):
        out, _ = tidar.step_attn_kv4(q, blk, blk, cache, k, max_prefix_len=1, step_keys=False, append=False, path=path)
        assert torch.equal(out, want[0].repeat_interleave(2, 0).expand(1, R, 2 * H, D)), path
    assert tidar.device_status() == (tidar.OK, 0)


def test_offsets_past_32_bits():
    # pages at both ends of 4.7 GB a tensor; every path, append, read back and commit
    H, D, ps, pages = 2, 128, 128, 256000
    assert pages * H * tidar.kv4_page_bytes(ps, D) > 2 ** 32
    used = [pages - 1, 0, pages - 7]
    table = torch.tensor([used + [-1]], dtype=torch.int32, device="cuda")
    small = torch.tensor([[2, 0, 1, -1]], dtype=torch.int32, device="cuda")
    P, k = 300, 4
    caches = [tidar.kv4_cache(n, H, ps, D, t, torch.tensor([P], dtype=torch.int32, device="cuda"))
              for n, t in ((pages, table), (3, small))]
    g = torch.Generator(device="cuda").manual_seed(8)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    rows, pos = (rnd(P, H, D), rnd(P, H, D)), torch.arange(P, device="cuda")
    slots = [c["page_table"][0, pos // ps].long() * ps + pos % ps for c in caches]
    for c, s in zip(caches, slots):
        tidar.kv4_append(c, *rows, s)
    back = [tidar.kv4_gather(c, s, head_dim=D) for c, s in zip(caches, slots)]
    assert torch.equal(back[0][0], back[1][0]) and torch.equal(back[0][1], back[1][1]) and (back[0][0] != 0).any()
    for kk in (0, k):
        R = 1 if kk == 0 else kk + kk * kk
        q, kb, vb = rnd(1, R, 2 * H, D), rnd(1, R, H, D), rnd(1, R, H, D)
        for path in paths(kk, 2, D, "bf16"):
            got = [tidar.step_attn_kv4(q, kb, vb, c, kk, max_prefix_len=P, path=path) for c in caches]
            assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]), path
    for c in caches:
        tidar.commit_kv4(c, torch.ones(1, dtype=torch.int32, device="cuda"), k, head_dim=D, max_prefix_len=P)
    for n in ("k_pages", "v_pages"):
        assert torch.equal(caches[0][n][torch.tensor(used, device="cuda")], caches[1][n][torch.tensor([2, 0, 1], device="cuda")])
        assert not caches[0][n][1:pages - 7].any()         # nothing went anywhere else
    assert tidar.device_status() == (tidar.OK, 0)


@pytest.mark.parametrize("k", [0, 1, 2, 4])
def test_many_calls_whose_append_leaves_lanes_idle(k):
    # 2n units of four lanes: with n = 1 or 2 most lanes of the warp that releases the
    # tensor memory store nothing.  As many calls as several rounds of the device's SMs,
    # each of which has to find all of it free again.
    st = make(61, [40] * 24, 8, 4, 128, k, 64, "bf16")
    want = run(st, "tc05")
    for _ in range(40):
        got = run(st, "tc05", append=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    compare(st, *got, seqs=[0, 23])


def compare_by_path(st, out, lse, path):
    """compare() with what each kernel's own arithmetic warrants: the codes' offset of 136,
    which widens compare()'s score term by 143/7, is the decode kernel's alone, and the
    CUDA-core kernel rounds no p.  Sums over the keys add 2^-23 a step (16 keys a step in
    the matrix products) of sum p|v|."""
    D = st["D"]
    q, kb, vb = (st[n].double().cpu().numpy() for n in ("q", "k_blk", "v_blk"))
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(len(st["P"])):
        wo, wl, spread, mag = kv4_ref.attention(q[b], kb[b], vb[b], st["pref"][0][b], st["pref"][1][b], st["k"])
        keys = st["P"][b] + q.shape[1]
        s_err = (D / 16 + 8) * 2.0 ** -23 * mag * (143 / 7 if path == "dec" else 1)
        steps = keys if path == "simt" else keys / 16
        tol = (2 * s_err + 2.0 ** -23 * (steps + 64)) * spread
        if st["dtype"] == "bf16":
            tol = tol + 2.0 ** -8 * np.abs(wo) + (0 if path == "simt" else 2.0 ** -8 * spread)
        l_tol = s_err + 2.0 ** -23 * (64 + np.abs(wl)) * 4
        assert (np.abs(l[b] - wl) <= l_tol).all(), (path, (np.abs(l[b] - wl) / l_tol).max())
        assert (np.abs(o[b] - wo) <= tol + 1e-30).all(), (path, (np.abs(o[b] - wo) / (tol + 1e-30)).max())


@pytest.mark.parametrize("q_scale", [1.0, 30.0])
@pytest.mark.parametrize("P,Hq,H,D,k,ps,dtype", SHAPES, ids=lambda v: str(v).replace(" ", ""))
def test_every_path_to_its_own_tolerance(P, Hq, H, D, k, ps, dtype, q_scale):
    st = make(67 + len(P) + k, P, Hq, H, D, k, ps, dtype, q_scale=q_scale, stale="ff")
    for path in paths(k, Hq // H, D, dtype):
        compare_by_path(st, *run(st, path, append=False), path)
