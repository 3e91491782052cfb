"""tidar_build_tables against its definition (integers: exact)."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import ar_decoding_b200 as tidar
import kv4_ref

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def state(seed, B, ps, ctx_hi, new_hi, width=None, spare=5, kept=0.0):
    """Tables whose rows hold ctx pages, some of the new entries already mapped."""
    r = np.random.default_rng(seed)
    ctx, new = r.integers(0, ctx_hi + 1, B), r.integers(0, new_hi + 1, B)
    width = width or -(-(ctx_hi + new_hi) // ps) + 1
    have, need = -(-ctx // ps), -(-(ctx + new) // ps)
    total = int(need.sum()) + spare
    ids = r.permutation(total)
    table, at = np.full((B, width), -1), 0
    for b in range(B):
        for e in range(need[b]):
            if e < have[b] or r.random() < kept:
                table[b, e] = ids[at]
                at += 1
    return dict(table=table.astype(np.int32), ctx=ctx, new=new, free=ids[at:].astype(np.int32), num_pages=total)


def check(st, ps, max_rows, in_place=False, count=None, stream=None):
    count = len(st["free"]) if count is None else count
    want = kv4_ref.tables(st["table"], st["ctx"], st["new"], st["free"], count, ps, st["num_pages"], max_rows)
    table, pool = dev(st["table"]), dict(free_pages=dev(st["free"]), free_count=dev([count]))
    out = dict(page_table=table, free_count=pool["free_count"]) if in_place else None
    torch.cuda.synchronize()
    got = tidar.build_tables(table, dev(st["ctx"]), dev(st["new"]), pool, page_size=ps, num_pages=st["num_pages"],
                             max_rows=max_rows, out=out)
    bits = tidar.device_status()[1]
    assert bits == want[5]
    for name, w in zip(("page_table", "free_count", "row_starts", "slots", "positions"), want):
        np.testing.assert_array_equal(got[name].cpu().numpy().reshape(-1), np.asarray(w).reshape(-1), err_msg=name)
    assert (pool["free_pages"].cpu().numpy() == st["free"]).all()
    if not in_place:
        assert (table.cpu().numpy() == st["table"]).all() and int(pool["free_count"]) == count
    return got


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("B,ctx,new", [(1, 0, 1), (1, 0, 0), (1, 4000, 3000), (3, 100, 17), (33, 0, 700), (130, 900, 16),
                                       (700, 40, 3)])
def test_matches_definition(B, ctx, new, ps):
    for seed in range(2):
        st = state(seed, B, ps, ctx, new, kept=0.3 * seed)
        check(st, ps, int(st["new"].sum()) + seed, in_place=bool(seed))


def test_large_batch_and_odd_width():
    st = state(5, 9000, 16, 5, 3, width=3)                  # past the starts kept in shared memory
    check(st, 16, int(st["new"].sum()) + 1)


def test_one_long_sequence():
    st = state(6, 1, 16, 0, 131072)
    st["new"][:] = 131072
    st = dict(st, free=np.arange(8200, dtype=np.int32)[::-1].copy(), num_pages=8200)
    check(st, 16, 131072)


def test_bad_lengths_and_entries_skip_their_sequence():
    st = state(1, 6, 16, 60, 40, kept=0.0)
    st["ctx"][0], st["new"][1], st["ctx"][2] = -3, -1, 10 ** 6
    st["ctx"][3], st["new"][3] = 20, 30
    st["table"][3, :] = [7, -1] + [-1] * (st["table"].shape[1] - 2)      # rows below ctx unmapped
    st["ctx"][4], st["new"][4] = 0, 30
    st["table"][4, 1] = -5
    check(st, 16, 400)


def test_pool_and_row_limits_change_nothing():
    st = state(2, 5, 16, 0, 90)
    need = len(st["free"]) - 5
    check(st, 16, 500, count=need)                    # just enough
    for in_place in (False, True):
        check(st, 16, 500, count=need - 1, in_place=in_place)
        check(st, 16, int(st["new"].sum()) - 1, in_place=in_place)
    check(st, 16, 500, count=-1)
    check(st, 16, 500, count=len(st["free"]) + 1)
    check(st, 16, 0)


def test_popped_id_out_of_range_is_reported():
    st = state(3, 2, 16, 0, 40)
    st["new"][:] = 40
    st["free"] = np.array([0, 1, 2, 3, 4, 999, 5, 6], dtype=np.int32)
    st["num_pages"] = 8
    check(st, 16, 100)


def test_empty_batch_is_a_noop():
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    pool = dict(free_pages=dev([1]), free_count=dev([1]))
    out = tidar.build_tables(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), z, z, pool, page_size=16, num_pages=2,
                             max_rows=4)
    assert out["page_table"].shape == (0, 4) and tidar.device_status() == (tidar.OK, 0)


def test_empty_batch_has_no_rows():
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    pool = dict(free_pages=dev([1, 0]), free_count=dev([2]))
    torch.full((64,), 7, device="cuda")                  # what the call is given to allocate is not zeros
    out = tidar.build_tables(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), z, z, pool, page_size=16, num_pages=2,
                             max_rows=5)
    assert out["free_count"].tolist() == [2] and out["row_starts"].tolist() == [0]
    assert out["slots"].tolist() == [-1] * 5 and out["positions"].tolist() == [-1] * 5
    cache = tidar.kv4_cache(2, 2, 16, 64, out["page_table"], z)
    assert tidar.commit_kv4(cache, z, 4, head_dim=64, max_prefix_len=16, num_released=dev([9]))[1].tolist() == [0]
    assert tidar.device_status() == (tidar.OK, 0)


def test_captured_and_on_another_stream():
    st = state(4, 40, 16, 200, 30)
    rows = int(st["new"].sum()) + 3
    args = (dev(st["table"]), dev(st["ctx"]), dev(st["new"]))
    pool = dict(free_pages=dev(st["free"]), free_count=dev([len(st["free"])]))
    kw = dict(page_size=16, num_pages=st["num_pages"], max_rows=rows)
    want = tidar.build_tables(*args, pool, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = tidar.build_tables(*args, pool, **kw, stream=side)
    g, out = torch.cuda.CUDAGraph(), {k: torch.zeros_like(v) for k, v in want.items()}
    with torch.cuda.graph(g):
        tidar.build_tables(*args, pool, **kw, out=out)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(want[k], other[k]) and torch.equal(want[k], out[k]), k


@pytest.mark.parametrize("sizes", [((4, 250000), (4, 205000)), ((60000, 60000), (20000, 20000))])
def test_two_host_threads_and_two_sizes_of_shared_memory(sizes):
    # Both sizes of a pair take more shared memory than a launch gets unasked (48 KB):
    # 15633 and 12821 table entries in the one-launch form, 7500 and 2500 sequences a CTA
    # in the other.  Two threads call the library at once, each on its own stream and
    # with its own results; no call may depend on what the other's asked for.
    def inputs(B, rows):
        ps, each = 16, rows // B
        need, width = B * -(-each // ps), -(-each // ps) + 1
        t = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        pool = dict(free_pages=torch.arange(need, dtype=torch.int32, device="cuda"), free_count=dev([need]))
        ctx, new = dev(np.zeros(B)), dev(np.full(B, each))
        kw = dict(page_size=ps, num_pages=need, max_rows=B * each)
        want = tidar.build_tables(t, ctx, new, pool, **kw)
        out = {n: torch.empty_like(w) for n, w in want.items()}
        d = tidar.TablesDesc(B, ps, need, width, B * each)
        p = tidar.PagePool(pool["free_pages"].data_ptr(), pool["free_count"].data_ptr(), need)

        def raw(stream):                                   # the call alone, as another language's program makes it
            return tidar.lib().tidar_build_tables(
                ctypes.byref(d), t.data_ptr(), ctx.data_ptr(), new.data_ptr(), ctypes.byref(p),
                *(out[n].data_ptr() for n in ("page_table", "free_count", "row_starts", "slots", "positions")), stream)
        raw.keep = (t, pool, ctx, new)
        return raw, out, want, lambda: tidar.build_tables(t, ctx, new, pool, **kw)

    calls = [inputs(*s) for s in sizes]
    torch.cuda.synchronize()
    status, start = [set(), set()], threading.Barrier(2)

    def work(i):
        stream = torch.cuda.Stream()
        start.wait()
        for _ in range(10000):
            status[i].add(calls[i][0](stream.cuda_stream))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert status == [{tidar.OK}, {tidar.OK}], status
    for _, out, want, _ in calls:
        assert all(torch.equal(out[n], want[n]) for n in want)
    # and both in one graph, the smaller last
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = [c[3]() for c in calls]
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a[n], c[2][n]) for a, c in zip(got, calls) for n in a)
    assert tidar.device_status() == (tidar.OK, 0)
