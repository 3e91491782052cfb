"""The serving operators together, as a decode loop over a 4-bit cache uses them:
admission (page tables, slots, the prompts' rows stored), then steps of reserve ->
projection and rotation -> step attention -> output projection with the residual
-> MLP -> verification -> commit, eagerly and as one captured graph."""
import numpy as np
import pytest
import torch

import ar_decoding_b200 as tidar
import kv4_ref

pytestmark = pytest.mark.gpu

HQ, HKV, D, DM, PS, K, V, STEPS = 8, 2, 128, 256, 32, 4, 512, 3


def weights(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = lambda n, k: (torch.randn(n, k, generator=g, device="cuda") / k ** 0.5).bfloat16()  # noqa: E731
    return dict(qkv=w((HQ + 2 * HKV) * D, DM), o=w(DM, HQ * D), up=w(4 * DM, DM), down=w(DM, 4 * DM),
                bias=torch.randn(4 * DM, generator=g, device="cuda").bfloat16())


def admit(prompts, seed):
    """Tables, slots and stored rows of the prompts."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, total = len(prompts), sum(prompts)
    pages = sum(-(-p // PS) for p in prompts) + 4 * B
    width = -(-(max(prompts) + K * (STEPS + 1)) // PS) + 1
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    pool = dict(free_pages=torch.randperm(pages, generator=g, device="cuda").int(),
                free_count=torch.tensor([pages], dtype=torch.int32, device="cuda"))
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    free = pool["free_pages"].cpu().numpy()
    t = tidar.build_tables(table, torch.zeros_like(lens), lens, pool, page_size=PS, num_pages=pages, max_rows=total + 5)
    want = kv4_ref.tables(table.cpu().numpy(), [0] * B, prompts, free, pages, PS, pages, total + 5)
    for name, w in zip(("page_table", "free_count", "row_starts", "slots", "positions"), want):
        np.testing.assert_array_equal(t[name].cpu().numpy().reshape(-1), np.asarray(w).reshape(-1), err_msg=name)
    cache = tidar.kv4_cache(pages, HKV, PS, D, t["page_table"], lens)
    kv = torch.randn(total + 5, 2 * HKV, D, generator=g, device="cuda").bfloat16()
    tidar.kv4_append(cache, kv[:, :HKV], kv[:, HKV:], t["slots"])      # the 5 rows of padding have slot -1
    return cache, dict(pool, free_count=t["free_count"]), kv


def step(w, cache, pool, x, logits, drafts, released, num, mp):
    B, R = x.shape[:2]
    tidar.reserve(cache, pool, K, max_prefix_len=mp, head_dim=D, returned=released, num_returned=num)
    q, kb, vb = tidar.qkv_rope(x, w["qkv"], cache["seq_lens"], K, HQ, HKV, max_prefix_len=mp)
    a, lse = tidar.step_attn_kv4(q, kb, vb, cache, K, max_prefix_len=mp)
    h = tidar.linear_fused(a.view(B, R, HQ * D), w["o"], residual=x)
    u = tidar.linear_fused(h, w["up"], bias=w["bias"], activation="gelu_tanh")
    y = tidar.linear_fused(u, w["down"], residual=h, out=h)
    res = tidar.verify(logits, drafts, K, "greedy")
    rel, nrel = tidar.commit_kv4(cache, res["accept_count"], K, head_dim=D, max_prefix_len=mp)
    return dict(q=q, k_blk=kb, v_blk=vb, a=a, lse=lse, y=y, acc=res["accept_count"], rel=rel, num=nrel)


def inputs(B, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    R = K + K * K
    x = torch.randn(B, R, DM, generator=g, device="cuda").bfloat16()
    logits = torch.randn(B, K, V, generator=g, device="cuda").bfloat16()
    drafts = torch.randint(0, V, (B, K), generator=g, device="cuda", dtype=torch.int32)
    best = logits.float().argmax(-1).int()
    hit = torch.rand(B, K, generator=g, device="cuda") < 0.7
    drafts[:, 1:] = torch.where(hit[:, 1:], best[:, :-1], drafts[:, 1:])
    return x, logits, drafts


def check_attention(r, before):
    """The step's attention against the reference on the rows that the cache held before it."""
    B = r["q"].shape[0]
    lens, table = before["seq_lens"].tolist(), before["page_table"].cpu().numpy()
    for b in range(B):
        rows = torch.tensor([int(table[b, p // PS]) * PS + p % PS for p in range(lens[b])], device="cuda", dtype=torch.int64)
        pk, pv = tidar.kv4_gather(before, rows, head_dim=D, dtype=torch.float32)
        n = lambda t: t.double().cpu().numpy()  # noqa: E731
        o, lse, spread, mag = kv4_ref.attention(n(r["q"][b]), n(r["k_blk"][b]), n(r["v_blk"][b]), n(pk), n(pv), K)
        err = (D / 16 + 8) * 2.0 ** -23 * mag * 143 / 7
        assert (np.abs(n(r["a"][b]) - o) <= 2.0 ** -8 * (np.abs(o) + spread) + 2 * err * spread + 1e-30).all()
        assert np.abs(n(r["lse"][b]) - lse).max() <= err + 2.0 ** -19 * (1 + np.abs(lse).max())


def test_loop_eager_and_captured():
    prompts = [70, 1, 33]
    B, mp = len(prompts), 70 + K * STEPS
    w = weights(1)
    cache, pool, _ = admit(prompts, 2)
    copy = lambda d: {k: v.clone() for k, v in d.items()}  # noqa: E731
    start, start_pool = copy(cache), copy(pool)
    ins = [inputs(B, 10 + i) for i in range(STEPS)]
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    rel, num = torch.full((B * 2,), -1, dtype=torch.int32, device="cuda"), none
    eager = []
    for x, logits, drafts in ins:
        before = copy(cache)
        r = step(w, cache, pool, x, logits, drafts, rel, num, mp)
        assert tidar.device_status() == (tidar.OK, 0)
        check_attention(r, before)
        lens = before["seq_lens"] + r["acc"]
        assert torch.equal(cache["seq_lens"], lens)
        rel, num = r["rel"], r["num"]
        eager.append(r)
    assert any(int(r["num"]) for r in eager) or any((r["acc"] < K).any() for r in eager)

    # the same steps as one graph, on a copy of the state
    gc, gp = copy(start), copy(start_pool)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                  # workspaces of this stream's pool, first-call attributes
        step(w, copy(start), copy(start_pool), *ins[0], torch.full((B * 2,), -1, dtype=torch.int32, device="cuda"), none, mp)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    rel0, num0 = torch.full((B * 2,), -1, dtype=torch.int32, device="cuda"), none.clone()
    captured = []
    with torch.cuda.graph(g):
        rel, num = rel0, num0
        for x, logits, drafts in ins:
            r = step(w, gc, gp, x, logits, drafts, rel, num, mp)
            rel, num = r["rel"], r["num"]
            captured.append(r)
    for _ in range(2):
        for k in gc:
            gc[k].copy_(start[k])
        for k in gp:
            gp[k].copy_(start_pool[k])
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, captured):
            for k in a:
                assert torch.equal(a[k], b[k]), k
        for k in gc:
            assert torch.equal(gc[k], cache[k]), k
        for k in gp:
            assert torch.equal(gp[k], pool[k]), k
    assert tidar.device_status() == (tidar.OK, 0)


def test_two_graphs_with_their_own_workspaces_overlap():
    """Two captured steps on two streams, each with its own outputs and workspaces."""
    w = weights(3)
    runs = []
    for i in range(2):
        cache, pool, _ = admit([50 + i, 20], 5 + i)
        x, logits, drafts = inputs(2, 20 + i)
        q, kb, vb = tidar.qkv_rope(x, w["qkv"], cache["seq_lens"], K, HQ, HKV, max_prefix_len=80)
        tidar.reserve(cache, pool, K, max_prefix_len=80, head_dim=D)
        runs.append((cache, q, kb, vb))
    call = lambda c, q, kb, vb: tidar.step_attn_kv4(q, kb, vb, c, K, max_prefix_len=80, append=False)  # noqa: E731
    want = [call(*r) for r in runs]
    torch.cuda.synchronize()
    streams, graphs, outs = [torch.cuda.Stream() for _ in runs], [], []
    for s, r in zip(streams, runs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(call(*r))
        graphs.append(g)
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, outs):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
