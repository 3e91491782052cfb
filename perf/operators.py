"""What is measured of the serving operators: page tables and slot maps built from request lengths, the cache
held in 4 bits (its store and read-back, and the step attention over it) and the projection with bias,
activation and residual in its epilogue.

Every case can be run two ways: `own = False` computes it in elementary torch operations in 32 bits, `own = True`
makes the calls that a user of ar_decoding_b200 makes.  `exact` computes it in 64 bits, written apart from both.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
GROUP = 32          # dims that share a scale in the 4-bit cache


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # Admission of the serving batch: 32 prompts of 512..16384 tokens get their pages, every prompt token its slot.
        dict(name="tables-admit", op="tables", batch=32, lo=512, hi=16384, ctx=0, page_size=64),
        # One decode step's rows for a large running batch: 1..16 new rows on top of long contexts, few new pages.
        dict(name="tables-step", op="tables", batch=256, lo=1, hi=16, ctx=16384, page_size=64),
        # The K/V rows of one 8192-token prompt (8 KV heads of 128) stored in 4 bits and read back for its own chunks.
        dict(name="store-prompt", op="store", rows=8192, hkv=8, d=128, dtype="bf16", page_size=64, skip=0.0),
        # A ragged, padded batch of fp32 rows with small pages: rows whose slot is -1 are padding.
        dict(name="store-ragged-f32", op="store", rows=1237, hkv=2, d=64, dtype="f32", page_size=16, skip=0.05),
        # Plain decode of one sequence at the 8B-class prefix: the smallest call, where latency counts.
        dict(name="attn-decode", op="attn", batch=1, hq=32, hkv=8, d=128, k=0, lo=8192, hi=8192, dtype="bf16",
             page_size=64, append=False),
        # Plain decode of the ragged serving batch: a stream of the whole cache.
        dict(name="attn-decode-serving", op="attn", batch=32, hq=32, hkv=8, d=128, k=0, lo=512, hi=16384, dtype="bf16",
             page_size=64, append=False),
        # The 8B-class step: 272 rows (16 drafts, 16 blocks of 16 mask slots) against 8192 cached keys.
        dict(name="attn-step-k16", op="attn", batch=1, hq=32, hkv=8, d=128, k=16, lo=8192, hi=8192, dtype="bf16",
             page_size=64, append=False),
        # The serving batch's step at k = 8, its drafts stored in the cache as it runs: the largest attention.
        dict(name="attn-step-serving", op="attn", batch=32, hq=32, hkv=8, d=128, k=8, lo=512, hi=16384, dtype="bf16",
             page_size=64, append=True),
        # The tiny fp32 workload.
        dict(name="attn-tiny-f32", op="attn", batch=1, hq=2, hkv=2, d=64, k=4, lo=256, hi=256, dtype="f32",
             page_size=64, append=True),
        # The output projection of the 8B-class step with the residual stream added.
        dict(name="linear-out", op="linear", rows=272, n=4096, kdim=4096, act="none", bias=False, residual=True),
        # The first MLP product of a 2048-token prompt chunk: bias and tanh GELU, four times the hidden size.
        dict(name="linear-up-prompt", op="linear", rows=2048, n=16384, kdim=4096, act="gelu_tanh", bias=True,
             residual=False),
        # An odd-sized product with everything in its epilogue (the 1.5B-class hidden size on one side).
        dict(name="linear-odd", op="linear", rows=77, n=1000, kdim=1544, act="silu", bias=True, residual=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "store", "attn", "attn", "linear", "linear"])
    if op == "tables":
        batch = _log_int(rng, 1, 256)
        if rng.random() < 0.5:      # admission: whole prompts
            hi = _log_int(rng, 16, 16384)
            hi = max(1, min(hi, 32 * 16384 // batch))
            return dict(op=op, batch=batch, lo=rng.randint(0, hi), hi=hi, ctx=0, page_size=rng.choice([16, 32, 64, 128]))
        return dict(op=op, batch=batch, lo=0, hi=rng.randint(1, 16), ctx=_log_int(rng, 1, 16384),
                    page_size=rng.choice([16, 32, 64, 128]))
    if op == "store":
        f32 = rng.random() < 0.3
        return dict(op=op, rows=_log_int(rng, 1, 4096 if f32 else 8192), hkv=rng.choice([1, 2, 4, 8] if not f32 else [1, 2, 4]),
                    d=rng.choice([64, 128]), dtype="f32" if f32 else "bf16", page_size=rng.choice([16, 32, 64, 128]),
                    skip=rng.choice([0.0, 0.0, 0.1]))
    if op == "attn":
        if rng.random() < 0.2:      # the fp32 class
            hkv = rng.choice([1, 2, 4])
            hi = _log_int(rng, 1, 1024)
            return dict(op=op, batch=rng.randint(1, 4), hq=hkv * rng.choice([1, 2]), hkv=hkv, d=64, k=rng.choice([0, 1, 4]),
                        lo=rng.randint(0, hi), hi=hi, dtype="f32", page_size=rng.choice([16, 32, 64, 128]),
                        append=rng.random() < 0.5)
        hkv, g = rng.choice([(8, 4), (2, 6), (8, 1), (4, 8), (1, 16), (4, 4)])
        k = rng.choice([0, 0, 1, 2, 4, 8, 16])
        batch = _log_int(rng, 1, 32)
        hi = _log_int(rng, 16, 131072)
        rows = 1 if k == 0 else k + k * k
        # neither more keys nor more row-key products than the serving cases
        hi = max(16, min(hi, 32 * 8448 * 8 // (batch * hkv), 72 * 32 * 32 * 8448 // (batch * rows * hkv * g)))
        return dict(op=op, batch=batch, hq=hkv * g, hkv=hkv, d=128, k=k, lo=rng.randint(0, hi), hi=hi, dtype="bf16",
                    page_size=rng.choice([16, 32, 64, 64, 64, 128]), append=rng.random() < 0.5)
    n, kdim = _log_int(rng, 8, 16384), 8 * _log_int(rng, 8, 1024)
    rows = max(1, min(_log_int(rng, 1, 4096), 2048 * 16384 * 4096 // (n * kdim)))
    return dict(op=op, rows=rows, n=n, kdim=kdim, act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                bias=rng.random() < 0.6, residual=rng.random() < 0.5)


def _lengths(case, seed):
    """Lengths lo..hi, one for each sequence, the same for one case and seed wherever they are asked."""
    r = np.random.default_rng(seed)
    return r.integers(case["lo"], case["hi"] + 1, case["batch"])


def _row_buffer(case):
    """Rows of the token buffer that a program of such batches allocates: their mean total and four deviations."""
    mean, dev = (case["lo"] + case["hi"]) / 2, (case["hi"] - case["lo"]) / math.sqrt(12)
    return 1 + min(case["batch"] * case["hi"], math.ceil(case["batch"] * mean + 4 * math.sqrt(case["batch"]) * dev))


def _typed(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


# ------------------------------------------------------------------ the 4-bit page, in torch
# A page of one KV head is page_size rows of D/2 bytes of codes, then page_size rows of D/32 bf16 scales.
# Code c of dim d = 32 G + 8 y + 2 i + h (G < D/32, y < 4, i < 4, h < 2) is a 4-bit two's-complement integer, nibble i
# (lowest first) of the 16-bit unit number  y D/16 + 2 G + h  of a key row,  y D/16 + h D/32 + G  of a value row.
def _quantise(x):
    """Codes (int32) and scales (fp32) of rows x [..., D]: s = max|x| / 7 rounded to 5 significant bits."""
    v = x.float().reshape(*x.shape[:-1], -1, GROUP)
    top = v.abs().amax(-1)
    bits = (top / 7).view(torch.int32)
    bits = (bits + 0x3FFFF + ((bits >> 19) & 1)) & ~0x7FFFF
    s = bits.view(torch.float32)
    c = torch.where(s[..., None] > 0, v.double() / s[..., None].double().clamp_min(1e-300), torch.zeros_like(v).double())
    return c.round().to(torch.int32), s


def _values(c, s, dtype):
    return (c.float() * s[..., None]).reshape(*c.shape[:-2], -1).to(dtype)


def _pack(x, key):
    """Pages [P][H][bytes] uint8 of rows x [P][H][ps][D]."""
    c, s = _quantise(x)
    P, H, ps, n, _ = c.shape
    u = (c & 15).reshape(P, H, ps, n, 4, 4, 2)                       # G, y, i, h
    u = u.permute(0, 1, 2, 4, 3, 6, 5) if key else u.permute(0, 1, 2, 4, 6, 3, 5)
    u = u.reshape(P, H, ps, n * GROUP // 2, 2)
    codes = (u[..., 0] | (u[..., 1] << 4)).to(torch.uint8).reshape(P, H, -1)
    scales = s.to(torch.bfloat16).contiguous().view(torch.uint8).reshape(P, H, -1)
    return torch.cat([codes, scales], -1).contiguous()


def _unpack(pages, ps, d, key):
    """fp32 rows [..., ps, D] of pages [..., bytes]."""
    n = d // GROUP
    lead = pages.shape[:-1]
    b = pages[..., :ps * d // 2].to(torch.int32)
    nib = torch.stack([b & 15, b >> 4], -1).reshape(*lead, ps, d)
    nib = nib.reshape(*lead, ps, 4, n, 2, 4) if key else nib.reshape(*lead, ps, 4, 2, n, 4)
    L = len(lead) + 1
    order = (L + 1, L, L + 3, L + 2) if key else (L + 2, L, L + 3, L + 1)
    c = ((nib ^ 8) - 8).permute(*range(L), *order).reshape(*lead, ps, n, GROUP).float()
    s = pages[..., ps * d // 2:].contiguous().view(torch.bfloat16).float().reshape(*lead, ps, n, 1)
    return (c * s).reshape(*lead, ps, d)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return globals()["_prepare_" + case["op"]](case, seed, g)


def _prepare_tables(case, seed, g):
    B, ps, most = case["batch"], case["page_size"], _row_buffer(case)
    new = _lengths(case, seed)
    new = new * most // max(most, int(new.sum()))
    r = np.random.default_rng(seed + 1)
    ctx = r.integers(0, case["ctx"] + 1, B) if case["ctx"] else np.zeros(B, dtype=np.int64)
    have, need = -(-ctx // ps), -(-(ctx + new) // ps)
    width = -(-(case["ctx"] + case["hi"]) // ps) + 2
    spare = 7
    total = int(need.sum()) + spare
    ids = r.permutation(total).astype(np.int32)
    table = np.full((B, width), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    free = ids[at:]
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a.astype(np.int32))).to(DEV)  # noqa: E731
    return dict(case=case, page_table=dev(table), ctx_lens=dev(ctx), new_lens=dev(new), num_pages=total,
                pool=dict(free_pages=dev(free), free_count=dev(np.array([free.size]))), max_rows=most)


def _prepare_store(case, seed, g):
    T, H, D, ps = case["rows"], case["hkv"], case["d"], case["page_size"]
    dt = _typed(case)
    k = torch.randn(T, H, D, generator=g, device=DEV).to(dt)
    v = torch.randn(T, H, D, generator=g, device=DEV).to(dt)
    pages = -(-T // ps) + 3
    where = torch.randperm(pages, generator=g, device=DEV)[torch.arange(T, device=DEV) // ps] * ps + torch.arange(T, device=DEV) % ps
    where = torch.where(torch.rand(T, generator=g, device=DEV) < case["skip"], torch.full_like(where, -1), where)
    bytes_ = ps * (D // 2 + D // 16)
    cache = dict(k_pages=torch.zeros(pages, H, bytes_, dtype=torch.uint8, device=DEV),
                 v_pages=torch.zeros(pages, H, bytes_, dtype=torch.uint8, device=DEV))
    return dict(case=case, k=k, v=v, slots=where, cache=cache, k_out=torch.zeros_like(k), v_out=torch.zeros_like(v))


def _prepare_attn(case, seed, g):
    B, Hq, H, D, k, ps = (case[n] for n in ("batch", "hq", "hkv", "d", "k", "page_size"))
    dt = _typed(case)
    P = _lengths(case, seed)
    n, R = max(k, 1), (1 if k == 0 else k + k * k)
    need = -(-(P + n) // ps)
    total = int(need.sum()) + 2
    r = np.random.default_rng(seed + 1)
    ids = r.permutation(total).astype(np.int32)
    table = np.full((B, -(-(case["hi"] + n) // ps) + 1), -1, dtype=np.int32)
    at, slots = 0, np.zeros((B, n), dtype=np.int64)
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
        pos = P[b] + np.arange(n)
        slots[b] = table[b, pos // ps].astype(np.int64) * ps + pos % ps
    sides = []
    for key in (True, False):
        step = max(1, (1 << 26) // (H * ps * D))
        sides.append(torch.cat([_pack(torch.randn(min(step, total - i), H, ps, D, generator=g, device=DEV).to(dt), key)
                                for i in range(0, total, step)]))
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dt)  # noqa: E731
    cache = dict(k_pages=sides[0], v_pages=sides[1], page_table=torch.from_numpy(table).to(DEV),
                 seq_lens=torch.from_numpy(P.astype(np.int32)).to(DEV))
    return dict(case=case, cache=cache, q=rnd(B, R, Hq, D), k_blk=rnd(B, R, H, D), v_blk=rnd(B, R, H, D),
                slots=torch.from_numpy(slots.reshape(-1)).to(DEV))


def _prepare_linear(case, seed, g):
    T, N, K = case["rows"], case["n"], case["kdim"]
    bf = lambda t: t.to(torch.bfloat16)  # noqa: E731
    st = dict(case=case, x=bf(torch.randn(T, K, generator=g, device=DEV)),
              w=bf(torch.randn(N, K, generator=g, device=DEV) / math.sqrt(K)), bias=None, residual=None)
    if case["bias"]:
        st["bias"] = bf(torch.randn(N, generator=g, device=DEV))
    if case["residual"]:
        st["residual"] = bf(torch.randn(T, N, generator=g, device=DEV))
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


def _own_tables(st):
    import ar_decoding_b200 as tidar
    return tidar.build_tables(st["page_table"], st["ctx_lens"], st["new_lens"], st["pool"],
                              page_size=st["case"]["page_size"], num_pages=st["num_pages"], max_rows=st["max_rows"])


def _plain_tables(st):
    ps, rows = st["case"]["page_size"], st["max_rows"]
    ctx, new, table = st["ctx_lens"].long(), st["new_lens"].long(), st["page_table"]
    free, count = st["pool"]["free_pages"], st["pool"]["free_count"].long()
    B, width = table.shape
    starts = torch.zeros(B + 1, dtype=torch.int64, device=DEV)
    starts[1:] = new.cumsum(0)
    entry = torch.arange(width, device=DEV)
    first, last = -(-ctx // ps), -(-(ctx + new) // ps)
    wants = (entry >= first[:, None]) & (entry < last[:, None]) & (table == -1)
    order = wants.reshape(-1).long().cumsum(0).reshape(B, width)      # 1, 2, ... of the entries that need a page
    taken = free[(count - order).clamp(0, free.numel() - 1)]
    out = torch.where(wants, taken, table)
    row = torch.arange(rows, device=DEV)
    b = torch.searchsorted(starts[1:], row, right=True).clamp(max=B - 1)
    live = row < starts[-1]
    pos = ctx[b] + row - starts[b]
    slot = out[b, (pos // ps).clamp(0, width - 1)].long() * ps + pos % ps
    return dict(page_table=out, free_count=(count - wants.sum()).int(), row_starts=starts.int(),
                slots=torch.where(live, slot, torch.full_like(slot, -1)),
                positions=torch.where(live, pos, torch.full_like(pos, -1)).int())


def _own_store(st):
    import ar_decoding_b200 as tidar
    tidar.kv4_append(st["cache"], st["k"], st["v"], st["slots"])
    return tidar.kv4_gather(st["cache"], st["slots"], out=(st["k_out"], st["v_out"]))


def _plain_store(st):
    live = (st["slots"] >= 0)[:, None, None]
    out = []
    for x in (st["k"], st["v"]):
        v = _values(*_quantise(x), x.dtype)
        out.append(torch.where(live, v, torch.zeros_like(v)))
    return out


def _own_attn(st):
    import ar_decoding_b200 as tidar
    c = st["case"]
    out, lse = tidar.step_attn_kv4(st["q"], st["k_blk"], st["v_blk"], st["cache"], c["k"], max_prefix_len=c["hi"],
                                   append=c["append"])
    if not c["append"]:
        return dict(out=out, lse=lse)
    ks, vs = tidar.kv4_gather(st["cache"], st["slots"], head_dim=c["d"], dtype=st["q"].dtype)
    return dict(out=out, lse=lse, k_rows=ks, v_rows=vs)


def _zone_mask(k, R):
    """[R][R] truth values: which step keys a row sees."""
    row, key = torch.arange(R, device=DEV)[:, None], torch.arange(R, device=DEV)[None, :]
    if k == 0:
        return key <= row
    block = (row - k) // k                       # 0-based block of a mask row
    mine = (key >= k + block * k) & (key < k + block * k + k)
    return torch.where(row < k, key <= row, (key <= block) | mine)


def _plain_attn(st):
    c = st["case"]
    B, Hq, H, D, k, ps = (c[n] for n in ("batch", "hq", "hkv", "d", "k", "page_size"))
    R, G, cache = st["q"].shape[1], Hq // H, st["cache"]
    width = -(-c["hi"] // ps)
    ids = cache["page_table"][:, :width].clamp(min=0).long()
    rows = lambda pages, key: (_unpack(pages[ids], ps, D, key).permute(0, 2, 1, 3, 4)  # noqa: E731
                               .reshape(B, H, width * ps, D))
    heads = lambda x: x.float().reshape(B, R, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * R, D)  # noqa: E731
    step = lambda x: x.float().permute(0, 2, 1, 3)  # noqa: E731
    q = heads(st["q"]) / math.sqrt(D)
    old = torch.matmul(q, rows(cache["k_pages"], True).transpose(-1, -2))
    old.masked_fill_((torch.arange(width * ps, device=DEV) >= cache["seq_lens"][:, None])[:, None, None, :], -math.inf)
    new = torch.matmul(q, step(st["k_blk"]).transpose(-1, -2))
    new.masked_fill_(~_zone_mask(k, R).repeat(G, 1), -math.inf)
    top = torch.maximum(old.amax(-1), new.amax(-1)) if width else new.amax(-1)
    old, new = old.sub_(top[..., None]).exp_(), new.sub_(top[..., None]).exp_()
    total = old.sum(-1) + new.sum(-1)
    o = torch.matmul(old, rows(cache["v_pages"], False)) + torch.matmul(new, step(st["v_blk"]))
    o = (o / total[..., None]).reshape(B, H, G, R, D).permute(0, 3, 1, 2, 4).reshape(B, R, Hq, D)
    lse = (top + total.log()).reshape(B, H, G, R).permute(0, 3, 1, 2).reshape(B, R, Hq)
    res = dict(out=o.to(st["q"].dtype), lse=lse)
    if c["append"]:
        n = max(k, 1)
        for name, x in (("k_rows", st["k_blk"]), ("v_rows", st["v_blk"])):
            res[name] = _values(*_quantise(x[:, :n]), x.dtype).reshape(B * n, H, D)
    return res


def _own_linear(st):
    import ar_decoding_b200 as tidar
    return tidar.linear_fused(st["x"], st["w"], bias=st["bias"], activation=st["case"]["act"], residual=st["residual"])


def _act(y, name):
    if name == "relu":
        return y.clamp(min=0)
    if name == "gelu":
        return 0.5 * y * (1 + torch.erf(y / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    return y * torch.sigmoid(y) if name == "silu" else y


def _plain_linear(st):
    y = torch.matmul(st["x"].float(), st["w"].float().t())
    if st["bias"] is not None:
        y = y + st["bias"].float()
    y = _act(y, st["case"]["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "tables":
        mean = (case["lo"] + case["hi"]) / 2
        rows = _row_buffer(case)             # every slot and position is written
        pages = case["batch"] * ((case["ctx"] / 2 + mean) / case["page_size"] + 1)
        return dict(bytes=12 * rows + 8 * pages + 12 * case["batch"], flops=0)
    if op == "store":
        e = 4 if case["dtype"] == "f32" else 2
        live = case["rows"] * (1 - case["skip"])
        row = 2 * case["hkv"] * case["d"]
        return dict(bytes=live * (2 * row * e + 2 * row * 0.5625) + 8 * case["rows"], flops=0)
    if op == "attn":
        e = 4 if case["dtype"] == "f32" else 2
        k = case["k"]
        R = 1 if k == 0 else k + k * k
        keys = case["batch"] * (case["lo"] + case["hi"]) / 2
        cache = keys * case["hkv"] * 2 * case["d"] * 0.5625
        io = case["batch"] * R * (2 * case["hq"] + 2 * case["hkv"]) * case["d"] * e + case["batch"] * R * case["hq"] * 4
        return dict(bytes=cache + io, flops=4.0 * R * case["hq"] * case["d"] * keys)
    T, N, K = case["rows"], case["n"], case["kdim"]
    return dict(bytes=2.0 * (T * K + N * K + T * N * (2 if case["residual"] else 1) + (N if case["bias"] else 0)),
                flops=2.0 * T * N * K)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return globals()["_exact_" + case["op"]](case, st)


def _exact_tables(case, st):
    ps = case["page_size"]
    table, ctx, new = (st[n].cpu().numpy().astype(np.int64) for n in ("page_table", "ctx_lens", "new_lens"))
    stack = st["pool"]["free_pages"].cpu().numpy().tolist()
    slots, pos = np.full(st["max_rows"], -1, dtype=np.int64), np.full(st["max_rows"], -1, dtype=np.int32)
    starts = [0]
    for b in range(case["batch"]):
        lo, hi = int(ctx[b]), int(ctx[b] + new[b])
        for e in range(-(-lo // ps), -(-hi // ps)):
            if table[b, e] < 0:
                table[b, e] = stack.pop()
        p = np.arange(lo, hi)
        slots[starts[-1]:starts[-1] + len(p)] = table[b, p // ps] * ps + p % ps
        pos[starts[-1]:starts[-1] + len(p)] = p
        starts.append(starts[-1] + len(p))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32)  # noqa: E731
    return dict(page_table=i32(table), free_count=i32([len(stack)]), row_starts=i32(starts),
                slots=torch.from_numpy(slots), positions=torch.from_numpy(pos))


def _nearest(x):
    """The 4-bit group values nearest to x [..., D], in 64 bits, from the definition."""
    v = x.double().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    want = v.abs().max(-1, keepdim=True).values / 7
    e = torch.floor(torch.log2(want.clamp_min(1e-300)))
    unit = torch.exp2(e - 4)
    s = torch.round(want / unit) * unit
    return (torch.round(v / s.clamp_min(1e-300)) * s).reshape(x.shape)


def _exact_store(case, st):
    skip = (st["slots"] < 0)[:, None, None]
    return [_nearest(x).masked_fill(skip, 0.0) for x in (st["k"], st["v"])]


def _row_values(pages, ids, count, case, key):
    """Rows 0..count-1 of one sequence, [count][Hkv][D] in 64 bits, read nibble by nibble from the page's definition."""
    ps, D, H = case["page_size"], case["d"], case["hkv"]
    n = D // 32
    d = torch.arange(D, device=DEV)
    G, y, i, h = d // 32, (d % 32) // 8, (d % 8) // 2, d % 2
    unit = y * 2 * n + (2 * G + h if key else h * n + G)
    at, shift = unit * 2 + i // 2, 4 * (i % 2)
    p = pages[ids.long()]                                             # [pages][H][bytes]
    out = []
    for r in range(ps):
        byte = p[:, :, r * (D // 2) + at].to(torch.int64)
        c = (byte >> shift) & 15
        c = torch.where(c > 7, c - 16, c).double()
        sc = p[:, :, ps * D // 2 + r * 2 * n:ps * D // 2 + (r + 1) * 2 * n].contiguous().view(torch.bfloat16).double()
        out.append(c * sc[:, :, G])
    return torch.stack(out, 1).reshape(-1, H, D)[:count]


def _exact_attn(case, st):
    B, Hq, H, D, k = (case[n] for n in ("batch", "hq", "hkv", "d", "k"))
    R = st["q"].shape[1]
    cache = st["cache"]
    out = torch.zeros(B, R, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(B, R, Hq, dtype=torch.float64, device=DEV)
    sees = torch.zeros(R, R, dtype=torch.bool, device=DEV)
    for r in range(R):
        if k == 0 or r < k:
            sees[r, :r + 1] = True
        else:
            j = (r - k) // k + 1
            sees[r, :j] = True
            sees[r, k + (j - 1) * k:k + j * k] = True
    for b in range(B):
        P = int(cache["seq_lens"][b])
        ids = cache["page_table"][b, :-(-P // case["page_size"])]
        kk = torch.cat([_row_values(cache["k_pages"], ids, P, case, True), st["k_blk"][b].double()])
        vv = torch.cat([_row_values(cache["v_pages"], ids, P, case, False), st["v_blk"][b].double()])
        mask = torch.cat([torch.ones(R, P, dtype=torch.bool, device=DEV), sees], 1)
        for h in range(Hq):
            s = st["q"][b, :, h].double() @ kk[:, h // (Hq // H)].t() / math.sqrt(D)
            s = s.masked_fill(~mask, -math.inf)
            lse[b, :, h] = torch.logsumexp(s, 1)
            out[b, :, h] = torch.softmax(s, 1) @ vv[:, h // (Hq // H)]
    res = dict(out=out, lse=lse)
    if case["append"]:
        n = max(k, 1)
        res["k_rows"], res["v_rows"] = (_nearest(st[x][:, :n]).reshape(B * n, H, D) for x in ("k_blk", "v_blk"))
    return res


def _exact_linear(case, st):
    y = st["x"].double() @ st["w"].double().t()
    if case["bias"]:
        y += st["bias"].double()
    if case["act"] == "relu":
        y = torch.relu(y)
    elif case["act"] == "gelu":
        y = y * torch.special.ndtr(y)
    elif case["act"] == "gelu_tanh":
        y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
    elif case["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    return y + st["residual"].double() if case["residual"] else y
