"""NaN values in the 4-bit cache, in the step rows and in q: the rows that attend
them come out NaN, no other row does, whatever the kernel family and however the
keys are split.  (An infinity is stored as a NaN.)"""
import math

import pytest
import torch

import ar_decoding_b200 as tidar
from test_gpu_kv4_attn import compare, make, paths

pytestmark = pytest.mark.gpu

TYPES = [("f32", 64), ("f32", 128), ("bf16", 64), ("bf16", 128)]


def poison(st, which, b, keys, head, group=0):
    """The scale of one group of these keys' rows becomes a NaN."""
    ps, D = st["ps"], st["D"]
    pages = st["cache"][which]
    for key in keys:
        at = ps * (D // 2) + (key % ps) * (D // 16) + 2 * group
        pages[int(st["table"][b, key // ps]), head, at:at + 2] = torch.tensor([0xc0, 0x7f], dtype=torch.uint8, device="cuda")


def call(st, path, **kw):
    out, lse = tidar.step_attn_kv4(st["q"], st["k_blk"], st["v_blk"], st["cache"], st["k"],
                                   max_prefix_len=max(max(st["P"]), 1), path=path, append=False, **kw)
    assert tidar.device_status() == (tidar.OK, 0)
    return out, lse


# The NaN keys of sequence 1: a lone key; every key; the first keys of a sequence (the
# first batch, and part of it, of whatever walks the keys); the first keys of the last
# 32, the shortest split; and that split's only key.
KEYS = [(1, range(1)), (20, range(20)), (40, range(8)), (40, range(3)), (72, range(64, 72)), (33, [32])]


@pytest.mark.parametrize("step_keys", [False, True])
@pytest.mark.parametrize("P,keys", KEYS, ids=lambda v: str(list(v)) if not isinstance(v, int) else str(v))
@pytest.mark.parametrize("k", [0, 2])
@pytest.mark.parametrize("dtype,D", TYPES)
def test_nan_keys_met_before_any_finite_one(dtype, D, k, P, keys, step_keys):
    st = make(51, [P, P, 50], 4, 2, D, k, 16, dtype)
    poison(st, "k_pages", 1, keys, 0)
    for path in paths(k, 2, D, dtype):
        out, lse = call(st, path, step_keys=step_keys)
        assert torch.isnan(out[1, :, :2]).all() and torch.isnan(lse[1, :, :2]).all(), path
        assert torch.isfinite(out[1, :, 2:]).all() and torch.isfinite(lse[1, :, 2:]).all(), path
        compare(st, out, lse, step_keys=step_keys, seqs=[0, 2])


@pytest.mark.parametrize("k", [0, 2])
@pytest.mark.parametrize("dtype,D", TYPES)
def test_nan_in_one_query_row(dtype, D, k):
    st = make(52, [70, 0], 4, 2, D, k, 16, dtype)
    st["q"][:, -1, 1] = math.nan
    for path in paths(k, 2, D, dtype):
        out, lse = call(st, path)
        hit = torch.zeros_like(lse, dtype=torch.bool)
        hit[:, -1, 1] = True
        assert (torch.isnan(lse) == hit).all() and (torch.isnan(out) == hit[..., None]).all(), path


@pytest.mark.parametrize("k", [0, 2])
@pytest.mark.parametrize("dtype,D", TYPES)
def test_nan_in_a_step_key(dtype, D, k):
    # draft 1 is seen by every row; with an empty prefix it is all that the first row sees
    st = make(53, [0, 70], 4, 2, D, k, 16, dtype)
    st["k_blk"][:, 0, 0] = math.nan
    for path in paths(k, 2, D, dtype):
        out, lse = call(st, path)
        assert torch.isnan(out[:, :, :2]).all() and torch.isnan(lse[:, :, :2]).all(), path
        assert torch.isfinite(out[:, :, 2:]).all() and torch.isfinite(lse[:, :, 2:]).all(), path


@pytest.mark.parametrize("k", [2, 4])
@pytest.mark.parametrize("dtype,D", TYPES)
def test_nan_in_a_key_that_a_row_does_not_see(dtype, D, k):
    # the last slot of the last mask block is seen by that block's rows only
    st = make(54, [70], 4, 2, D, k, 16, dtype)
    st["k_blk"][:, -1] = math.nan
    for path in paths(k, 2, D, dtype):
        out, lse = call(st, path)
        assert torch.isnan(out[:, -k:]).all() and torch.isnan(lse[:, -k:]).all(), path
        assert torch.isfinite(out[:, :-k]).all() and torch.isfinite(lse[:, :-k]).all(), path


@pytest.mark.parametrize("force", [0, 1])
@pytest.mark.parametrize("P", [64, 600, 4096])
@pytest.mark.parametrize("k", [0, 4])
@pytest.mark.parametrize("dtype,D", TYPES)
def test_nan_value_of_a_key_whose_weight_is_nothing(dtype, D, k, P, force):
    # Scores are 200 in the second half of the prefix and -200 in the first, so the first
    # half's weight is exp(-400) = 0 in fp32, as are the weights of the splits that hold
    # it; the definition's 0 * NaN is NaN all the same, in that group of that head.
    ps, H, B = 16, 2, 2
    table = torch.arange(B * (P // ps + 2), dtype=torch.int32, device="cuda").view(B, -1)
    cache = tidar.kv4_cache(table.numel(), H, ps, D, table, torch.full((B,), P, dtype=torch.int32, device="cuda"))
    sign = torch.where(torch.arange(P, device="cuda") < P // 2, -1.0, 1.0)[None, :, None, None]
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    rows = (sign * torch.ones(B, P, H, D, device="cuda")).to(dt)
    vals = torch.randn(B, P, H, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).to(dt)
    pos = torch.arange(P, device="cuda")
    slots = (table.long()[:, pos // ps] * ps + pos % ps).reshape(-1)
    tidar.kv4_append(cache, rows.reshape(-1, H, D), vals.reshape(-1, H, D), slots)
    st = dict(cache=cache, table=table, ps=ps, D=D, k=k, P=[P] * B)
    poison(st, "v_pages", 1, [P // 4], 1, group=1)
    R = 1 if k == 0 else k + k * k
    st["q"] = torch.full((B, R, 2 * H, D), 200 / math.sqrt(D), device="cuda").to(dt)
    st["k_blk"] = st["v_blk"] = torch.zeros(B, R, H, D, dtype=dt, device="cuda")
    tidar.debug_set(tidar.DEBUG_FORCE_SPLIT_PARTIALS, force)
    try:
        for path in paths(k, 2, D, dtype):
            out, lse = call(st, path)
            hit = torch.zeros_like(out, dtype=torch.bool)
            hit[1, :, 2:, 32:64] = True
            assert (torch.isnan(out) == hit).all() and torch.isfinite(lse).all(), path
    finally:
        tidar.debug_set(tidar.DEBUG_FORCE_SPLIT_PARTIALS, 0)
