"""tidar_linear_fused against act(x w^T + bias) + residual in 64 bits.

Tolerance: the fp32 sum of K exact products is off by at most (K/16 + 16) 2^-23
of sum |x||w| + |bias| (blocks of 16 products, then splits); every activation
here has a slope of at most 1.13, its own fp32 evaluation adds 16 roundings of
its argument's size; the result is rounded to bf16 once (2^-8 of itself)."""
import math

import pytest
import torch

import ar_decoding_b200 as tidar

pytestmark = pytest.mark.gpu


def reference(x, w, bias, act, res):
    x, w = x.double(), w.double()
    y = x @ w.t()
    mag = x.abs() @ w.abs().t()
    if bias is not None:
        y, mag = y + bias.double(), mag + bias.double().abs()
    s = y
    if act == "relu":
        s = y.clamp(min=0)
    elif act == "gelu":
        s = y * torch.special.ndtr(y)
    elif act == "gelu_tanh":
        s = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
    elif act == "silu":
        s = y * torch.sigmoid(y)
    want = s if res is None else s + res.double()
    tol = 1.13 * (x.shape[-1] / 16 + 16) * 2.0 ** -23 * mag + 16 * 2.0 ** -23 * (y.abs() + want.abs()) + 2.0 ** -8 * want.abs()
    return want, tol + 2.0 ** -133


def data(seed, T, N, K, bias=True, res=True, x_scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    bf = lambda t: t.to(torch.bfloat16)  # noqa: E731
    return (bf(r(T, K) * x_scale), bf(r(N, K) / math.sqrt(K)), bf(r(N)) if bias else None, bf(r(T, N)) if res else None)


def check(got, want, tol):
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all() and (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("act", sorted(tidar.ACTIVATIONS))
@pytest.mark.parametrize("bias,res", [(False, False), (True, False), (False, True), (True, True)])
def test_epilogues(act, bias, res):
    x, w, b, r = data(1, 50, 200, 256, bias, res, x_scale=3.0)
    y = tidar.linear_fused(x, w, bias=b, activation=act, residual=r)
    check(y, *reference(x, w, b, act, r))
    assert tidar.device_status() == (tidar.OK, 0)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 77, 255, 256, 257, 272, 288, 289, 513, 1111])
@pytest.mark.parametrize("N,K", [(1, 8), (7, 64), (127, 72), (128, 4096), (130, 1544), (1000, 520), (2049, 200)])
def test_odd_sizes(T, N, K):
    x, w, b, r = data(T * 7 + N, T, N, K)
    check(tidar.linear_fused(x, w, bias=b, activation="silu", residual=r), *reference(x, w, b, "silu", r))


@pytest.mark.parametrize("T,N,K", [(272, 4096, 4096), (2048, 2048, 1024), (300, 6000, 8192), (4096, 384, 640)])
def test_large(T, N, K):
    x, w, b, r = data(3, T, N, K)
    check(tidar.linear_fused(x, w, bias=b, activation="gelu_tanh", residual=r), *reference(x, w, b, "gelu_tanh", r))


def test_neighbouring_memory_is_left_alone():
    for T, N, K in ((5, 7, 64), (130, 129, 200), (300, 136, 64)):
        x, w, b, r = data(5, T, N, K)
        flat = torch.full((T * N + 64,), 77.0, dtype=torch.bfloat16, device="cuda")
        tidar.linear_fused(x, w, bias=b, residual=r, out=flat[:T * N].view(T, N))
        assert (flat[T * N:] == 77).all()
        check(flat[:T * N].view(T, N), *reference(x, w, b, "none", r))


def test_plain_epilogue_is_the_linear_layer():
    # The two kernels cut the reduction at different places, and fp32 sums of the same
    # products in another order differ in their last bits (a + b + c with a = -b =
    # 2^24, c = 1 is 1 or 0), so their bf16 results need not be equal: both are within
    # the tolerance of the same sum, and of each other within twice that.
    x, w, _, _ = data(9, 64, 256, 512)
    want, tol = reference(x, w, None, "none", None)
    a, b = tidar.linear_fused(x, w), tidar.linear(x, w)
    check(a, want, tol)
    check(b, want, tol)
    check(a, b.double(), 2 * tol)


def test_residual_in_place_and_leading_dims():
    x, w, b, r = data(11, 60, 256, 512)
    want, tol = reference(x, w, b, "gelu", r)
    h = r.clone().view(3, 20, 256)
    y = tidar.linear_fused(x.view(3, 20, 512), w, bias=b, activation="gelu", residual=h, out=h)
    assert y is h
    check(h.view(60, 256), want, tol)
    assert tidar.linear_fused(x[:0], w).shape == (0, 256)


def test_extreme_values():
    x, w, b, _ = data(13, 4, 64, 64)
    big = torch.tensor([3e38, -3e38, float("inf"), float("nan")], dtype=torch.bfloat16, device="cuda")
    b[:4] = big
    for act in tidar.ACTIVATIONS:
        y = tidar.linear_fused(x * 0, w, bias=b, activation=act).float()
        assert torch.isnan(y[:, 3]).all()
        assert torch.isposinf(y[:, 2]).all() and (y[:, 0] > 2.9e38).all()
        assert (y[:, 1] == (float(b[1]) if act == "none" else 0)).all()


def test_refusals():
    x, w, b, r = data(15, 6, 64, 64)
    for kw in (dict(bias=b[:8]), dict(residual=r[:2]), dict(activation="tanh"), dict(out=r.float()), dict(bias=b.float()),
               dict(residual=r.t())):
        with pytest.raises(ValueError):
            tidar.linear_fused(x, w, **kw)
    with pytest.raises(ValueError):
        tidar.linear_fused(x, w[:, :32].contiguous())
    with pytest.raises(tidar.TidarError):
        tidar.linear_fused(x[:, :60].contiguous(), w[:, :60].contiguous())


def test_two_streams_and_capture():
    x, w, b, r = data(17, 272, 2048, 4096)
    want = tidar.linear_fused(x, w, bias=b, activation="silu", residual=r)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        got.append(tidar.linear_fused(x, w, bias=b, activation="silu", residual=r, stream=s))
    out, g = torch.zeros_like(want), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tidar.linear_fused(x, w, bias=b, activation="silu", residual=r, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got) and torch.equal(out, want)


@pytest.mark.parametrize("N", [65536, 65537])
def test_outputs_past_32_bits(N):
    T, K = 33000, 8
    assert T * N > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(N)
    # whole numbers: products and sums are exact, so the order of the sums is no matter
    x = torch.randint(-3, 4, (T, K), generator=g, device="cuda").bfloat16()
    w = torch.randint(-3, 4, (N, K), generator=g, device="cuda").bfloat16()
    y = tidar.linear_fused(x, w, activation="relu")
    for r in (0, 255, 32767, 32768, 32999):
        assert torch.equal(y[r].float(), torch.relu(w.float() @ x[r].float())), r
    assert torch.equal(y[:, N - 1].float(), torch.relu(x.float() @ w[N - 1].float()))


@pytest.mark.parametrize("T", [4097, 4103, 4127])
@pytest.mark.parametrize("N,K", [(2048, 512), (2056, 200)])
def test_ragged_rows_on_the_paired_tiles(T, N, K):
    # Rows that end inside a warp's 32 while N % 8 == 0: some lanes of the last row tile
    # store nothing between two loads of the whole warp.  The paired tiles take these
    # sizes: 136 or 153 tiles are three waves of 74 pairs at most, 16000 + 3 * 8 * 760 =
    # 34000 clocks; the split kernel's 88 tiles or more are two waves of 24000 at least
    # (6000 + 55 a row of 320), before a slice is counted.
    x, w, b, r = data(T + N, T, N, K)
    flat = torch.full((T * N + 64,), 77.0, dtype=torch.bfloat16, device="cuda")
    y = tidar.linear_fused(x, w, bias=b, activation="silu", residual=r, out=flat[:T * N].view(T, N))
    check(y, *reference(x, w, b, "silu", r))
    assert (flat[T * N:] == 77).all() and tidar.device_status() == (tidar.OK, 0)


def act_of_every_bf16(act, T):
    """activation(b) of every finite bf16 number b, by x = 0 and the bias, and of the
    definition in 64 bits, written without cancellation."""
    b = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    b = b[torch.isfinite(b)].contiguous()
    x, w = (torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda") for n in (T, b.numel()))
    # one row: a few thousand features a call, which the split kernel takes; 2048 rows of
    # all of them are the paired tiles'
    y = torch.cat([tidar.linear_fused(x, w[:c.numel()], bias=c.clone(), activation=act)
                   for c in b.split(4080 if T == 1 else b.numel())], 1)
    assert (y == y[:1]).all()
    v = b.double()
    if act == "gelu":
        want = 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    else:
        u = v if act == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        e = torch.exp(-u.abs())
        want = torch.where(u < 0, v * e, v) / (1 + e)
    return v, y[0].double(), want


# Relative error: half a step of bf16, 2^-8, and the fp32 evaluation.  A factor exp(-z)
# carries z's rounding times z, and an activation's value is above 2^-133 only for z < 93;
# three roundings of z and 110 units of the exponential's own are (3 * 93 + 110) 2^-24 <
# 2^-15.  Below bf16's normal numbers half a step is 2^-134.
TAIL_REL, TAIL_ABS = 2.0 ** -8 + 2.0 ** -15, 2.0 ** -133


@pytest.mark.parametrize("T", [1, 2048])
def test_erf_gelu_of_every_bf16_number(T):
    v, y, want = act_of_every_bf16("gelu", T)
    bad = (y - want).abs() > TAIL_REL * want.abs() + TAIL_ABS
    assert not bad.any(), v[bad]


@pytest.mark.parametrize("T", [1, 2048])
@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_sigmoid_forms_of_every_bf16_number(act, T):
    v, y, want = act_of_every_bf16(act, T)
    bad = (y - want).abs() > TAIL_REL * want.abs() + TAIL_ABS
    assert not bad.any(), v[bad]
