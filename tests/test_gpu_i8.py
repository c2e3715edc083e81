"""GPU tests of the 8-bit linear layer against its 64-bit definition (oracle/low_precision.py).

Tolerances.  The integer sum is exact, so y = act(acc * xs * ws + b) carries the roundings of a few fp32 operations:
acc to fp32, xs * ws, the FMA, and the activation: x / (1 + exp(-x)) (each within a few ulp, and exp(-x) passes an
error of its argument on multiplied by |x|, at most 100 before the result is negligible) for fp32 results, or
h + h tanh(h) with |tanh.approx - tanh| <= 2^-10.9 for bf16 ones.
  fp32, no activation: 4 roundings, |err| <= 4 * 2^-24 * (|acc xs ws| + |b|)
  fp32, SiLU:          the argument's error times SiLU' <= 1.1, plus 8 ulp of the result, plus 2^-24 |x|
  bf16:                one rounding 2^-8 |y| (twice half a step), and with SiLU |h| 2^-10 for the tanh
"""
import numpy as np
import pytest
import torch

import generative_recommender_attention_jagged_b200 as hstu
from oracle import low_precision as lp

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(T, K, N, x_dtype, seed=0, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, K, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).to(DT[x_dtype])
    w = torch.randn(K, N, generator=g) / K ** 0.5
    b = 0.3 * torch.randn(N, generator=g) if bias else None
    return x, w, b


def check(y, x, codes, ws, b, silu, out):
    lin = lp.linear_i8(x.double().numpy(), codes, ws, None)
    bias = 0.0 if b is None else b.double().numpy()
    pre = lin + bias
    want = pre / (1 + np.exp(-pre)) if silu else pre
    arg = 4 * 2.0 ** -24 * (np.abs(lin) + np.abs(bias))
    if out == "f32":
        tol = 1.1 * arg + 8 * 2.0 ** -24 * np.abs(want) + 2.0 ** -24 * np.abs(pre) if silu else arg
    else:
        tol = arg + 2.0 ** -8 * np.abs(want) + (2.0 ** -10 * np.abs(pre) / 2 if silu else 0)
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= tol + 1e-30).all(), float((err - tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,N", [(16, 8), (512, 2048), (208, 40), (1040, 72)])
def test_weight_quantisation_is_exact(K, N, dtype):
    _, w, _ = inputs(1, K, N, "f32", seed=K)
    w = w.to(DT[dtype])
    w[:, 1] = 0
    w[3, 2] = float("nan")
    w[0, 3] = float("inf")
    w[0, 4] = 2 * w[1:, 4].abs().max()     # halves of a step
    w[1, 4] = w[0, 4] / 2
    wq, ws = hstu.hstu_quant_i8_weight(w.cuda())
    codes, scale = lp.quant_weight_i8(w.double().numpy())
    assert np.array_equal(wq.cpu().numpy(), codes)
    assert np.array_equal(ws.double().cpu().numpy(), scale, equal_nan=True)


@pytest.mark.parametrize("T,K,N,x,out,silu,bias", [
    (1, 16, 8, "bf16", "bf16", False, False),
    (1, 512, 2048, "bf16", "bf16", True, True),
    (3, 48, 24, "f32", "f32", True, True),
    (8, 512, 2048, "bf16", "f32", False, True),
    (16, 1024, 264, "f32", "bf16", False, True),
    (37, 512, 512, "bf16", "bf16", False, True),
    (64, 4096, 136, "bf16", "f32", False, False),
    (65, 272, 520, "f32", "bf16", True, False),
    (127, 128, 128, "bf16", "bf16", True, True),
    (128, 256, 256, "bf16", "f32", True, True),
    (129, 144, 1032, "f32", "f32", False, True),
    (300, 1040, 88, "bf16", "bf16", True, True),
    (1000, 512, 512, "bf16", "bf16", False, True),
    (1025, 528, 776, "bf16", "bf16", True, True),
    (5000, 512, 2048, "bf16", "bf16", True, True),
    (4097, 2064, 1000, "f32", "f32", False, False),
    (20000, 64, 256, "bf16", "f32", True, True),
    (20000, 64, 264, "bf16", "bf16", False, False),
])
def test_linear_i8_matches_definition(T, K, N, x, out, silu, bias):
    xt, w, b = inputs(T, K, N, x, seed=T + K + N, bias=bias)
    wq, ws = hstu.hstu_quant_i8_weight(w.cuda())
    y = hstu.hstu_linear_i8(xt.cuda(), wq, ws, None if b is None else b.cuda(), silu=silu, out_dtype=DT[out])
    assert y.dtype == DT[out] and y.shape == (T, N)
    check(y, xt, wq.cpu().numpy(), ws.cpu().numpy(), b, silu, out)


def test_ties_and_special_rows():
    """Half steps go to the even code, zero and tiny rows give the bias, rows with an infinity or NaN give NaN and
    leave the others alone."""
    K, N = 64, 16
    x = torch.randn(6, K, generator=torch.Generator().manual_seed(3)).bfloat16()
    x[0, :] = 0
    x[1, 0], x[1, 1:20] = 4.0, 2.0           # 63.5 steps
    x[2, 5] = float("nan")
    x[3, 7] = float("-inf")
    x[4, :] = 1e-38
    w = torch.eye(K)[:, :N].contiguous()      # y = the first codes
    b = torch.arange(N).float()
    wq, ws = hstu.hstu_quant_i8_weight(w.cuda())
    y = hstu.hstu_linear_i8(x.cuda(), wq, ws, b.cuda(), out_dtype=torch.float32).cpu()
    assert torch.equal(y[0], b) and torch.equal(y[4], b)
    assert torch.isnan(y[2:4]).all()
    ok = [1, 5]
    check(y[ok], x[ok], wq.cpu().numpy(), ws.cpu().numpy(), b, False, "f32")


def test_row_scales_are_exact():
    """An element of code 1 under an identity matrix comes out as its row's scale, for amax over the whole fp32 range."""
    rng = np.random.default_rng(77)
    amax = rng.integers(1, 0x7F800000, size=20000, dtype=np.int64).astype(np.int32).view(np.float32)
    edge = np.float32(127) * np.float32(2.0 ** -126)
    amax[:64] = (np.full(64, edge).view(np.int32) + np.arange(-32, 32, dtype=np.int32)).view(np.float32)
    amax[64:67] = np.finfo(np.float32).max, np.float32(2.0 ** -149), 127.0
    want = amax / np.float32(127)             # IEEE division: rounded once
    want[want < 2.0 ** -126] = 0
    x = np.zeros((len(amax), 16), np.float32)
    x[:, 0], x[:, 1] = amax, want
    out = hstu.hstu_linear_i8(torch.from_numpy(x).cuda(), torch.eye(16, dtype=torch.int8, device="cuda"),
                              torch.ones(16, device="cuda"))
    assert np.array_equal(out[:, 1].cpu().numpy(), want)


def test_strided_rows_and_neighbours_left_alone():
    T, K, N = 70, 256, 136
    xt, w, b = inputs(T, K, N, "bf16", seed=11)
    wide = torch.full((T, K + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 32:32 + K] = xt.cuda()
    out = torch.full((T + 2, N + 24), -5.0, dtype=torch.bfloat16, device="cuda")
    wq, ws = hstu.hstu_quant_i8_weight(w.cuda())
    y = hstu.hstu_linear_i8(wide[:, 32:32 + K], wq, ws, b.cuda(), out=out[1:T + 1, 8:8 + N])
    check(y, xt, wq.cpu().numpy(), ws.cpu().numpy(), b, False, "bf16")
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1:T + 1, 8:8 + N] = False
    assert (out[keep] == -5.0).all()


def test_empty_rows_and_refusals():
    wq = torch.zeros(16, 32, dtype=torch.int8, device="cuda")
    ws = torch.ones(16, device="cuda")
    y = hstu.hstu_linear_i8(torch.zeros(0, 32, dtype=torch.bfloat16, device="cuda"), wq, ws)
    assert y.shape == (0, 16)
    x = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: hstu.hstu_linear_i8(x[:, ::2], wq, ws), lambda: hstu.hstu_linear_i8(x[:, :16], wq, ws),
                lambda: hstu.hstu_linear_i8(x.half(), wq, ws), lambda: hstu.hstu_linear_i8(x, wq, ws[:8]),
                lambda: hstu.hstu_linear_i8(x, wq.t(), ws), lambda: hstu.hstu_linear_i8(x, wq, ws, ws[:4]),
                lambda: hstu.hstu_linear_i8(x, wq, ws, out=torch.zeros(4, 8, device="cuda")),
                lambda: hstu.hstu_linear_i8(x, wq, ws, out_dtype=torch.float16),
                lambda: hstu.hstu_linear_i8(x, wq, ws, workspace=torch.zeros(64, dtype=torch.uint8)),
                lambda: hstu.hstu_quant_i8_weight(x.t())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(hstu.HstuError, match="WORKSPACE"):
        hstu.hstu_linear_i8(x, wq, ws, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(hstu.HstuError, match="ALIGNMENT"):
        hstu.hstu_linear_i8(torch.zeros(4, 33, dtype=torch.bfloat16, device="cuda")[:, 1:], wq, ws)


@pytest.mark.parametrize("T", [5, 700])
def test_captured_replay_and_second_stream(T):
    """A captured call follows new inputs in the same buffers; a call on another stream gives the same bits."""
    K, N = 512, 520
    xt, w, b = inputs(T, K, N, "bf16", seed=21)
    x2 = inputs(T, K, N, "bf16", seed=22)[0]
    wq, ws = hstu.hstu_quant_i8_weight(w.cuda())
    x, bc = xt.cuda(), b.cuda()
    buf = torch.empty(hstu.hstu_linear_i8_workspace_size(T, K, N), dtype=torch.uint8, device="cuda")
    out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    first = hstu.hstu_linear_i8(x, wq, ws, bc, silu=True, out=out, workspace=buf).clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hstu.hstu_linear_i8(x, wq, ws, bc, silu=True, out=out, workspace=buf)
    x.copy_(x2.cuda())
    graph.replay()
    torch.cuda.synchronize()
    check(out, x2, wq.cpu().numpy(), ws.cpu().numpy(), b, True, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x.copy_(xt.cuda())
    side.wait_stream(torch.cuda.current_stream())
    other = hstu.hstu_linear_i8(x, wq, ws, bc, silu=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, first)
    assert hstu.hstu_check_device_error(buf) == 0


def test_output_on_another_stream_takes_no_memory_in_use():
    """The result of a call on a side stream may not land in memory that the current stream still reads."""
    x, wq, ws = torch.randn(256, 64, device="cuda"), torch.ones(64, 64, dtype=torch.int8, device="cuda"), torch.ones(64, device="cuda")
    copy = torch.empty(256, 64, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        kept = torch.full((256, 64), 7.0, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(2_000_000)          # about a millisecond
        copy.copy_(kept)
        del kept
        hstu.hstu_linear_i8(x, wq, ws, stream=side)
        torch.cuda.synchronize()
        assert (copy == 7.0).all()
