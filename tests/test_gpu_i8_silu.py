"""GPU tests of the 8-bit linear layer's SiLU where it is small: pre-activations far below 0.

With an identity for w_q, scales of 1 for its channels and a largest element of 127 / 8, the rows' scale is 1 / 8 and the
pre-activation is code / 8 + bias, exact in fp32 for the biases used here.  What is left is the activation and one rounding:
  bf16: half a step, 2^-8 |y|, and the fp32 roundings of x / (1 + exp(-x)): the exponent's argument (2^-23 |x|), the
        exponential, the sum, the reciprocal and the product (2^-21 together), relative to y
  fp32: the same with 2^-24 |y| for the last rounding
Below x = -87 the exponential leaves fp32's range and the result may be 0: 2^-118 covers |SiLU(x)| there.
"""
import numpy as np
import pytest
import torch

import generative_recommender_attention_jagged_b200 as hstu

pytestmark = pytest.mark.gpu

N = 256


@pytest.mark.parametrize("T", [1, 300, 20000])     # 20000 x 256: more than one wave of single tiles
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bias", [None, -6.0, -24.0, -80.0])
def test_silu_of_negative_values_is_rounded_once(T, out, bias):
    rng = np.random.default_rng(T)
    code = rng.integers(-127, 128, size=(T, N))
    code[:, 0] = 127
    x = torch.from_numpy(code / 8.0).float().cuda()
    b = None if bias is None else torch.full((N,), bias, device="cuda")
    y = hstu.hstu_linear_i8(x, torch.eye(N, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda"), b, silu=True,
                            out_dtype=out).double().cpu().numpy()
    pre = code / 8.0 + (bias or 0.0)
    want = pre / (1 + np.exp(-pre))
    last = 2.0 ** -8 if out == torch.bfloat16 else 2.0 ** -24
    tol = np.abs(want) * (last + 2.0 ** -21 + 2.0 ** -23 * np.abs(pre)) + 2.0 ** -118
    err = np.abs(y - want)
    assert (err <= tol).all(), (float(pre.flat[(err / tol).argmax()]), float((err / tol).max()))
