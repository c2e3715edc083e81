"""GPU tests of the 8-bit linear layer's integer sums beyond the 24 bits that fp32 holds exactly, up to the largest d_in.

Rows with a largest element of 127 have scale 1, the channels' scales are 1: with fp32 results y is the sum rounded once to
fp32.  With SiLU (another conversion) it is too: exp(-x) is 0 beside 1 for these x.
"""
import numpy as np
import pytest
import torch

import generative_recommender_attention_jagged_b200 as hstu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("T,N", [(100, 136), (1664, 1536)])      # single tiles; SM pairs
def test_sums_of_random_codes(T, N, silu):
    K = 8192
    rng = np.random.default_rng(T)
    x, w = rng.integers(100, 128, size=(T, K)), rng.integers(100, 128, size=(N, K))
    x[:, 0] = 127
    acc = torch.from_numpy(x).double().cuda() @ torch.from_numpy(w).double().cuda().T     # exact: below 2^53
    assert acc.min() > 2 ** 26 and (acc.long() % 2).any()
    y = hstu.hstu_linear_i8(torch.from_numpy(x).float().cuda(), torch.from_numpy(w).to(torch.int8).cuda(),
                            torch.ones(N, device="cuda"), silu=silu)
    assert torch.equal(y, acc.float())


@pytest.mark.parametrize("out,silu", [(torch.float32, False), (torch.float32, True), (torch.bfloat16, True)])
@pytest.mark.parametrize("T,N", [(40, 24), (1664, 1536)])
def test_longest_rows(T, N, out, silu):
    """d_in = 131072: row t has 127 in its first m_t places and 0 or, without SiLU, -127 behind, channel n 127 - n % 3
    everywhere; the last sums are 127 * 127 * 131072 = 0.98 * 2^31."""
    K = 131072
    m = torch.linspace(1, K, T).round().long().cuda()
    x = torch.full((T, K), 0.0 if silu else -127.0, dtype=torch.bfloat16, device="cuda")
    x[torch.arange(K, device="cuda") < m[:, None]] = 127.0
    c = 127 - torch.arange(N, device="cuda") % 3
    w = c.to(torch.int8)[:, None].expand(N, K).contiguous()
    acc = 127 * (m if silu else 2 * m - K)[:, None] * c
    assert acc.max() == 127 * 127 * K
    y = hstu.hstu_linear_i8(x, w, torch.ones(N, device="cuda"), silu=silu, out_dtype=out)
    if out == torch.float32:
        assert torch.equal(y, acc.float())
    else:                                      # one rounding, and the activation's 2^-21
        err = (y.double() - acc.double()).abs()
        assert (err <= (2.0 ** -8 + 2.0 ** -21 + 2.0 ** -24) * acc.double()).all()
