"""GPU tests of the 4-bit cache's read-back with offsets that do not fit the output."""
import numpy as np
import pytest
import torch

import generative_recommender_attention_jagged_b200 as hstu

from .gpu_helpers import dev

pytestmark = pytest.mark.gpu

H, D, P = 2, 32, 8
LENGTH = -4


def read(offsets, total, lens=(20, 10), fill=-3.0):
    """Status and keys of a read-back of a cache of two users whose rows all stand for 2.0."""
    code = torch.full((8, H, P, D // 2), 0x22, dtype=torch.uint8, device="cuda")
    meta = torch.tensor([1.0, 0.0], dtype=torch.bfloat16, device="cuda").expand(8, H, P, 2).contiguous()
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    out = torch.full((total, H, D), fill, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(hstu.hstu_kv_q4_workspace_size(2), dtype=torch.uint8, device="cuda")
    hstu.hstu_kv_read_q4(code, code, meta, meta, table, dev(np.array(lens, np.int32)), dev(np.zeros(2, np.int32)),
                         dev(np.array(offsets, np.int32)), total_tokens=total, k_out=out, v_out=out.clone(),
                         workspace=ws)
    return hstu.hstu_check_device_error(ws), out


@pytest.mark.parametrize("total", [30, 33])
def test_offsets_that_fit(total):
    status, out = read([0, 20, 30], total)
    assert status == 0 and (out[:30] == 2.0).all() and (out[30:] == -3.0).all()


@pytest.mark.parametrize("offsets,total", [
    ([0, 20, 30], 29),    # the last user's last row is behind the output
    ([0, 20, 30], 20),    # the whole last user is
    ([0, 20, 30], 7),
    ([0, 20, 30], 0),     # an output without rows
    ([0, 30, 20], 20),    # decreasing, and past the output in the middle
    ([0, 25, 20], 30),
    ([2, 20, 30], 30),
    ([-2, 20, 30], 30),
    ([5, 5, 5], 0),
])
def test_offsets_that_do_not_fit_are_reported(offsets, total):
    assert read(offsets, total)[0] == LENGTH


def test_no_rows():
    assert read([0, 0, 0], 0)[0] == 0
    status, out = read([0, 0, 0], 3)
    assert status == 0 and (out == -3.0).all()
