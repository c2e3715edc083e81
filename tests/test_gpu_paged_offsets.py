"""GPU test of the paged attention's checks: a user's numbers hold by themselves, but another user's wrong ones put its
timestamps past the array."""
import dataclasses

import numpy as np
import pytest
import torch

import generative_recommender_attention_jagged_b200 as hstu
import synth

from .gpu_helpers import run_paged

pytestmark = pytest.mark.gpu

LENGTH = -4


@pytest.mark.parametrize("force_simt", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [1, 20, 200])
@pytest.mark.parametrize("B", [2, 300, 1100])  # more users than a block has threads, than a block checks
def test_offsets_past_the_timestamps_are_not_followed(B, rows, dtype, force_simt):
    acts = [rows, rows] + [0] * (B - 2)
    pb = synth.paged_batch([100, 60] + [5] * (B - 2), acts, [0] * B, 2, 128, 512, rng=np.random.default_rng(rows),
                           page_size=32, dtype=dtype)
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    good = run_paged(pb, force_simt=force_simt, workspace=ws)
    assert hstu.hstu_check_device_error(ws) == 0
    off = pb.ts_offsets.copy()
    off[1:] += 10 ** 9
    run_paged(dataclasses.replace(pb, ts_offsets=off), force_simt=force_simt, workspace=ws)
    assert hstu.hstu_check_device_error(ws) == LENGTH
    assert torch.equal(run_paged(pb, force_simt=force_simt, workspace=ws), good)
    assert hstu.hstu_check_device_error(ws) == 0
