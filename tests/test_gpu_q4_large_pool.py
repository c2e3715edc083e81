"""GPU test of the 4-bit cache in a pool of more than 2^32 bytes: what is appended to, read from and attended to in its last
pages is, bit for bit, what a small pool gives."""
import numpy as np
import pytest
import torch

import generative_recommender_attention_jagged_b200 as hstu
import synth

from .gpu_helpers import dev

pytestmark = pytest.mark.gpu

H, D, P, B, WIDTH = 4, 128, 32, 2, 8
BIG = 2 ** 32 // (H * P * D // 2) + 1000


def run(num_pages, first, rows, force_simt=False):
    """Keys and values of 300 tokens appended to pages first, first + 1, ..., read back, and attended to by new rows."""
    g = torch.Generator().manual_seed(rows)
    k, v, q, kn, vn = (torch.randn(n, H, D, generator=g).bfloat16().cuda() for n in (300, 300, 2 * rows, 2 * rows, 2 * rows))
    pools = [torch.empty(num_pages, H, P, n, dtype=t, device="cuda") for n, t in
             ((D // 2, torch.uint8), (D // 2, torch.uint8), (2, torch.bfloat16), (2, torch.bfloat16))]
    table = torch.full((B, WIDTH), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    free = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
    free[:16] = torch.arange(first, first + 16, dtype=torch.int32, device="cuda")
    count = torch.tensor([16], dtype=torch.int32, device="cuda")
    off = dev(np.array([0, 130, 300], np.int32))
    ws = hstu.hstu_kv_append_q4(k, v, off, *pools, table, lens, free, count)
    assert hstu.hstu_check_device_error(ws) == 0 and int(table.max()) >= first
    back = hstu.hstu_kv_read_q4(*pools, table, lens, torch.zeros_like(lens), off, total_tokens=300)
    rng = np.random.default_rng(1)
    rab_pos, rab_ts = synth.draw_rab(rng, 1024)
    n = np.array([130 + rows, 170 + rows])
    ts = np.concatenate([np.cumsum(rng.integers(1, 900, size=m)) for m in n]).astype(np.int64)
    y = hstu.hstu_attn_fwd_paged_q4(q, kn, vn, q.flatten(1), dev(np.array([0, rows, 2 * rows], np.int32)), dev(ts),
                                    dev(synth.offsets_from_lengths(n)), dev(rab_pos), dev(rab_ts), *pools, table, lens,
                                    n_max=1024, max_cached_len=170, force_simt=force_simt)
    return (*back, y)


@pytest.mark.parametrize("rows,force_simt", [(2, False), (40, False), (2, True)])
def test_pages_behind_four_gigabytes(rows, force_simt):
    small = run(32, 3, rows, force_simt)
    large = run(BIG, BIG - 16, rows, force_simt)
    assert all(torch.equal(a, b) for a, b in zip(small, large))
    assert all(torch.isfinite(x.float()).all() for x in small)
