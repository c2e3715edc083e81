"""GPU tests of 4-bit attention calls that mix users with one new row and a user with hundreds, few on average."""
import numpy as np
import pytest
import torch

import generative_recommender_attention_jagged_b200 as hstu

from .gpu_helpers import dev
from .test_gpu_q4 import batch, check_raw
from .test_gpu_q4_precision import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("at", [0, 20, 39])
@pytest.mark.parametrize("acts,cands", [(200, 0), (1, 190), (97, 64)])
def test_one_long_user_among_short_ones(at, acts, cands):
    a, c = [1] * 40, [0] * 40
    a[at], c[at] = acts, cands
    a[7], a[30] = 0, 9                       # one without new rows, one with a row more than a pass takes
    rng = np.random.default_rng(at)
    pb, p4, val = batch(rng.integers(0, 90, size=40), a, c, 1, 128, 1024, 16, seed=acts, gamma=True)
    check(pb, p4, val, "few")
    pb, p4, val = batch(rng.integers(0, 90, size=40), a, c, 2, 64, 1024, 16, "f32", seed=acts)
    check_raw(pb, p4, val, False)


@pytest.mark.parametrize("B", [600, 1100])     # more users than are put in order
def test_one_long_user_among_many(B):
    a = [1] * B
    a[B // 2], a[3] = 100, 0
    pb, p4, val = batch([5] * B, a, [0] * B, 1, 128, 256, 8, seed=B)
    check_raw(pb, p4, val, True)


@pytest.mark.parametrize("d", [32, 128])
def test_more_users_than_a_grid_dimension_holds(d):
    """70,000 users of three cached keys and one new row, biases of 0: fp32 within 2^-24 (n + 8 d) of sum |S| |v| / n_max."""
    B, L, n_max = 70000, 3, 16
    g = torch.Generator(device="cuda").manual_seed(d)
    code = torch.randint(0, 256, (2, B, 1, 4, d // 2), generator=g, device="cuda", dtype=torch.uint8)
    meta = torch.tensor([0.25, 7.0], device="cuda").bfloat16().expand(B, 1, 4, 2).contiguous()
    q, k, v = torch.randn(3, B, 1, d, generator=g, device="cuda")
    table = torch.randperm(B, generator=g, device="cuda").int()
    ends = torch.arange(B + 1, device="cuda", dtype=torch.int32)
    ws = torch.empty(hstu.hstu_attn_paged_q4_workspace_size(batch=B, num_heads=1, head_dim=d, n_max=n_max, total_tokens=B,
                                                            dtype=torch.float32, max_cached_len=L),
                     dtype=torch.uint8, device="cuda")
    o = hstu.hstu_attn_fwd_paged_q4(
        q, k, v, q.view(B, d), ends, torch.zeros(B * (L + 1), dtype=torch.int64, device="cuda"), ends * (L + 1),
        torch.zeros(2 * n_max - 1, device="cuda"), torch.zeros(128, device="cuda"), code[0], code[1], meta, meta,
        table.view(B, 1), torch.full((B,), L, dtype=torch.int32, device="cuda"), n_max=n_max, max_cached_len=L, raw_av=True,
        workspace=ws)
    assert hstu.hstu_check_device_error(ws) == 0
    e = torch.arange(d, device="cuda")
    at, shift = 4 * (e // 8), 4 * (e % 8 // 2 + 4 * (e % 2))
    old = [0.25 * (((x[table.long(), 0, :L].long()[..., at + shift // 8] >> (shift % 8)) & 15).double() - 7) for x in code]
    K, V = (torch.cat([x, y.double()], 1) for x, y in zip(old, (k, v)))
    S = d ** -0.5 * (q.double() * K).sum(-1, keepdim=True)
    want, bound = (S * torch.sigmoid(S) * V).sum(1) / n_max, (S.abs() * V.abs()).sum(1) / n_max
    size = d ** -0.5 * (q.double().abs() * K.abs()).sum(-1, keepdim=True)
    bound = bound + (size * V.abs()).sum(1) / n_max
    assert ((o[:, 0].double() - want).abs() <= 2.0 ** -24 * (L + 1 + 8 * d) * bound + 1e-12).all()


def time_us(pb, p4):
    """Median time of a replayed call."""
    args = [dev(x) for x in (pb.q, pb.k, pb.v, pb.u, pb.new_offsets, pb.timestamps, pb.ts_offsets, pb.rab_pos, pb.rab_ts,
                             p4.k_pool, p4.v_pool, p4.k_scales, p4.v_scales, pb.kv_page_table, pb.cached_lens)]
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")

    def call():
        hstu.hstu_attn_fwd_paged_q4(*args, n_max=pb.n_max, max_cached_len=int(pb.cached_lens.max()), workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    times = []
    for _ in range(7):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end) * 1e3)
    return sorted(times)[3]


def test_a_long_user_costs_about_what_it_costs_alone():
    """The rows are given out by what each user has: together takes a few times as long as the two calls apart (the long
    user's own keys are done a row a warp), not its passes one behind the other, which was sixty times as long."""
    def make(acts, cached):
        return batch(cached, acts, [0] * len(acts), 4, 128, 4096, 32, seed=1)[:2]
    together = time_us(*make([400] + [1] * 63, [2000] + [500] * 63))
    apart = time_us(*make([400], [2000])) + time_us(*make([1] * 63, [500] * 63))
    assert together < 10 * apart, (together, apart)
