"""GPU test of the attention's time buckets where the rows of one warp lie on both sides of a gap of 2^32 time units: for
some of them a block of keys crosses many bucket edges at short distances, for the others it lies in one bucket farther
away than 32 bits hold."""
import numpy as np
import pytest
import torch

import oracle
import synth

from .gpu_helpers import host64, rel_err, run_jagged, run_paged

pytestmark = pytest.mark.gpu

N, N_MAX = 64, 256
GAP = 4_310_000_000                        # above 2^32, and 2^28 below the next bucket edge


def timestamps():
    """Keys 0 .. 31 at doubling distances before t = 0, rows 32 .. 47 right behind, rows 48 .. 63 a gap later."""
    old = -np.exp2(np.maximum(28 - np.arange(32), 0)).astype(np.int64)
    return np.concatenate([old, np.arange(16), GAP + np.arange(16)]).astype(np.int64)


def test_the_timestamps_do_what_they_are_for():
    t = timestamps()
    assert (np.diff(t) >= 0).all()
    near, far = oracle.ts_bucket(t[40] - t[:32], 128), oracle.ts_bucket(t[60] - t[:32], 128)
    assert len(set(near.tolist())) > 20 and len(set(far.tolist())) == 1
    assert (t[48:, None] - t[:48] >= 2 ** 32).all() and far[0] == 73


@pytest.mark.parametrize("bucket", [73, 62, 40, 0])
def test_one_hot_bucket_jagged(bucket):
    b = synth.jagged_batch([N], 2, 128, N_MAX, rng=np.random.default_rng(bucket))
    b.timestamps = timestamps()
    b.q.zero_(), b.k.zero_()
    b.rab_pos[:], b.rab_ts[:] = 0, 0
    b.rab_ts[bucket] = 4.0
    want = oracle.batch_attn(b, want_o=True)[1]
    assert rel_err(host64(run_jagged(b, raw_av=True)), want) <= 1e-2


@pytest.mark.parametrize("cached", [32, 40])
@pytest.mark.parametrize("bucket", [73, 62, 40, 0])
def test_one_hot_bucket_paged(bucket, cached):
    pb = synth.paged_batch([cached], [N - cached], [0], 2, 128, N_MAX, rng=np.random.default_rng(bucket), page_size=16,
                           dtype=torch.bfloat16)
    pb.timestamps[:] = timestamps()
    pb.q.zero_(), pb.k.zero_(), pb.k_pool.zero_()
    pb.rab_pos[:], pb.rab_ts[:] = 0, 0
    pb.rab_ts[bucket] = 4.0
    v = np.concatenate([pb.v_pool.double().numpy()[pb.kv_page_table[0][j // 16], :, j % 16][None] for j in range(cached)] +
                       [pb.v.double().numpy()])
    t, j = pb.timestamps, np.arange(N)
    want = np.zeros((N - cached, 2, 128))
    for i in range(cached, N):
        hit = (oracle.ts_bucket(t[i] - t, 128) == bucket) & (j <= i)
        want[i - cached] = 4 / (1 + np.exp(-4.0)) / N_MAX * v[hit].sum(0)
    assert rel_err(host64(run_paged(pb, raw_av=True)), want) <= 1e-2
