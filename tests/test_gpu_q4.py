"""GPU tests of the 4-bit paged cache (append, read-back, evict) and of the attention over it.

Append is compared code for code with the 64-bit definition.  The attention's raw sums o are compared with the dense
64-bit formula over the values the codes stand for, within the roundings of each path, all relative to
E = sum_j (|s_ij| + |bias_ij|) |v_j| / n_max, which bounds |a_ij| |v_j| since |SiLU(s)| <= |s|:
  CUDA cores, fp32: the score's dot product (d + 4 roundings of 2^-24 on sum_e |q_e k_e|, at most 4 E-units here), the
    SiLU and the sum over n keys (worst case n roundings): 2^-24 * (n + 8 d) * E covers them.
  tensor cores, bf16: half the score and the bias are rounded to bf16 (2 x 2^-9 on s / 2, passed on by a derivative of
    at most 2.2), tanh in bf16 (2^-8 on s / 2), the weight and the weight times the value's scale rounded once each
    (2^-9 on a, and 2^-9 on the product): at most 2^-9 * (2.2 + 1 + 1 + 1 + 1) = 6.2 * 2^-9, taken as 2^-6 E.
y = LayerNorm gate is compared by the framework's own bounds for the paged forward (gpu_helpers: 2e-2 and 1e-5 of max |y|).
"""
import dataclasses

import numpy as np
import pytest
import torch

import generative_recommender_attention_jagged_b200 as hstu
import oracle
import synth
from oracle import kv_cache as okv
from oracle import low_precision as lp

from .gpu_helpers import BF16_TOL, F32_TOL, dev, host64, rel_err

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- append, read, evict ------------------------------------------------------------------------
class Cache4:
    """A 4-bit cache on the device and the definition's copy of it (codes and meta words as integers)."""

    def __init__(self, B, H, d, num_pages, max_pages, P, seed):
        rng = np.random.default_rng(seed)
        self.H, self.d, self.P, self.num_pages = H, d, P, num_pages
        fill = lambda *s: torch.from_numpy(rng.integers(0, 256, size=s).astype(np.uint8))  # noqa: E731
        self.pools = [fill(num_pages, H, P, d // 2), fill(num_pages, H, P, d // 2)]
        self.metas = [torch.ones(num_pages, H, P, 2, dtype=torch.bfloat16) for _ in range(2)]
        self.free_np = rng.permutation(num_pages).astype(np.int32)
        self.o = [np.full((B, max_pages), -1, np.int64), np.zeros(B, np.int64), self.free_np.astype(np.int64), num_pages]
        self.ok = [p.numpy().copy() for p in self.pools] + [m.view(torch.int16).numpy().copy() for m in self.metas]
        self.g = [t.cuda() for t in self.pools + self.metas]
        self.table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.free, self.fc = dev(self.free_np), torch.tensor([num_pages], dtype=torch.int32, device="cuda")

    def append(self, k, v, counts, num_append=None, ws=None):
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        ws = hstu.hstu_kv_append_q4(k.cuda(), v.cuda(), dev(off), *self.g, self.table, self.lens, self.free, self.fc,
                                    num_append=dev(num_append, torch.int32), workspace=ws)
        status = hstu.hstu_check_device_error(ws)
        rows = []
        for x in (k, v):                 # what the definition stores, as integers
            codes, s, z = lp.quant4(x.double().numpy())
            meta = torch.from_numpy(np.stack([s, z], -1)).bfloat16().view(torch.int16).numpy()
            rows.append((lp.pack4(codes), meta))
        new = [None, None, None, None]
        st = okv.OK
        for i in range(2):               # the allocator's model moves bytes and meta words alike
            st, new[i], _, *rest = okv.kv_append(self.ok[i], self.ok[i], *self.o, rows[i][0], rows[i][0], off, num_append)
            _, new[2 + i], _, *rest = okv.kv_append(self.ok[2 + i], self.ok[2 + i], *self.o, rows[i][1], rows[i][1], off,
                                                    num_append)
        if st == okv.OK:
            self.ok, self.o = new, rest
        return status, st

    def assert_same(self):
        for i in range(2):
            assert np.array_equal(self.g[i].cpu().numpy(), self.ok[i])
            got, want = self.g[2 + i].cpu().float().numpy(), torch.from_numpy(self.ok[2 + i]).view(torch.bfloat16).float().numpy()
            assert np.array_equal(got, want, equal_nan=True)
        assert np.array_equal(self.table.cpu().numpy(), self.o[0])
        assert np.array_equal(self.lens.cpu().numpy(), self.o[1])
        assert int(self.fc.item()) == self.o[3]


def rows_of(rng, T, H, d, dtype):
    x = rng.standard_normal((T, H, d)).astype(np.float32) * np.exp(rng.standard_normal((T, H, 1))).astype(np.float32)
    x[0::5] = np.abs(x[0::5])
    x[1::7] *= 0.5 + 0.5 * np.tanh(x[1::7] / 2)
    if T > 8:
        x[2], x[3], x[4] = 0, 5.0, -5.0
        x[5, 0, 3], x[6, 0, 1], x[7] = np.nan, np.inf, 1e-38
    return torch.from_numpy(x).to(DT[dtype])


@pytest.mark.parametrize("d,P,H,dtype", [(128, 32, 4, "bf16"), (128, 24, 1, "f32"), (64, 8, 3, "bf16"), (32, 1, 2, "f32"),
                                         (96, 17, 2, "bf16"), (160, 16, 1, "bf16"), (256, 64, 2, "f32"),
                                         (224, 5, 3, "bf16")])
def test_append_is_exact_over_sequences(d, P, H, dtype):
    rng = np.random.default_rng(d * 100 + P)
    B = 5
    c = Cache4(B, H, d, num_pages=max(20, 400 // P), max_pages=max(4, 200 // P), P=P, seed=d)
    for step in range(6):
        counts = rng.integers(0, 40, size=B)
        if step == 3:
            counts = np.array([1, 0, 1, 1, 1])
        acts = np.minimum(counts, rng.integers(0, 40, size=B)).astype(np.int32)
        T = int(counts.sum())
        status, st = c.append(rows_of(rng, T, H, d, dtype), rows_of(rng, T, H, d, dtype), counts,
                              acts if step % 2 else None)
        assert status == st
        c.assert_same()
        if step == 4:
            mask = dev(np.array([1, 0, 0, 1, 0], np.int32))
            ws = hstu.hstu_kv_evict(mask, c.g[0], c.table, c.lens, c.free, c.fc)
            assert hstu.hstu_check_device_error(ws) == 0
            st, *c.o = okv.kv_evict(*c.o, [1, 0, 0, 1, 0], P, c.num_pages)
            assert st == 0
            c.assert_same()


def test_append_many_users_and_long_rows():
    rng = np.random.default_rng(8)
    B, H, d, P = 1300, 2, 32, 8              # more users than one block has threads
    c = Cache4(B, H, d, num_pages=1400, max_pages=3, P=P, seed=1)
    counts = (rng.random(B) < 0.5) * rng.integers(0, 20, size=B)
    counts[1299] = 11
    T = int(counts.sum())
    assert c.append(rows_of(rng, T, H, d, "bf16"), rows_of(rng, T, H, d, "bf16"), counts) == (0, 0)
    c.assert_same()


@pytest.mark.parametrize("B", [255, 256, 257])
def test_append_users_of_one_block(B):
    rng = np.random.default_rng(B)
    c = Cache4(B, 1, 32, num_pages=2 * B, max_pages=3, P=8, seed=B)
    for _ in range(2):
        counts = rng.integers(0, 8, size=B)
        counts[-1] = 5
        T = int(counts.sum())
        assert c.append(rows_of(rng, T, 1, 32, "bf16"), rows_of(rng, T, 1, 32, "bf16"), counts) == (0, 0)
        c.assert_same()


def test_the_other_pools_append_takes_no_4bit_pool():
    c = Cache4(2, 1, 32, num_pages=4, max_pages=2, P=8, seed=1)
    k = torch.zeros(3, 1, 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(KeyError):
        hstu.hstu_kv_append(k, k, dev(np.array([0, 2, 3], np.int32)), c.g[0], c.g[1], c.table, c.lens, c.free, c.fc)
    c.assert_same()


def test_append_failures_change_nothing():
    rng = np.random.default_rng(4)
    H, d = 2, 64
    c = Cache4(3, H, d, num_pages=5, max_pages=8, P=32, seed=2)
    x = rows_of(rng, 200, H, d, "bf16")
    assert c.append(x, x, [100, 90, 10]) == (okv.ERR_POOL, okv.ERR_POOL)
    c.assert_same()
    assert c.append(x[:80], x[:80], [40, 30, 10]) == (0, 0)
    c.assert_same()
    c.table[0, 1] = 99                       # the partly filled last page of user 0
    c.o[0][0, 1] = 99
    assert c.append(x[:5], x[:5], [5, 0, 0]) == (okv.ERR_PAGE, okv.ERR_PAGE)
    c.assert_same()
    assert c.append(x[:5], x[:5], [2, 2, 1], np.array([3, 0, 0])) == (okv.ERR_LENGTH, okv.ERR_LENGTH)
    c.assert_same()
    assert c.append(x[:0], x[:0], [0, 0, 0]) == (0, 0)
    c.assert_same()


def test_append_takes_strided_rows():
    rng = np.random.default_rng(6)
    H, d, T = 4, 128, 33
    uvqk = torch.from_numpy(rng.standard_normal((T, 4 * H * d)).astype(np.float32)).bfloat16()
    _, v, _, k = hstu.split_uvqk(uvqk, H, d)
    c = Cache4(2, H, d, num_pages=10, max_pages=4, P=16, seed=3)
    w = uvqk.cuda()
    _, vg, _, kg = hstu.split_uvqk(w, H, d)
    ws = hstu.hstu_kv_append_q4(kg, vg, dev(np.array([0, 20, 33], np.int32)), *c.g, c.table, c.lens, c.free, c.fc)
    assert hstu.hstu_check_device_error(ws) == 0
    got = [t.clone() for t in c.g]
    d2 = Cache4(2, H, d, num_pages=10, max_pages=4, P=16, seed=3)
    assert d2.append(k.contiguous(), v.contiguous(), [20, 13]) == (0, 0)
    d2.assert_same()
    assert all(torch.equal(a, b) for a, b in zip(got, d2.g))


@pytest.mark.parametrize("d,P,dtype", [(128, 32, "bf16"), (64, 7, "f32"), (256, 128, "bf16")])
def test_read_gives_the_stored_values(d, P, dtype):
    rng = np.random.default_rng(d + P)
    H = 2
    c = Cache4(3, H, d, num_pages=60, max_pages=20, P=P, seed=4)
    k, v = rows_of(rng, 150, H, d, "f32"), rows_of(rng, 150, H, d, "f32")
    assert c.append(k, v, [70, 0, 80]) == (0, 0)
    starts, n = [3, 0, 0], [67, 0, 41]
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    total = int(off[-1]) + 2                  # two rows behind the last user
    ko = torch.full((total, H, d), -3.0, dtype=DT[dtype], device="cuda")
    vo = ko.clone()
    ws = torch.empty(hstu.hstu_kv_q4_workspace_size(3), dtype=torch.uint8, device="cuda")
    hstu.hstu_kv_read_q4(*c.g, c.table, c.lens, dev(np.array(starts, np.int32)), dev(off), total_tokens=total,
                         dtype=DT[dtype], k_out=ko, v_out=vo, workspace=ws)
    assert hstu.hstu_check_device_error(ws) == 0
    for x, o in ((k, ko), (v, vo)):
        val = lp.dequant4(*lp.quant4(x.double().numpy()))
        want = torch.from_numpy(np.concatenate([val[3:70], val[70:111]])).to(torch.float32).to(DT[dtype])
        assert torch.equal(torch.nan_to_num(o[:-2].cpu(), nan=77.0), torch.nan_to_num(want, nan=77.0))
        assert (o[-2:] == -3.0).all()


def test_read_reports_bad_ranges_and_pages_and_leaves_their_rows():
    rng = np.random.default_rng(1)
    H, d, P = 1, 32, 8
    c = Cache4(2, H, d, num_pages=10, max_pages=4, P=P, seed=5)
    x = rows_of(rng, 30, H, d, "bf16")
    assert c.append(x, x, [20, 10]) == (0, 0)
    ws = torch.empty(hstu.hstu_kv_q4_workspace_size(2), dtype=torch.uint8, device="cuda")

    def read(starts, n):
        out = torch.full((sum(n), H, d), -3.0, dtype=torch.bfloat16, device="cuda")
        hstu.hstu_kv_read_q4(*c.g, c.table, c.lens, dev(np.array(starts, np.int32)),
                             dev(np.array([0, n[0], sum(n)], np.int32)), total_tokens=sum(n), k_out=out,
                             v_out=out.clone(), workspace=ws)
        return hstu.hstu_check_device_error(ws), out

    assert read([0, 0], [20, 10])[0] == 0
    status, out = read([15, 0], [6, 10])      # one token past user 0's last
    assert status == -4 and (out[5] == -3.0).all() and not (out[6:] == -3.0).all(-1).any()
    assert read([-1, 0], [3, 1])[0] == -4
    c.table[1, 1] = 10
    status, out = read([0, 0], [20, 10])
    assert status == -9 and (out[28:] == -3.0).all()


# ---- attention --------------------------------------------------------------------------------------
def run_q4(pb, p4, *, raw_av=False, workspace=None, num_splits=None, **kw):
    return hstu.hstu_attn_fwd_paged_q4(
        dev(pb.q), dev(pb.k), dev(pb.v), dev(pb.u), dev(pb.new_offsets, torch.int32), dev(pb.timestamps, torch.int64),
        dev(pb.ts_offsets, torch.int32), dev(pb.rab_pos, torch.float32), dev(pb.rab_ts, torch.float32), dev(p4.k_pool),
        dev(p4.v_pool), dev(p4.k_scales), dev(p4.v_scales), dev(pb.kv_page_table, torch.int32),
        dev(pb.cached_lens, torch.int32), n_max=pb.n_max, alpha=pb.alpha,
        num_candidates=dev(pb.num_candidates, torch.int32), ln_gamma=dev(pb.ln_gamma, torch.float32),
        ln_beta=dev(pb.ln_beta, torch.float32), ln_eps=pb.ln_eps, num_splits=num_splits,
        max_cached_len=int(pb.cached_lens.max()), raw_av=raw_av, workspace=workspace, **kw)


def dense(pb):
    """o and E (see above) of every new row in 64 bits, user by user; pb's pools hold values."""
    H, d, P = pb.num_heads, pb.head_dim, pb.page_size
    kp, vp = pb.k_pool.double().numpy(), pb.v_pool.double().numpy()
    q, k, v = (x.double().numpy() for x in (pb.q, pb.k, pb.v))
    O, E = np.zeros((len(q), H, d)), np.zeros((len(q), H, d))
    for u in range(pb.batch):
        r0, r1, L = int(pb.new_offsets[u]), int(pb.new_offsets[u + 1]), int(pb.cached_lens[u])
        if r1 == r0:
            continue
        n = L + r1 - r0
        h = n - (0 if pb.num_candidates is None else int(pb.num_candidates[u]))
        idx = [(int(pb.kv_page_table[u][j // P]), j % P) for j in range(L)]
        K = np.concatenate([np.array([kp[p, :, s] for p, s in idx]).reshape(L, H, d), k[r0:r1]])
        V = np.concatenate([np.array([vp[p, :, s] for p, s in idx]).reshape(L, H, d), v[r0:r1]])
        ts = pb.timestamps[pb.ts_offsets[u]:pb.ts_offsets[u + 1]]
        j = np.arange(n)
        for i in range(L, n):
            ok = j <= i if i < h else (j < h) | (j == i)
            bias = (pb.rab_pos.astype(np.float64)[min(i, h) - np.minimum(j, h) + pb.n_max - 1] +
                    pb.rab_ts.astype(np.float64)[oracle.ts_bucket(ts[i] - ts, len(pb.rab_ts))])[ok]
            S = pb.alpha * np.einsum("hd,jhd->jh", q[r0 + i - L], K[ok])
            s = S + bias[:, None]
            O[r0 + i - L] = np.einsum("jh,jhd->hd", s / (1 + np.exp(-s)), V[ok]) / pb.n_max
            E[r0 + i - L] = np.einsum("jh,jhd->hd", np.abs(S) + np.abs(bias)[:, None], np.abs(V[ok])) / pb.n_max
    return O, E


def check_raw(pb, p4, val, tc, **kw):
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    o = run_q4(pb, p4, raw_av=True, workspace=ws, **kw).double().cpu().numpy()
    assert hstu.hstu_check_device_error(ws) == 0
    O, E = dense(val)
    n = int(max(pb.cached_lens + np.diff(pb.new_offsets)))
    tol = (2.0 ** -6 if tc else 2.0 ** -24 * (n + 8 * pb.head_dim)) * E
    assert (np.abs(o - O) <= tol + 1e-12).all(), float((np.abs(o - O) / (E + 1e-12)).max())
    return o


def check_y(pb, p4, val, **kw):
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    y = run_q4(pb, p4, workspace=ws, **kw)
    assert hstu.hstu_check_device_error(ws) == 0
    want = oracle.batch_paged(val)[0] if isinstance(oracle.batch_paged(val), tuple) else oracle.batch_paged(val)
    assert rel_err(host64(y), want) < (F32_TOL if pb.q.dtype == torch.float32 else BF16_TOL)
    return y


def batch(cached, acts, cands, H=4, d=128, n_max=1024, P=32, dtype="bf16", seed=0, gamma=False):
    rng = np.random.default_rng(seed)
    pb = synth.paged_batch(cached, acts, cands, H, d, n_max, rng=rng, page_size=P, dtype=DT[dtype])
    if gamma:
        pb = dataclasses.replace(pb, ln_gamma=(1 + 0.2 * rng.standard_normal(H * d)).astype(np.float32),
                                 ln_beta=(0.2 * rng.standard_normal(H * d)).astype(np.float32))
    return (pb, *lp.quantised(pb))


CASES = [
    # cached, new actions, candidates, H, d, page
    ([0], [1], [0], 4, 128, 32),
    ([1], [1], [0], 4, 128, 32),
    ([100], [1], [0], 4, 128, 32),
    ([31, 32, 33, 0], [1, 1, 1, 1], [0, 0, 0, 0], 4, 128, 32),
    ([300, 5, 129], [1, 0, 1], [0, 1, 0], 2, 128, 8),
    ([500, 127, 128], [4, 4, 0], [4, 0, 8], 1, 128, 24),
    ([640, 0, 77], [0, 16, 3], [16, 0, 13], 4, 128, 16),
    ([200, 130], [17, 0], [0, 33], 4, 128, 128),
    ([257, 0, 64], [40, 100, 0], [24, 28, 128], 4, 128, 32),
    ([90, 400], [130, 1], [5, 300], 2, 128, 40),
    ([700], [150], [140], 4, 128, 1),
    ([33, 0, 150], [5, 7, 0], [2, 0, 9], 8, 128, 64),
    ([64, 3], [3, 9], [4, 0], 3, 64, 24),
    ([50], [6], [3], 4, 32, 7),
    ([40, 2], [2, 1], [1, 1], 3, 256, 16),
    ([45], [5], [0], 5, 96, 20),
    ([70, 20], [10, 3], [4, 12], 2, 64, 16),
    ([70, 20], [10, 3], [4, 12], 2, 96, 16),
    ([70, 20], [8, 0], [0, 8], 4, 128, 16),
    ([70, 20], [9, 0], [0, 8], 4, 128, 16),
]


@pytest.mark.parametrize("cached,acts,cands,H,d,P", CASES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_matches_definition(cached, acts, cands, H, d, P, dtype):
    pb, p4, val = batch(cached, acts, cands, H, d, 1024, P, dtype, seed=len(cached) + d + P, gamma=True)
    tc = dtype == "bf16"
    check_raw(pb, p4, val, tc)
    check_y(pb, p4, val)


@pytest.mark.parametrize("splits", [1, 2, 7, 64])
@pytest.mark.parametrize("acts,cands", [([1, 1], [0, 0]), ([9, 3], [2, 5]), ([70, 90], [20, 64])])
def test_splits_do_not_change_the_result(splits, acts, cands):
    pb, p4, val = batch([611, 95], acts, cands, seed=splits)
    check_raw(pb, p4, val, True, num_splits=splits)
    check_y(pb, p4, val, num_splits=splits)


@pytest.mark.parametrize("kw", [dict(force_simt=True), dict(precise_silu=True)])
@pytest.mark.parametrize("acts", [[1, 2], [60, 70]])
def test_flags(kw, acts):
    pb, p4, val = batch([300, 41], acts, [1, 0], seed=3)
    check_raw(pb, p4, val, "force_simt" not in kw, **kw)
    check_y(pb, p4, val, **kw)


@pytest.mark.parametrize("acts", [[1], [5], [40], [200]])
def test_all_weights_negative_and_large_scores(acts):
    """Scores of both signs far from 0 (weights near the score itself and near -0)."""
    pb, p4, val = batch([200], acts, [0], seed=9)
    pb = dataclasses.replace(pb, alpha=1.0)
    val = dataclasses.replace(val, alpha=1.0)
    check_raw(pb, p4, val, True)


@pytest.mark.parametrize("rows", [1, 12, 130])
def test_nan_row_reaches_only_the_rows_that_see_it(rows):
    """A cached token whose value row is not finite makes its own user's rows NaN (candidates and actions alike: all
    follow it) and no other user's; new rows behind a row do not reach it."""
    pb, p4, val = batch([100, 60], [rows, rows], [0, 0], seed=12)
    pid = int(pb.kv_page_table[1][0])
    p4.v_scales[pid, 2, 5, 0] = float("nan")
    y = run_q4(pb, p4).float().cpu()
    assert torch.isfinite(y[:rows]).all() and torch.isnan(y[rows:]).all()
    # a NaN in the last new token's k and v stays in its row
    pb, p4, val = batch([100, 60], [rows, rows], [0, 0], seed=13)
    pb.k[rows - 1], pb.v[rows - 1] = float("nan"), float("nan")
    y = run_q4(pb, p4).float().cpu()
    bad = torch.zeros(2 * rows, dtype=torch.bool)
    bad[rows - 1] = True
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()


@pytest.mark.parametrize("rows", [3, 50, 140])
def test_nan_candidate_stays_with_itself(rows):
    pb, p4, val = batch([70, 10], [1, 1], [rows, rows], seed=14)
    pb.k[2], pb.v[2] = float("nan"), float("inf")           # the second candidate of user 0
    y = run_q4(pb, p4).float().cpu()
    ok = torch.ones(len(y), dtype=torch.bool)
    ok[2] = False
    assert not torch.isfinite(y[2]).any() and torch.isfinite(y[ok]).all()


@pytest.mark.parametrize("rows", [1, 20, 200])
def test_device_errors(rows):
    pb, p4, val = batch([100, 60], [rows, rows], [0, 0], seed=20)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")

    def status(pb, **kw):
        run_q4(pb, p4, workspace=ws, **kw)
        return hstu.hstu_check_device_error(ws)

    assert status(pb) == 0
    t = pb.timestamps.copy()
    t[50] = t[51] + 5
    assert status(dataclasses.replace(pb, timestamps=t)) == -8
    t = pb.timestamps.copy()
    t[int(pb.ts_offsets[2]) - 1] -= 10 ** 7                   # the last token of the last user
    assert status(dataclasses.replace(pb, timestamps=t)) == -8
    for bad in (-1, p4.k_pool.shape[0]):
        table = pb.kv_page_table.copy()
        table[1, 1] = bad
        assert status(dataclasses.replace(pb, kv_page_table=table)) == -9
    assert status(dataclasses.replace(pb, cached_lens=np.array([100, 61], np.int32))) == -4
    assert status(dataclasses.replace(pb, cached_lens=np.array([-1, 60], np.int32))) == -4
    assert status(dataclasses.replace(pb, n_max=99 + rows, rab_pos=np.zeros(2 * (99 + rows) - 1, np.float32))) == -4
    assert status(dataclasses.replace(pb, num_candidates=np.array([0, rows + 1], np.int32))) == -4
    assert status(dataclasses.replace(pb, num_candidates=np.array([-1, 0], np.int32))) == -4
    off = pb.new_offsets.copy()
    off[1] = 2 * rows + 1
    assert status(dataclasses.replace(pb, new_offsets=off)) == -4
    off = pb.new_offsets.copy()
    off[2] -= 1
    assert status(dataclasses.replace(pb, new_offsets=off)) == -4
    off = pb.ts_offsets.copy()
    off[2] -= 1
    assert status(dataclasses.replace(pb, ts_offsets=off)) == -4
    assert status(pb) == 0
    check_raw(pb, p4, val, True)


@pytest.mark.parametrize("kw", [dict(), dict(force_simt=True)])
@pytest.mark.parametrize("rows", [1, 20, 200])
def test_offsets_past_the_timestamps_are_not_followed(rows, kw):
    """User 1's own numbers hold, but only user 0's wrong ones put its timestamps where they are said to be."""
    pb, p4, val = batch([100, 60], [rows, rows], [0, 0], seed=21)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    off = np.array([0, 10 ** 9, 10 ** 9 + 60 + rows], np.int32)
    run_q4(dataclasses.replace(pb, ts_offsets=off), p4, workspace=ws, **kw)
    assert hstu.hstu_check_device_error(ws) == -4
    check_raw(pb, p4, val, not kw, **kw)


@pytest.mark.parametrize("H,d", [(2, 128), (3, 64), (1, 32), (2, 96)])
@pytest.mark.parametrize("acts,cands", [([1, 2], [0, 0]), ([4, 9], [6, 3])])
def test_long_histories(H, d, acts, cands):
    """Sequences past the length up to which a weight of a few-row call is held in two bf16 terms."""
    pb, p4, val = batch([2500, 130], acts, cands, H, d, n_max=4096, seed=d, gamma=True)
    check_raw(pb, p4, val, True)
    check_y(pb, p4, val)


@pytest.mark.parametrize("cached,acts,cands", [([2500, 130], [20, 9], [6, 3]), ([1500, 2300], [70, 140], [64, 128])])
def test_long_histories_with_many_rows(cached, acts, cands):
    """The packed weights of calls with long sequences."""
    pb, p4, val = batch(cached, acts, cands, 2, n_max=4096, seed=5, gamma=True)
    check_raw(pb, p4, val, True)
    check_raw(pb, p4, val, True, precise_silu=True)
    check_y(pb, p4, val)


@pytest.mark.parametrize("B,rows", [(150, 2), (513, 1), (600, 3), (530, 17)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_users(B, rows, dtype):
    """More users than are put in order of their lengths, some without cached and some without new tokens."""
    rng = np.random.default_rng(B)
    cached = rng.integers(0, 40, size=B)
    acts = rng.integers(0, 2 * rows + 1, size=B)
    acts[7] = acts[-1] = rows
    pb, p4, val = batch(cached, acts, rng.integers(0, 2, size=B), 1, 128, 256, 8, dtype, seed=B)
    check_raw(pb, p4, val, dtype == "bf16")


def test_one_user_has_most_of_the_rows():
    pb, p4, val = batch([3] * 20 + [333], [1] * 20 + [150], [0] * 20 + [90], 2, seed=22)
    check_raw(pb, p4, val, True)
    check_y(pb, p4, val)
    pb, p4, val = batch([3] * 20 + [333], [1] * 20 + [150], [0] * 20 + [90], 2, 64, dtype="f32", seed=23)
    check_raw(pb, p4, val, False)


def test_users_without_new_rows_are_checked_in_small_calls():
    pb, p4, val = batch([100, 60, 20], [1, 0, 2], [0, 0, 0], seed=24)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    table = pb.kv_page_table.copy()
    table[1, 0] = p4.k_pool.shape[0]
    run_q4(dataclasses.replace(pb, kv_page_table=table), p4, workspace=ws)
    assert hstu.hstu_check_device_error(ws) == -9
    check_raw(pb, p4, val, True)


def test_no_new_rows():
    pb, p4, _ = batch([10, 20], [0, 0], [0, 0], seed=2)
    assert run_q4(pb, p4).shape == (0, 512)


@pytest.mark.parametrize("gap", [1, 40_000_000_000])
@pytest.mark.parametrize("acts", [[2], [70]])
def test_time_gaps(gap, acts):
    """Equal timestamps and gaps beyond 32 bits."""
    pb, p4, val = batch([250], acts, [2], seed=30)
    rng = np.random.default_rng(31)
    t = np.cumsum(rng.integers(0, 2, size=len(pb.timestamps)).astype(np.int64)) * gap - 10 ** 12
    t[-2:] = t[-3]
    pb, val = dataclasses.replace(pb, timestamps=t), dataclasses.replace(val, timestamps=t)
    check_raw(pb, p4, val, True)


@pytest.mark.parametrize("acts,cands", [([1, 1, 1], [0, 0, 0]), ([3, 9, 5], [2, 0, 7]), ([60, 100, 10], [20, 30, 100])])
def test_captured_replay_other_stream_and_repeat(acts, cands):
    pb, p4, val = batch([300, 0, 77], acts, cands, seed=40)
    args = [dev(x) for x in (pb.q, pb.k, pb.v, pb.u)]
    ints = [dev(pb.new_offsets, torch.int32), dev(pb.timestamps, torch.int64), dev(pb.ts_offsets, torch.int32),
            dev(pb.rab_pos, torch.float32), dev(pb.rab_ts, torch.float32)]
    pool = [dev(x) for x in (p4.k_pool, p4.v_pool, p4.k_scales, p4.v_scales)]
    tail = [dev(pb.kv_page_table, torch.int32), dev(pb.cached_lens, torch.int32)]
    kw = dict(n_max=pb.n_max, alpha=pb.alpha, num_candidates=dev(pb.num_candidates, torch.int32), max_cached_len=300)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    out = torch.empty(len(pb.q), 512, dtype=torch.bfloat16, device="cuda")

    def call(**more):
        return hstu.hstu_attn_fwd_paged_q4(*args, *ints, *pool, *tail, **kw, **more)

    first = call(out=out, workspace=ws).clone()
    assert torch.equal(call(), first)                        # the same bits each time
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=out, workspace=ws)
    q0 = args[0].clone()
    args[0].copy_(torch.randn_like(args[0].float()).to(torch.bfloat16))
    want = call().clone()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    args[0].copy_(q0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    again = call()                                           # two calls at once, workspaces of their own
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, first) and torch.equal(again, first)


def test_rows_from_a_projection_and_a_serving_step():
    """A layer's serving step in low precision: the 8-bit projection, attention over the 4-bit cache, the new tokens
    appended, the next request over the longer cache, the 8-bit output projection.  Each operator is compared with the
    definition on its own inputs (the bf16 tensors the step before produced)."""
    rng = np.random.default_rng(50)
    H, d, B, P = 4, 128, 3, 16
    D = H * d
    w1 = torch.from_numpy(rng.standard_normal((256, 4 * D)).astype(np.float32) / 16)
    w2 = torch.from_numpy(rng.standard_normal((D, 256)).astype(np.float32) / 23)
    q1, q2 = hstu.hstu_quant_i8_weight(w1.cuda()), hstu.hstu_quant_i8_weight(w2.bfloat16().cuda())
    c = Cache4(B, H, d, num_pages=40, max_pages=10, P=P, seed=6)
    ts = [np.cumsum(rng.integers(1, 5000, size=200)).astype(np.int64) for _ in range(B)]
    rab_pos, rab_ts = synth.draw_rab(rng, 256)
    for step, counts in enumerate(([30, 1, 0], [5, 20, 17], [1, 1, 1], [40, 3, 60])):
        T = sum(counts)
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        x = torch.from_numpy(rng.standard_normal((T, 256)).astype(np.float32)).bfloat16()
        f1 = hstu.hstu_linear_i8(x.cuda(), *q1, silu=True)
        want = lp.linear_i8(x.double().numpy(), q1[0].cpu().numpy(), q1[1].cpu().numpy(), silu=True)
        assert np.abs(f1.double().cpu().numpy() - want).max() <= 2.0 ** -7 * np.abs(want).max()
        u, v, q, k = hstu.split_uvqk(f1, H, d)
        lens = c.lens.cpu().numpy()
        n = lens + counts
        val = synth.PagedBatch(
            q=q.cpu().contiguous(), k=k.cpu().contiguous(), v=v.cpu().contiguous(), u=u.cpu().contiguous(),
            new_offsets=off, timestamps=np.concatenate([t[:m] for t, m in zip(ts, n)]),
            ts_offsets=synth.offsets_from_lengths(n), num_candidates=np.zeros(B, np.int32), rab_pos=rab_pos,
            rab_ts=rab_ts, k_pool=lp.dequant_pool(c.g[0].cpu(), c.g[2].cpu()),
            v_pool=lp.dequant_pool(c.g[1].cpu(), c.g[3].cpu()), kv_page_table=c.table.cpu().numpy(), cached_lens=lens,
            page_size=P, alpha=d ** -0.5, n_max=256, num_heads=H, head_dim=d)
        y = hstu.hstu_attn_fwd_paged_q4(q, k, v, u, dev(off), dev(val.timestamps), dev(val.ts_offsets), dev(rab_pos),
                                        dev(rab_ts), *c.g, c.table, c.lens, n_max=256)
        ref = oracle.batch_paged(val)
        ref = ref[0] if isinstance(ref, tuple) else ref
        assert rel_err(host64(y), ref) < BF16_TOL
        assert c.append(val.k, val.v, counts) == (0, 0)
        c.assert_same()
        out = hstu.hstu_linear_i8(y, *q2)
        want = lp.linear_i8(y.double().cpu().numpy(), q2[0].cpu().numpy(), q2[1].cpu().numpy())
        assert np.abs(out.double().cpu().numpy() - want).max() <= 2.0 ** -7 * np.abs(want).max()


def test_refusals():
    pb, p4, _ = batch([10], [2], [0], seed=1)
    bad = [
        (dict(k_pool=p4.k_pool[..., :32].contiguous()), ValueError), (dict(k_scales=p4.k_scales.float()), ValueError),
        (dict(v_pool=p4.v_pool.to(torch.int8)), ValueError), (dict(v_scales=p4.v_scales[:1]), ValueError),
        (dict(v_scales=p4.v_scales.transpose(1, 2)), ValueError),
    ]
    for change, err in bad:
        with pytest.raises(err):
            run_q4(pb, dataclasses.replace(p4, **change))
    with pytest.raises(ValueError):
        run_q4(pb, p4, out=torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        run_q4(dataclasses.replace(pb, rab_pos=pb.rab_pos[:-2]), p4)
    with pytest.raises(hstu.HstuError, match="WORKSPACE"):
        run_q4(pb, p4, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(hstu.HstuError, match="INVALID"):
        run_q4(pb, p4, num_splits=65)
