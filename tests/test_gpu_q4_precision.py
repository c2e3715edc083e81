"""GPU tests of the precision that the two paths of the 4-bit attention promise for bf16 calls (include/hstu.h): a weight in
fp16 under a power of two (few rows, or d other than 128), or in two bf16 terms (tcgen05), whatever n_max and max_seq_len are.

The raw sums o are compared with the 64-bit formula, element by element, within the roundings of the path.  With S the scaled
score, p and t the position and time bias, s = S + p + t, a = SiLU(s) (|SiLU'| <= 1.1), and half a step of bf16 being 2^-8:
  all paths    scores and biases added in fp32, 2^-22 (|S| + |p| + |t|); exponential and quotient (2 + 1.2 |s| + 4) 2^-23 |a|;
               the sum over n keys in fp32, some of it on the tensor cores (every 16 keys one sum, to 2^-22): (n + 64) 2^-23
  few rows     the products take 128 + code and subtract (128 + zero) sum q after them: d / 16 sums of 16 products, each to
               2^-22 of 143 sum |q|, twelve fp32 additions of q and one subtraction: below 2^-11 sum |q| for d <= 128,
               times alpha and the key's scale.  Weights of cached keys: 2^-11 |a|.  New keys: fp32
  tcgen05      d / 16 sums of 16 products, each to 2^-22: 2^-19 alpha sum |q k|; position bias, time bias and their sum in bf16
               (0 for values that bf16 holds); tanh to 2^-10.9, that is 2^-11.9 |s|; the weight in two terms, 2^-16 |a|
y = LayerNorm gate follows from o: with delta the row's largest error, mean and deviation move by at most 2 delta, so
  |dy| <= |u| (|gamma| rstd 2.1 delta (1 + |x|) + 2^-18 (|gamma x| + |beta|)) + 2^-8 |y|,  x the normalised element.
"""
import dataclasses

import numpy as np
import pytest
import torch

import generative_recommender_attention_jagged_b200 as hstu
import oracle

from .test_gpu_q4 import batch, run_q4

pytestmark = pytest.mark.gpu

def half_step(x):
    """The largest error of rounding x to bf16."""
    return np.where(torch.from_numpy(x).bfloat16().double().numpy() == x, 0, 2.0 ** -8 * np.abs(x))


def reference(pb, p4, val, path):
    """o and the bound on its error [T, H, d] in 64 bits."""
    H, d, P, alpha = pb.num_heads, pb.head_dim, pb.page_size, pb.alpha
    q, k, v = (x.double().numpy() for x in (pb.q, pb.k, pb.v))
    kp, vp, ks = val.k_pool.numpy(), val.v_pool.numpy(), p4.k_scales[..., 0].double().numpy()
    O, B = np.zeros((len(q), H, d)), np.zeros((len(q), H, d))
    for u in range(pb.batch):
        r0, r1, L = int(pb.new_offsets[u]), int(pb.new_offsets[u + 1]), int(pb.cached_lens[u])
        n = L + r1 - r0
        h = n - int(pb.num_candidates[u])
        at = [(int(pb.kv_page_table[u][j // P]), j % P) for j in range(L)]
        K = np.concatenate([np.array([kp[x, :, y] for x, y in at]).reshape(L, H, d), k[r0:r1]])
        V = np.concatenate([np.array([vp[x, :, y] for x, y in at]).reshape(L, H, d), v[r0:r1]])
        scale = np.concatenate([np.array([ks[x, :, y] for x, y in at]).reshape(L, H), np.zeros((r1 - r0, H))])
        ts = pb.timestamps[pb.ts_offsets[u]:pb.ts_offsets[u + 1]]
        j = np.arange(n)
        for i in range(L, n):
            ok = j <= i if i < h else (j < h) | (j == i)
            r = r0 + i - L
            p = pb.rab_pos.astype(np.float64)[min(i, h) - np.minimum(j, h) + pb.n_max - 1][ok][:, None]
            t = pb.rab_ts.astype(np.float64)[oracle.ts_bucket(ts[i] - ts, len(pb.rab_ts))][ok][:, None]
            S = alpha * np.einsum("hd,jhd->jh", q[r], K[ok])
            s = S + p + t
            a = s / (1 + np.exp(-s))
            cached = (j < L)[ok][:, None]
            da = 1.1 * 2.0 ** -22 * (np.abs(S) + np.abs(p) + np.abs(t)) + (6 + 1.2 * np.abs(s)) * 2.0 ** -23 * np.abs(a)
            if path == "few":
                da = da + 1.1 * alpha * scale[ok] * 2.0 ** -11 * np.abs(q[r]).sum(-1)
                da = da + np.where(cached, 2.0 ** -11 * np.abs(a), 0)
                da = da + np.where(cached, 0, 1.1 * d * 2.0 ** -24 * alpha * np.einsum("hd,jhd->jh", np.abs(q[r]), np.abs(K[ok])))
            else:
                da = da + 1.1 * 2.0 ** -19 * alpha * np.einsum("hd,jhd->jh", np.abs(q[r]), np.abs(K[ok]))
                da = da + 1.1 * (half_step(p) + half_step(t) + np.where(half_step(p) + half_step(t) > 0, 2.0 ** -8 * np.abs(p + t),
                                                                        half_step(p + t)))
                da = da + 2.0 ** -11.9 * np.abs(s) + 2.0 ** -16 * np.abs(a)
            O[r] = np.einsum("jh,jhd->hd", a, V[ok]) / pb.n_max
            B[r] = np.einsum("jh,jhd->hd", da + (n + 64) * 2.0 ** -23 * np.abs(a), np.abs(V[ok])) / pb.n_max
    return O, 1.01 * B                         # 1.01: products of two of these


def check(pb, p4, val, path, **kw):
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    o = run_q4(pb, p4, raw_av=True, workspace=ws, **kw).double().cpu().numpy()
    assert hstu.hstu_check_device_error(ws) == 0
    O, B = reference(pb, p4, val, path)
    assert (np.abs(o - O) <= B + 1e-15).all(), float((np.abs(o - O) / (B + 1e-15)).max())
    y = run_q4(pb, p4, workspace=ws, **kw).double().cpu().numpy()
    T = len(y)
    flat, delta = O.reshape(T, -1), B.reshape(T, -1).max(1, keepdims=True)
    rstd = 1 / np.sqrt(flat.var(1, keepdims=True) + pb.ln_eps)
    x = (flat - flat.mean(1, keepdims=True)) * rstd
    g, b, u = pb.ln_gamma.astype(np.float64), pb.ln_beta.astype(np.float64), pb.u.double().numpy()
    want = (g * x + b) * u
    tol = np.abs(u) * (np.abs(g) * rstd * 2.1 * delta * (1 + np.abs(x)) + 2.0 ** -18 * (np.abs(g * x) + np.abs(b)))
    tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    assert (np.abs(y - want) <= tol + 1e-15).all(), float((np.abs(y - want) / (tol + 1e-15)).max())


def biased(pb, val, bias, seed):
    """large: one time bias of 16, exact in bf16, so that the roundings of the weights outweigh all others; random: of the
    scores' size."""
    rng = np.random.default_rng(seed)
    if bias == "large":
        p, t = np.zeros_like(pb.rab_pos), np.full_like(pb.rab_ts, 16.0)
    else:
        p, t = (0.5 * rng.standard_normal(x.shape).astype(np.float32) for x in (pb.rab_pos, pb.rab_ts))
    return tuple(dataclasses.replace(x, rab_pos=p, rab_ts=t) for x in (pb, val))


FEW = [(3, 0, 128), (8, 2, 128), (3, 1, 96), (2, 2, 64), (3, 0, 32), (12, 3, 64), (9, 4, 32), (12, 0, 96)]
SIZES = [(256, None), (2049, None), (4096, 300)]        # n_max, max_seq_len


@pytest.mark.parametrize("bias", ["large", "random"])
@pytest.mark.parametrize("acts,cands,d", FEW)
@pytest.mark.parametrize("n_max,longest", SIZES)
def test_few_rows(acts, cands, d, n_max, longest, bias):
    pb, p4, val = batch([100, 7], [acts, 1], [cands, 0], 2, d, n_max, 16, seed=acts + d, gamma=True)
    pb, val = biased(pb, val, bias, d)
    check(pb, p4, val, "few", max_seq_len=longest)


@pytest.mark.parametrize("bias", ["large", "random"])
@pytest.mark.parametrize("acts,cands", [(20, 0), (40, 100)])
@pytest.mark.parametrize("n_max,longest", SIZES)
@pytest.mark.parametrize("precise", [False, True])
def test_many_rows(acts, cands, n_max, longest, precise, bias):
    pb, p4, val = batch([100, 7], [acts, 9], [cands, 0], 2, 128, n_max, 16, seed=acts, gamma=True)
    pb, val = biased(pb, val, bias, acts)
    check(pb, p4, val, "tcgen05", max_seq_len=longest, precise_silu=precise)


@pytest.mark.parametrize("d", [32, 128])
@pytest.mark.parametrize("kind", ["offset", "outlier"])
@pytest.mark.parametrize("rows,path", [(3, "few"), (30, "tcgen05")])
def test_queries_with_an_offset_or_an_outlier(rows, path, kind, d):
    """What the few-row kernel takes off after the product is 128 sum q, however small the score is."""
    if d != 128:
        path = "few"                           # 16 rows a pass
    pb, p4, val = batch([150], [rows], [0], 2, d, 1024, 16, seed=rows + d, gamma=True)
    if kind == "offset":
        pb.q.add_(8.0)
    else:
        pb.q[:, :, 5] = 300.0
    check(pb, p4, val, path)


@pytest.mark.parametrize("rows,path", [(1, "few"), (30, "tcgen05")])
def test_thousands_of_keys(rows, path):
    pb, p4, val = batch([2500, 2100], [rows, rows], [0, 0], 2, 128, 4096, 32, seed=rows, gamma=True)
    check(pb, p4, val, path)
    pb, val = biased(pb, val, "random", 3)
    check(pb, p4, val, path)


@pytest.mark.parametrize("acts,path", [(3, "few"), (20, "tcgen05")])
@pytest.mark.parametrize("n_max,longest", SIZES)
def test_weight_of_one_key(acts, path, n_max, longest):
    """One cached key a user, new values of 0: o is one weight times one row, with no other key's error to hide in."""
    pb, p4, val = batch([1] * 8, [acts] * 8, [0] * 8, 2, 128, n_max, 16, seed=acts, gamma=True)
    pb, val = biased(pb, val, "large", 1)
    pb.v.zero_()
    check(pb, p4, val, path, max_seq_len=longest)


@pytest.mark.parametrize("acts,d", [(2, 128), (30, 128), (2, 64), (12, 64), (3, 32), (12, 96)])
@pytest.mark.parametrize("cached", [20, 300, 3000])
def test_one_head_is_as_exact_as_its_rounding(cached, acts, d):
    """With one head nothing but what the weights' noise shares with the signal is left after LayerNorm.  y's own rounding
    has a root mean square of r; weights of 11 bits add at most 2^-3 of it where the terms are as large as their sum, so
    sqrt(1 + 2^-6) r, and the sum over keys of both signs is taken at up to four times its size: below 1.15 r."""
    pb, p4, val = batch([cached] * 4, [acts] * 4, [0] * 4, 1, d, cached + acts + 8, 32, seed=cached + d, gamma=True)
    y = run_q4(pb, p4).double().cpu().numpy()
    O, _ = reference(pb, p4, val, "few")
    flat = O.reshape(len(y), -1)
    x = (flat - flat.mean(1, keepdims=True)) / np.sqrt(flat.var(1, keepdims=True) + pb.ln_eps)
    want = (pb.ln_gamma.astype(np.float64) * x + pb.ln_beta) * pb.u.double().numpy()
    own = torch.from_numpy(want).bfloat16().double().numpy() - want
    assert np.sqrt(((y - want) ** 2).mean()) <= 1.15 * np.sqrt((own ** 2).mean())


@pytest.mark.parametrize("d", [32, 128])
@pytest.mark.parametrize("log2", [-110, -30, 30, 100])
def test_value_scales_far_from_one(log2, d):
    """Weights beyond fp16's range and below it: the values' scales times 2^log2 give o times 2^log2."""
    pb, p4, val = batch([150, 40], [3, 1], [1, 0], 2, d, 256, 16, seed=d, gamma=True)
    pb.v.zero_()
    p4.v_scales[..., 0] *= 2.0 ** log2
    val = dataclasses.replace(val, v_pool=val.v_pool * 2.0 ** log2)
    O, B = reference(pb, p4, val, "few")
    o = run_q4(pb, p4, raw_av=True).double().cpu().numpy()
    assert (np.abs(o - O) <= B + 2.0 ** -140).all()


@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_very_different_weights(d):
    """A row's scale is its own: a row of tiny weights beside rows of large ones, and beside one of NaN."""
    pb, p4, val = batch([100], [4], [0], 2, d, 256, 16, seed=d, gamma=True)
    pb.q[1] *= 2.0 ** -20
    pb, val = (dataclasses.replace(x, rab_pos=np.zeros_like(pb.rab_pos), rab_ts=np.zeros_like(pb.rab_ts)) for x in (pb, val))
    pb.v.zero_()
    O, B = reference(pb, p4, val, "few")
    o = run_q4(pb, p4, raw_av=True).double().cpu().numpy()
    assert (np.abs(o - O) <= B).all()
    pb.q[2] = float("nan")
    o = run_q4(pb, p4, raw_av=True).double().cpu().numpy()
    rest = [0, 1, 3]
    assert np.isnan(o[2]).all() and (np.abs(o - O) <= B)[rest].all()
