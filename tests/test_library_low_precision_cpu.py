"""CPU-only checks of the 8-bit linear layer's and the 4-bit cache's entry points: struct sizes, workspace sizes and
the refusals that come before any launch."""
import ctypes

import pytest
import torch

import generative_recommender_attention_jagged_b200 as hstu
from generative_recommender_attention_jagged_b200 import _lib, build as hbuild

A = ctypes.c_void_p(0x1000)       # never dereferenced: every call below is refused before a launch
ODD = ctypes.c_void_p(0x1008)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    hbuild.build()
    return _lib.load()


def lin(**kw):
    base = dict(rows=300, d_in=512, d_out=2048, x_stride=0, out_stride=0, dtype=_lib.DT_BF16, out_dtype=_lib.DT_BF16,
                flags=0)
    base.update(kw)
    return _lib.LinearI8Params(**base)


def test_linear_i8_struct_and_workspace(lib):
    assert ctypes.sizeof(_lib.LinearI8Params) == 48
    small, big = hstu.hstu_linear_i8_workspace_size(8, 512, 2048), hstu.hstu_linear_i8_workspace_size(80, 512, 2048)
    assert small >= 256 + 8 * 512 + 8 * 4 and big >= 256 + 80 * 512 + 80 * 4
    assert hstu.hstu_linear_i8_workspace_size(8, 500, 2048) == 0


@pytest.mark.parametrize("bad,want", [
    (dict(rows=-1), -1), (dict(d_in=0), -1), (dict(d_out=-8), -1), (dict(dtype=2), -1), (dict(out_dtype=7), -1),
    (dict(flags=2), -1), (dict(x_stride=256), -1), (dict(out_stride=64), -1), (dict(d_in=520), -3),
    (dict(d_out=2044), -3), (dict(x_stride=516), -3), (dict(out_stride=2052), -3), (dict(d_in=131088), -2),
    (dict(x_stride=514, dtype=_lib.DT_F32), -3), (dict(rows=1 << 31), -2)])
def test_linear_i8_refuses_bad_params(lib, bad, want):
    p = lin(**bad)
    assert lib.hstu_linear_i8_workspace_size(ctypes.byref(p)) == 0
    assert lib.hstu_linear_i8(ctypes.byref(p), A, A, A, A, A, A, BIG, None) == want


def test_linear_i8_refuses_bad_pointers(lib):
    p = ctypes.byref(lin())
    assert lib.hstu_linear_i8(None, A, A, A, A, A, A, BIG, None) == -1
    for i in (0, 1, 2, 4, 5):
        args = [A] * 6
        args[i] = None
        assert lib.hstu_linear_i8(p, *args, BIG, None) == -1
    for i in range(6):
        args = [A] * 6
        args[i] = ODD
        assert lib.hstu_linear_i8(p, *args, BIG, None) == -3
    assert lib.hstu_linear_i8(p, *[A] * 6, 256, None) == -5
    assert lib.hstu_linear_i8(ctypes.byref(lin(rows=0)), *[None] * 6, 0, None) == 0


def test_quant_weight_refusals(lib):
    f = lib.hstu_quant_i8_weight
    assert f(None, 512, 512, 1, A, A, None) == -1 and f(A, 512, 512, 3, A, A, None) == -1
    assert f(A, 0, 512, 1, A, A, None) == -1
    assert f(A, 500, 512, 1, A, A, None) == -3 and f(ODD, 512, 512, 1, A, A, None) == -3
    assert f(A, 131088, 512, 1, A, A, None) == -2


def kvp(**kw):
    base = dict(batch=3, num_heads=4, head_dim=128, page_size=32, num_pages=100, max_pages_per_user=8, kv_stride=0,
                total_new=50, dtype=_lib.DT_BF16)
    base.update(kw)
    return _lib.KvParams(**base)


def test_kv_q4_refusals(lib):
    ok = ctypes.byref(kvp())
    assert lib.hstu_kv_q4_workspace_size(ok) >= 256 + 3 * 8
    for bad, want in ((dict(batch=0), -1), (dict(page_size=0), -1), (dict(dtype=5), -1), (dict(head_dim=48), -2),
                      (dict(head_dim=288), -2), (dict(total_new=-1), -1)):
        p = ctypes.byref(kvp(**bad))
        assert lib.hstu_kv_q4_workspace_size(p) == 0
        assert lib.hstu_kv_append_q4(p, *[A] * 13, BIG, None) == want
        assert lib.hstu_kv_read_q4(p, *[A] * 11, BIG, None) == want
    assert lib.hstu_kv_append_q4(ctypes.byref(kvp(kv_stride=100)), *[A] * 13, BIG, None) == -1
    for i in [0, 1, 2, 4, 5, 6, 7, 8, 9, 10, 11, 12]:      # 3 is num_append, which may be NULL
        args = [A] * 13
        args[i] = None
        assert lib.hstu_kv_append_q4(ok, *args, BIG, None) == -1
    for i in (0, 1, 4, 5, 6, 7, 12):
        args = [A] * 13
        args[i] = ODD
        assert lib.hstu_kv_append_q4(ok, *args, BIG, None) == -3
    assert lib.hstu_kv_append_q4(ok, *[A] * 13, 100, None) == -5
    for i in range(11):
        args = [A] * 11
        args[i] = None
        assert lib.hstu_kv_read_q4(ok, *args, BIG, None) == -1
    for i in (0, 1, 2, 3, 8, 9, 10):
        args = [A] * 11
        args[i] = ODD
        assert lib.hstu_kv_read_q4(ok, *args, BIG, None) == -3
    assert lib.hstu_kv_read_q4(ok, *[A] * 11, 100, None) == -5


def attn(**kw):
    base = dict(batch=2, num_heads=4, head_dim=128, n_max=1024, total_tokens=300, max_seq_len=200, dtype=torch.bfloat16)
    base.update(kw)
    return hstu.attn_params(**base)


def call_attn(lib, p, args=None, num_pages=10, max_pages=8, page_size=32, splits=1, ws=BIG):
    a = [A] * 16 if args is None else args
    return lib.hstu_attn_fwd_paged_q4(ctypes.byref(p), *a, num_pages, A, max_pages, page_size, A, splits, A, A, ws, None)


def test_attn_q4_refusals(lib):
    for i in (0, 1, 2, 3, 4, 5, 6, 8, 9, 12, 13, 14, 15):  # 7: num_candidates, 10 and 11: gamma and beta
        args = [A] * 16
        args[i] = None
        assert call_attn(lib, attn(), args) == -1, i
    for i in (0, 1, 2, 3, 10, 11, 12, 13, 14, 15):
        args = [A] * 16
        args[i] = ODD
        assert call_attn(lib, attn(), args) == -3, i
    assert call_attn(lib, attn(head_dim=48)) == -2
    assert call_attn(lib, attn(num_heads=9)) == -2
    assert call_attn(lib, attn(), page_size=0) == -1 and call_attn(lib, attn(), num_pages=0) == -1
    assert call_attn(lib, attn(), max_pages=0) == -1
    assert call_attn(lib, attn(), splits=0) == -1 and call_attn(lib, attn(), splits=65) == -1
    assert call_attn(lib, attn(), ws=64) == -5
    assert call_attn(lib, attn(flags=0x1000)) == -1
    for stage in (_lib.F_STAGE_PLAN, _lib.F_STAGE_ATTN, _lib.F_STAGE_EPILOGUE):
        assert call_attn(lib, attn(flags=stage)) == -2
    p = attn(head_dim=48)
    assert lib.hstu_attn_paged_q4_workspace_size(ctypes.byref(p), 1) == 0
    assert hstu.hstu_attn_paged_q4_workspace_size(batch=2, num_heads=4, head_dim=128, n_max=1024, total_tokens=300,
                                                  dtype=torch.bfloat16) > 256


def test_bindings_refuse_cpu_tensors():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        hstu.hstu_linear_i8(x, torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8))
    with pytest.raises(ValueError, match="CUDA"):
        hstu.hstu_quant_i8_weight(x)
    pool = torch.zeros(4, 1, 8, 16, dtype=torch.uint8)
    meta = torch.zeros(4, 1, 8, 2, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        hstu.hstu_kv_read_q4(pool, pool, meta, meta, i.view(1, 1), i, i, i, total_tokens=1)
    k = torch.zeros(4, 1, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        hstu.hstu_kv_append_q4(k, k, i, pool, pool, meta, meta, i.view(1, 1), i, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        hstu.hstu_attn_fwd_paged_q4(k, k, k, k.view(4, 32), i, i.long(), i, torch.zeros(7), torch.zeros(128), pool, pool,
                                    meta, meta, i.view(1, 1), i, n_max=4)


def test_the_bf16_cache_has_no_4bit_parameters():
    pool = torch.zeros(4, 1, 8, 16, dtype=torch.uint8)
    with pytest.raises(KeyError):
        hstu.api.kv_params(pool, torch.zeros(2, 2, dtype=torch.int32))
