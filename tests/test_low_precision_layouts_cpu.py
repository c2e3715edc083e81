"""CPU checks of the tensor layouts that the low-precision entry points take and refuse before anything is launched."""
import pytest
import torch

import generative_recommender_attention_jagged_b200 as hstu


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on a GPU, for the checks that come before anything is launched."""

    def get_device(self):
        return 0


def on_gpu(t):
    return t.as_subclass(OnGpu)


BF = torch.bfloat16


def ints(*v):
    return on_gpu(torch.tensor(v, dtype=torch.int32))


def pools(H=2, d=32):
    byte, meta = on_gpu(torch.zeros(4, H, 8, d // 2, dtype=torch.uint8)), on_gpu(torch.zeros(4, H, 8, 2, dtype=BF))
    return byte, byte.clone(), meta, meta.clone()


@pytest.mark.parametrize("stride", [0, 16])
def test_linear_i8_refuses_rows_that_overlap(stride):
    """A row stride of 0 means packed rows to the library: a broadcast x would be read, a broadcast out written, past its
    end."""
    w_q, w_scale = on_gpu(torch.zeros(8, 32, dtype=torch.int8)), on_gpu(torch.ones(8))
    x = on_gpu(torch.zeros(80, dtype=BF).as_strided((4, 32), (stride, 1)))
    with pytest.raises(ValueError, match="x: rows of 32 elements may not overlap"):
        hstu.hstu_linear_i8(x, w_q, w_scale)
    out = on_gpu(torch.zeros(1, 8, dtype=BF).expand(4, 8))
    with pytest.raises(ValueError, match="out: rows of 8 elements may not overlap"):
        hstu.hstu_linear_i8(on_gpu(torch.zeros(4, 32, dtype=BF)), w_q, w_scale, out=out)


def test_append_q4_refuses_broadcast_tokens():
    k = on_gpu(torch.zeros(1, 2, 32, dtype=BF).expand(4, 2, 32))
    with pytest.raises(ValueError, match="k_new: rows of 64 elements may not overlap"):
        hstu.hstu_kv_append_q4(k, k, ints(0, 4), *pools(), ints(0, 1).view(1, 2), ints(0), ints(0, 1, 2, 3), ints(4))


@pytest.mark.parametrize("which", ["q", "k", "v", "u"])
def test_attn_q4_refuses_broadcast_tokens(which):
    args = {x: on_gpu(torch.zeros(4, 2, 32, dtype=BF)) for x in "qkv"}
    args["u"] = on_gpu(torch.zeros(4, 64, dtype=BF))
    args[which] = on_gpu(args[which][:1].expand(args[which].shape))
    with pytest.raises(ValueError, match=f"{which}: rows of 64 elements may not overlap"):
        hstu.hstu_attn_fwd_paged_q4(*args.values(), ints(0, 4), on_gpu(torch.zeros(4, dtype=torch.int64)), ints(0, 4),
                                    on_gpu(torch.zeros(31)), on_gpu(torch.zeros(128)), *pools(),
                                    ints(0, 1).view(1, 2), ints(0), n_max=16)


def test_one_row_may_have_any_row_stride():
    one = torch.zeros(1, 32, dtype=BF).expand(1, 32)
    assert hstu.api._row_stride("x", one.as_strided((1, 32), (0, 1)), 32) == 32
    assert hstu.api._row_stride("x", torch.zeros(3, 48)[:, :32], 32) == 48
