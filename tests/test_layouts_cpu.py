"""CPU checks of the tensor layouts that the entry points refuse before anything is launched: rows that overlap.  A row
stride of 0 means packed rows to the library, so a broadcast would be read or written past its end."""
import pytest
import torch

import generative_recommender_attention_jagged_b200 as hstu

BF = torch.bfloat16
H, D, T = 2, 32, 4


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on a GPU, for the checks that come before anything is launched."""

    is_cuda = True


def on_gpu(t):
    return t.as_subclass(OnGpu)


def ints(*v):
    return on_gpu(torch.tensor(v, dtype=torch.int32))


def tokens(broadcast):
    """q, k, v, u of which one is a broadcast over the tokens."""
    args = {x: on_gpu(torch.zeros(T, H, D, dtype=BF)) for x in "qkv"}
    args["u"] = on_gpu(torch.zeros(T, H * D, dtype=BF))
    args[broadcast] = on_gpu(args[broadcast][:1].expand(args[broadcast].shape))
    return list(args.values())


TS = on_gpu(torch.zeros(T, dtype=torch.int64))
RAB = (on_gpu(torch.zeros(31)), on_gpu(torch.zeros(128)))


def pools():
    return on_gpu(torch.zeros(4, H, 8, D, dtype=BF)), on_gpu(torch.zeros(4, H, 8, D, dtype=BF))


CALLS = {
    "hstu_attn_fwd": lambda q, k, v, u: hstu.hstu_attn_fwd(q, k, v, u, ints(0, T), TS, *RAB, n_max=16),
    "hstu_attn_fwd_static_ws": lambda q, k, v, u: hstu.api.hstu_attn_fwd_static_ws(
        q, k, v, u, ints(0, T), TS, *RAB, n_max=16),
    "hstu_attn_fwd_paged": lambda q, k, v, u: hstu.hstu_attn_fwd_paged(
        q, k, v, u, ints(0, T), TS, ints(0, T), *RAB, *pools(), ints(0, 1).view(1, 2), ints(0), n_max=16),
    "hstu_mfalcon_fwd": lambda q, k, v, u: hstu.hstu_mfalcon_fwd(
        q, k, v, u, ints(0, T), TS[:0], ints(0, 0), TS, *RAB, *pools(), ints(0, 1).view(1, 2), ints(0), n_max=16,
        microbatch=4, max_candidates=4),
    "hstu_attn_bwd": lambda q, k, v, u: hstu.hstu_attn_bwd(
        q, k, v, ints(0, T), TS, *RAB, on_gpu(torch.zeros(T, H, D)), n_max=16),
}


@pytest.mark.parametrize("which", ["q", "k", "v", "u"])
@pytest.mark.parametrize("call", CALLS)
def test_attention_refuses_broadcast_tokens(call, which):
    if call == "hstu_attn_bwd" and which == "u":
        pytest.skip("takes no u")
    with pytest.raises(ValueError, match=f"^{which}.*: rows of 64 elements may not overlap"):
        CALLS[call](*tokens(which))


@pytest.mark.parametrize("stride", [0, 16])
@pytest.mark.parametrize("call", [hstu.hstu_linear, hstu.hstu_layer_f1, hstu.hstu_layer_f2])
def test_linear_refuses_rows_that_overlap(call, stride):
    w = on_gpu(torch.zeros(32, 8, dtype=BF))
    with pytest.raises(ValueError, match="x: rows of 32 elements may not overlap"):
        call(on_gpu(torch.zeros(80, dtype=BF).as_strided((T, 32), (stride, 1))), w)
    with pytest.raises(ValueError, match="out: rows of 8 elements may not overlap"):
        call(on_gpu(torch.zeros(T, 32, dtype=BF)), w, out=on_gpu(torch.zeros(80, dtype=BF).as_strided((T, 8), (0, 1))))


def test_append_refuses_broadcast_tokens():
    k = on_gpu(torch.zeros(1, H, D, dtype=BF).expand(T, H, D))
    with pytest.raises(ValueError, match="k_new: rows of 64 elements may not overlap"):
        hstu.hstu_kv_append(k, k, ints(0, T), *pools(), ints(0, 1).view(1, 2), ints(0), ints(0, 1, 2, 3), ints(4))
