"""Permute, finalize and finalize's gradients over more tokens than one grid dimension takes work-items for."""

import pytest
import torch

from gpu_util import dev
from mixture_experts_ffn_02_amd import moe_lora as ml

pytestmark = pytest.mark.gpu

H = 8


def whole(shape, seed):
    """Small whole numbers in bf16."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    return torch.randint(-4, 5, shape, generator=g, device=dev(), dtype=torch.int8).to(torch.bfloat16)


@pytest.mark.parametrize("codes", [False, True], ids=["bf16", "codes"])
def test_gradients_of_finalize(codes):
    """A workgroup of 256 for each of 2^24 tokens: 2^32 work-items."""
    T = 2 ** 24 + 5
    d = ml.dims(T, H, 8, 4, 1)
    d_out, y = whole((T, H), 5), whole((T, H), 6)
    w = torch.full((T, 1), 0.5, device=dev())
    e2p = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=dev())
    src = dict(y_perm=y)
    if codes:  # (exact for these values)
        c, e = torch.empty((T, H), dtype=torch.uint8, device=dev()), torch.empty((T, 1), dtype=torch.uint8, device=dev())
        ml.moe_lora_checkpoint_pack(y, c, e)
        src = dict(y_codes=c, y_exps=e)
    d_y, d_w = torch.full_like(y, float("nan")), torch.full_like(w, float("nan"))
    ml.moe_lora_finalize_backward(d, d_out, w, e2p, d_y, d_w, **src)
    assert torch.equal(d_y, d_out.flip(0) * 0.5)
    assert torch.equal(d_w[:, 0], (d_out.float() * y.flip(0).float()).sum(1))


def test_finalize():
    T = 2 ** 24 + 5
    y, w = whole((T, H), 7), torch.full((T, 1), 0.5, device=dev())
    e2p = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=dev())
    out = torch.full_like(y, float("nan"))
    ml.moe_lora_finalize(ml.dims(T, H, 8, 4, 1), y, w, e2p, out)
    assert torch.equal(out, y.flip(0) * 0.5)


def test_permute():
    """A wavefront to each row: 2^32 work-items from 2^26 rows."""
    R = 2 ** 26 + 5
    x = whole((R, H), 8)
    p2e = torch.arange(R - 1, -1, -1, dtype=torch.int32, device=dev())
    out = torch.full_like(x, float("nan"))
    ml.moe_lora_permute(ml.dims(R, H, 8, 4, 1), x, p2e, out)
    assert torch.equal(out, x.flip(0))
