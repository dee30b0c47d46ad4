"""Edges of the layer operators on the GPU: values that are not finite, gates close to 1,
and widths and paths that only some sizes reach."""
import numpy as np
import pytest
import torch

import linear_attention_lm_b200 as lab
from linear_attention_lm_b200 import build as lab_build

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lab_build.build()
    lab.load_library()
    torch.cuda.set_device(0)


def normal(seed, shape, dtype="f32", scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(DT[dtype])


def spread_lengths(B, L):
    """Lengths of a padded batch, none of them a whole number of tiles but the first."""
    return torch.tensor([L] + [(L * (2 * b + 1) // (2 * B)) | 1 for b in range(1, B)], device="cuda")


# one thread per two channels (the first three), tiles with one and several rounds, odd
# widths, several CTAs per sequence
REC_SHAPES = [(4, 14, 64), (5, 9, 33), (128, 40, 256), (4, 130, 256), (3, 700, 33), (2, 3000, 24),
              (8, 1500, 1024)]


@pytest.mark.parametrize("B,L,D", REC_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_gatedrec_gradient_padding_is_zero_beside_a_bad_final_gradient(B, L, D, dtype, bad):
    """dx and dg are zero past a sequence's length also where dh_last is not finite, and
    the other channels have the bits that they have without it."""
    x, g, dy = (normal(i, (B, L, D), dtype) for i in range(3))
    dh, n = normal(4, (B, D)), spread_lengths(B, L)
    _, chunks = lab.gatedrec(x, g, None, n, for_grad=True)
    want = lab.gatedrec_grad(x, g, dy, chunks, dh, n)
    dh2 = dh.clone()
    dh2[:, 1::7] = bad
    dx, dg, dh0 = lab.gatedrec_grad(x, g, dy, chunks, dh2, n)
    past = torch.arange(L, device="cuda")[None, :] >= n[:, None]
    assert not dx[past].any() and not dg[past].any()
    clean = torch.ones(D, dtype=torch.bool, device="cuda")
    clean[1::7] = False
    for a, b in zip((dx, dg, dh0), want):
        assert torch.equal(a[..., clean], b[..., clean])
    assert lab.based_get_device_error() == 0
