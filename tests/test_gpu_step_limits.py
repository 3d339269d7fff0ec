"""The step operators at the ends of their documented ranges that other tests
do not reach: the longest k of a product, the most channels of a norm."""
import pytest
import torch

import exact_replay_decode_amd as erd
from gpu_cases import same_bits
from step_cases import DEV, DT, gen, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N", [(1, 17), (130, 300), (600, 520)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_the_longest_k(M, N, io):
    """Entries in -4..4: partial sums are whole numbers of at most 16 * 2**20 =
    2**24, exact in any order."""
    K = 2 ** 20
    g = gen(M)
    x = torch.randint(-4, 5, (M, K), generator=g, device=DEV, dtype=torch.int8).to(DT[io])
    w = torch.randint(-4, 5, (N, K), generator=g, device=DEV, dtype=torch.int8).to(DT[io])
    y = erd.ssd_linear(x, w, out_dtype=torch.float32)
    assert torch.equal(y.double(), x.double() @ w.double().t())


@pytest.mark.parametrize("H", [1, 33])
def test_the_most_channels_of_a_norm(H):
    """2**34 channels: a group of 16 in two lanes, and one of 528, whose two waves
    are the most threads a channel."""
    sh = erd.Shape(H, 1, 16, 16, 64)
    T = 2 ** 34 // (16 * H)
    w = randn(gen(H), 16 * H) + 1
    y = torch.zeros(T, H, 16, dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, 1, T // 3, T // 2 + 1, T - 2, T - 1], device=DEV)
    few = randn(gen(1), 6, H, 16, dtype=torch.bfloat16)
    y[at] = few
    out = erd.ssd_gated_norm(sh, y, w, groups=1)
    del y
    assert same_bits(out[at], erd.ssd_gated_norm(sh, few, w, groups=1))
    near = torch.cat([at[:-1] + 2, at[-2:] - 2])
    near = near[~torch.isin(near, at) & (near < T)]
    assert not bool(out[near].any())
