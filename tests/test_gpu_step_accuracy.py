"""How far the operators around the scan are from 64 bits where fp32 results
are asked for, in units of the fp32 half step u = 2**-24 (relative)."""
import math

import pytest
import torch

import exact_replay_decode_amd as erd
from step_cases import DEV, DT, activate64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def relative(y, ref):
    return ((y.double() - ref).abs() / ref.abs()).nan_to_num(0.0)   # 0 / 0: equal


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("M", [300, 6000])
def test_silu_and_gelu_of_an_fp32_output(io, M):
    """The sum is one product by 1 and zeros, so exactly v. The sigmoid is
    within 7 u whatever v is (an ulp, 2 u, each from exp2 and the reciprocal,
    a half step each from the correction of the exponent, its product and
    1 + e), its product with v rounds once: 8 u, and less than u of second
    order. GELU's argument passes five roundings (0.044715 and 2 sqrt(2/pi) as
    stored among them, half a step each of their value) on its way, so e is off
    by 5 u |argument| more."""
    v = torch.linspace(-87.0, 20.0, M, device=DEV).to(DT[io])
    x = torch.zeros(M, 8, dtype=DT[io], device=DEV)
    x[:, 3] = v
    w = torch.zeros(3, 8, dtype=DT[io], device=DEV)
    w[:, 3] = 1.0
    v = v.double()
    y = erd.ssd_linear(x, w, activation="silu", out_dtype=torch.float32)
    assert float(relative(y[:, 1], activate64(v, "silu")).max()) <= 9 * U
    y = erd.ssd_linear(x, w, activation="gelu", out_dtype=torch.float32)
    arg = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    near = arg > -87.0
    bound = U * (9 + 5 * arg.clamp(max=0.0).abs())
    assert bool((relative(y[:, 1], activate64(v, "gelu")) <= bound)[near].all())


@pytest.mark.parametrize("H", [4, 32, 160])
def test_gate_of_an_fp32_norm(H):
    """Norm first, gate after, on rows of ones with weights of ones: r is the
    same for every element, 1 / sqrt(1 + eps) within 6 u (the sum of ones is
    exact, the division, eps, the sum and the reciprocal root, an ulp, round; half
    their error passes the root), the gate within 8 u (7 u and its product), two
    more products."""
    sh = erd.Shape(H, 1, 64, 128, 256, "f32", "f32")
    n = H * 64
    z = torch.linspace(-87.0, 20.0, 2 * n, device=DEV).view(2, H, 64)
    out = erd.ssd_gated_norm(sh, torch.ones_like(z), torch.ones(n, device=DEV), z=z, groups=1,
                             eps=1e-5, norm_before_gate=True)
    ref = activate64(z.double(), "silu") / math.sqrt(1 + 1e-5)
    assert float(relative(out, ref).max()) <= 17 * U


@pytest.mark.parametrize("M,N", [(5, 40), (64, 64), (300, 520), (1100, 700)])
def test_fp32_sums_are_chains_of_512(M, N):
    """Worst case: a chain of 512 loses at most 512 half steps of its partial
    sums, which sum |x w| bounds, and adding up the K / 512 chains one each. The
    terms 1 + 11 2**-15 lose all but the 1 in a single chain that has passed
    2**15: 11 of 65558, 1.7e-4, against the bound's 3.8e-5."""
    K = 65536
    x = torch.ones(M, K, device=DEV)
    w = torch.full((N, K), 1 + 11 * 2.0 ** -15, device=DEV)
    y = erd.ssd_linear(x, w)
    ref = K * (1 + 11 * 2.0 ** -15)
    assert float((y.double() - ref).abs().max()) <= (512 + K // 512 + 2) * U * ref


@pytest.mark.parametrize("M,N", [(64, 64), (300, 520), (1100, 700)])
@pytest.mark.parametrize("K", [512, 1000, 1024, 2056, 4096, 16384])
def test_fp32_error_does_not_grow_with_k(M, N, K):
    """Independent roundings, each of a root mean square of at most u / sqrt(3) of
    the partial sum, on partial sums of random signs, whose mean square is j of
    j terms: a chain of n has a mean square error of u^2 n^2 / 6, the chains of a
    sum of K add up to u^2 512 K / 6, the K / 512 additions of chains to
    u^2 (K / 512 + 1) K / 6, against the values' K. (One chain of 2056 would be
    at 8e-7, of 16384 at 2.3e-6; this bound stays below 5.8e-7.)"""
    g = torch.Generator(device=DEV)
    g.manual_seed(K + M)
    x, w = (torch.randn(n, K, generator=g, device=DEV) for n in (M, N))
    y = erd.ssd_linear(x, w)
    ref = x.double() @ w.double().t()
    err = float((y.double() - ref).square().mean().sqrt() / ref.square().mean().sqrt())
    assert err <= U * math.sqrt((min(K, 512) + K / 512 + 1) / 6)
