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
