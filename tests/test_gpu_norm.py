"""ssd_gated_norm on the GPU against fp64.

Tolerance, from the arithmetic (fp32 inside): the sum of squares has at most
86 additions on any element's way (32 in a thread, 6 in the wave's tree, 16
waves, the rounded squares included), all terms positive, so it is off by at
most 86 * 2**-24 = 5.2e-6 relative and its root by half; the gate is off by
(|z| + 8) 2**-24 relative (exp2 of a rounded product, reciprocal, product), in
the value and, once more at most, in the sum; division, reciprocal root and
the products add at most 8 * 2**-24. With |z| <= 8 that is below 6e-6 of the
value, plus half a step of the output type."""
import pytest
import torch

import exact_replay_decode_amd as erd
from gpu_cases import same_bits
from step_cases import DEV, DT, check_close, gen, randn

pytestmark = pytest.mark.gpu


def norm64(y, w, z, groups, eps, before):
    T = y.shape[0]
    y, w = y.cpu().double().reshape(T, -1), w.cpu().double()
    gate = 1.0
    if z is not None:
        z = z.cpu().double().reshape(T, -1)
        gate = z * torch.special.expit(z)
    v = y if before else y * gate
    ms = v.reshape(T, groups, -1).square().mean(2, keepdim=True)
    v = (v.reshape(T, groups, -1) / (ms + eps).sqrt()).reshape(T, -1) * w
    return v * gate if before else v


# group sizes 16 (one head) .. 32768: one wave, several, 16 waves, not whole waves
@pytest.mark.parametrize("H,P,groups", [(1, 16, 1), (5, 16, 5), (24, 64, 1), (8, 64, 8), (8, 64, 1),
                                        (12, 128, 2), (48, 64, 1), (64, 64, 8), (128, 64, 1),
                                        (65, 128, 1), (128, 128, 1), (130, 128, 1),
                                        (256, 128, 1)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_norm_matches_fp64(H, P, groups, io):
    sh = erd.Shape(H, groups, P, 16, 64, io, io)
    g = gen(H * P)
    for T in (1, 7):
        y = randn(g, T, H, P, dtype=DT[io], scale=3.0)
        z = randn(g, T, H, P, dtype=DT[io]).clamp(-8, 8)
        w = randn(g, H * P) + 1.0
        for zz in (z, None):
            for before in (False, True):
                out = erd.ssd_gated_norm(sh, y, w, z=zz, eps=1e-5, norm_before_gate=before)
                ref = norm64(y, w, zz, groups, 1e-5, before)
                check_close(out.reshape(T, -1), ref, 6e-6 * ref.abs(), (T, before, zz is None))


def test_rows_do_not_depend_on_the_call():
    g = gen(1)
    for H, G in ((32, 1), (64, 8), (130, 1)):
        sh = erd.Shape(H, G, 64, 16, 64)
        y, z = (randn(g, 500, H, 64, dtype=torch.bfloat16) for _ in range(2))
        w = randn(g, H * 64)
        whole = erd.ssd_gated_norm(sh, y, w, z=z)
        for a, n in ((0, 1), (3, 2), (17, 64), (100, 399)):
            assert same_bits(erd.ssd_gated_norm(sh, y[a:a + n], w, z=z[a:a + n]),
                             whole[a:a + n])
        # in place over y, and over z
        y2, z2 = y.clone(), z.clone()
        erd.ssd_gated_norm(sh, y2, w, z=z, out=y2)
        erd.ssd_gated_norm(sh, y, w, z=z2, out=z2)
        assert same_bits(y2, whole) and same_bits(z2, whole)


def test_zero_rows_and_bad_values():
    sh = erd.Shape(4, 2, 16, 16, 64, "f32", "f32")
    y = torch.zeros(4, 4, 16, device=DEV)
    w = torch.ones(64, device=DEV)
    y[1] = 1e-20                   # squares underflow: eps alone
    y[2, 0, 0] = float("nan")      # group 0 of row 2
    y[3] = 1.0
    out = erd.ssd_gated_norm(sh, y, w, eps=1e-5)
    assert bool((out[0] == 0).all())
    assert torch.allclose(out[1], y[1] / 1e-5 ** 0.5, rtol=1e-6, atol=0)
    assert bool(out[2, :2].isnan().all()) and bool((out[2, 2:] == 0).all())
    assert torch.allclose(out[3], torch.full_like(out[3], (1 + 1e-5) ** -0.5), rtol=1e-6)
    # a shut gate
    z = torch.full((4, 4, 16), -1e4, device=DEV)
    assert bool((erd.ssd_gated_norm(sh, y[3:], w, z=z[3:], eps=1e-5) == 0).all())


def test_refusals_and_empty():
    sh = erd.Shape(4, 2, 16, 16, 64)
    y, w = torch.zeros(3, 4, 16, dtype=torch.bfloat16, device=DEV), torch.ones(64, device=DEV)
    assert erd.ssd_gated_norm(sh, y[:0], w).shape == (0, 4, 16)
    with pytest.raises(erd.SsdError, match="SHAPE"):
        erd.ssd_gated_norm(sh, y, w, groups=3)
    with pytest.raises(ValueError, match="shape"):
        erd.ssd_gated_norm(sh, y, w[:32])
    with pytest.raises(ValueError, match="dtype"):
        erd.ssd_gated_norm(sh, y, w, z=y.float())


def test_rows_past_32_bits():
    """More than 2**31 elements in each array."""
    sh = erd.Shape(64, 8, 64, 16, 64)
    T, g = 530000, gen(6)
    y = torch.empty(T, 64, 64, dtype=torch.bfloat16, device=DEV)
    for a in range(0, T, 53000):
        y[a:a + 53000] = randn(g, 53000, 64, 64)
    z, w = y.flip(0), randn(g, 4096)
    whole = erd.ssd_gated_norm(sh, y, w, z=z)
    for a in (0, T // 2, T - 2):
        assert same_bits(erd.ssd_gated_norm(sh, y[a:a + 2], w, z=z[a:a + 2]), whole[a:a + 2])
