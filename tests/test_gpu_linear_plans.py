"""Products whose columns are two launches, in both types: exact in whole
numbers, and the same bits as the columns in calls of their own. (A host test
checks that the sizes do take two.)"""
import pytest
import torch

import exact_replay_decode_amd as erd
from gpu_cases import same_bits
from step_cases import DEV, DT, gen, randn

pytestmark = pytest.mark.gpu

TWICE = {1: [(129, 33000, 264), (65, 33000, 1000), (700, 6001, 520), (400, 33000, 264),
             (2049, 4100, 520), (1025, 8200, 520), (2049, 1000, 4104)],
         0: [(65, 33000, 1000), (129, 10300, 4104), (1025, 6001, 1000), (400, 8200, 2056),
             (4097, 2000, 2056), (1025, 33000, 520), (4097, 6001, 1000)]}
CASES = [("bf16" if b else "f32", *size) for b in TWICE for size in TWICE[b]]


@pytest.mark.parametrize("io,M,N,K", CASES)
def test_two_launches(io, M, N, K):
    g = gen(M + N + K)
    x = torch.randint(-4, 5, (M, K), generator=g, device=DEV).to(DT[io])
    w = torch.randint(-4, 5, (N, K), generator=g, device=DEV).to(DT[io])
    y = erd.ssd_linear(x, w, out_dtype=torch.float32)
    assert torch.equal(y.double(), x.double() @ w.double().t())
    x, w = randn(g, M, K, dtype=DT[io]), randn(g, N, K, dtype=DT[io], scale=K ** -0.5)
    b, r = randn(g, N), randn(g, M, N, dtype=DT[io])
    whole = erd.ssd_linear(x, w, b, "silu", r)
    for lo, hi in ((0, 500), (N // 2, N // 2 + 70), (N - 333, N)):
        part = erd.ssd_linear(x, w[lo:hi].contiguous(), b[lo:hi].contiguous(), "silu",
                              r[:, lo:hi].contiguous())
        assert same_bits(part, whole[:, lo:hi].contiguous()), (lo, hi)
