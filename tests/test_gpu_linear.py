"""ssd_linear and ssd_in_proj on the GPU: against fp64 within the bounds that
step_cases.linear64 derives, exactly where the sums are whole numbers, and bit
for bit across row counts, kernels and streams."""
import pytest
import torch

import exact_replay_decode_amd as erd
from gpu_cases import same_bits
from step_cases import DEV, DT, check_close, gen, linear64, randn

pytestmark = pytest.mark.gpu

# rows x columns x K: one of each, below / at / past the 16-wide tiles, K below, at and past
# the K steps (32 in bf16) and the K blocks, odd columns
SIZES = [(1, 1, 8), (1, 16, 32), (2, 17, 40), (5, 3, 1000), (16, 64, 64), (17, 33, 24),
         (31, 130, 72), (64, 257, 1000), (65, 63, 136), (100, 128, 2056), (130, 100, 264),
         (257, 300, 512), (300, 520, 96)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_linear_whole_numbers_are_exact(M, N, K, io):
    """Entries in -4..4: every product and partial sum is a whole number below
    2**24, exact in fp32, so nothing may be lost or counted twice."""
    g = gen(M * 7 + N + K)
    x = torch.randint(-4, 5, (M, K), generator=g, device=DEV).to(DT[io])
    w = torch.randint(-4, 5, (N, K), generator=g, device=DEV).to(DT[io])
    y = erd.ssd_linear(x, w, out_dtype=torch.float32)
    assert torch.equal(y.cpu().double(), x.cpu().double() @ w.cpu().double().t())


# Sizes of every tile, alone and as the first or the second of two launches over the
# columns, most with a partial last tile of k.
TILES = [(1, 17, 1000), (1, 4100, 40), (1, 4100, 136), (33, 4100, 40), (33, 4100, 136),
         (33, 4100, 520), (1, 16001, 40), (1, 16001, 4104), (65, 8200, 40), (65, 8200, 2056),
         (65, 16001, 136), (200, 8200, 520), (257, 10300, 40), (513, 10300, 264),
         (1025, 6001, 40), (2049, 6001, 264), (33, 33000, 520), (33, 33000, 1000),
         (65, 4100, 4104), (200, 8200, 1000), (65, 33000, 520), (129, 33000, 264),
         (400, 33000, 264), (700, 16001, 520), (2049, 4100, 520), (2049, 10300, 520),
         (4097, 1000, 520), (200, 33000, 40), (700, 8200, 40), (4097, 2000, 40),
         (513, 33000, 136), (4097, 17, 40), (33, 8200, 264), (129, 8200, 40), (100, 8200, 40),
         (65, 8200, 4104), (100, 8200, 2056), (129, 10300, 1000), (300, 10300, 520),
         (33, 33000, 264), (65, 33000, 136), (700, 8200, 136), (1025, 6001, 136),
         (200, 10300, 1000), (513, 8200, 264), (4097, 2000, 136), (2049, 8200, 40),
         (33, 33000, 40), (65, 33000, 40), (300, 33000, 40), (400, 33000, 72), (2049, 4100, 136),
         (2049, 4100, 1000), (513, 16001, 520), (2049, 10300, 264), (4097, 6001, 520),
         (4097, 1000, 136), (2049, 1000, 520), (400, 10300, 136), (4097, 4100, 40),
         (4097, 1000, 40), (4097, 10300, 40), (33, 16001, 264), (1, 16001, 520),
         (257, 16001, 136), (200, 8200, 264),
         (129, 33000, 40), (129, 33000, 520), (700, 33000, 40), (4097, 2000, 72), (4097, 6001, 40),
         (513, 16001, 1000), (513, 33000, 520), (1025, 10300, 520), (257, 16001, 520),
         (33, 8200, 520), (400, 33000, 136)]


@pytest.mark.parametrize("M,N,K", TILES)
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_every_tile_is_exact_in_whole_numbers(M, N, K, io):
    g = gen(M + N + K)
    x = torch.randint(-4, 5, (M, K), generator=g, device=DEV).to(DT[io])
    w = torch.randint(-4, 5, (N, K), generator=g, device=DEV).to(DT[io])
    y = erd.ssd_linear(x, w, out_dtype=torch.float32)
    assert torch.equal(y.double(), x.double() @ w.double().t())


@pytest.mark.parametrize("M,N,K", [(200, 8200, 1000), (2049, 4100, 520), (400, 33000, 264)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_columns_of_two_launches(M, N, K, io):
    """Bias, activation and residual where the columns are two launches: the
    bits of the same columns in calls of their own."""
    g = gen(N)
    x, w = randn(g, M, K, dtype=DT[io]), randn(g, N, K, dtype=DT[io], scale=K ** -0.5)
    b, r = randn(g, N), randn(g, M, N, dtype=DT[io])
    whole = erd.ssd_linear(x, w, b, "gelu", r)
    for lo, hi in ((0, 500), (N // 2, N // 2 + 70), (N - 333, N)):
        part = erd.ssd_linear(x, w[lo:hi].contiguous(), b[lo:hi].contiguous(), "gelu",
                              r[:, lo:hi].contiguous())
        assert same_bits(part, whole[:, lo:hi].contiguous()), (lo, hi)


@pytest.mark.parametrize("io,K", [("bf16", 1000), ("f32", 520)])
def test_in_proj_in_two_launches(io, K):
    sh = erd.Shape(64, 1, 64, 128, 64, io, "f32")
    g, M, a, cd = gen(K), 200, 64 * 64, 64 * 64 + 256
    x, w = randn(g, M, K, dtype=DT[io]), randn(g, a + cd + 64, K, dtype=DT[io])
    z, xBC, d = erd.ssd_in_proj(sh, x, w)
    for part, lo, hi in ((z.view(M, a), 0, a), (xBC, a, a + cd), (d, a + cd, a + cd + 64)):
        one = erd.ssd_linear(x, w[lo:hi].contiguous(), out_dtype=part.dtype)
        assert same_bits(part, one)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu2"])
def test_linear_epilogue(M, N, K, io, act):
    g = gen(M + N * 3 + K)
    x, w = randn(g, M, K, dtype=DT[io]), randn(g, N, K, dtype=DT[io], scale=K ** -0.5)
    for bias, res, out in ((None, None, io), (randn(g, N), None, "f32"),
                           (None, randn(g, M, N, dtype=DT[io]), "f32"),
                           (randn(g, N), randn(g, M, N, dtype=DT[io]), io),
                           (randn(g, N), randn(g, M, N, dtype=DT[io]), "bf16")):
        y = erd.ssd_linear(x, w, bias, act, res, out_dtype=DT[out])
        assert y.dtype == DT[out]
        check_close(y, *linear64(x, w, bias, act, res), (io, act, out))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(130, 264), (1024, 2048), (4000, 768), (520, 4096), (33, 1000)])
def test_rows_do_not_depend_on_the_call(io, N, K):
    """Any slice of the rows, alone or at another place, gives the same bits."""
    g = gen(N + K)
    M = 1100
    x, w = randn(g, M, K, dtype=DT[io]), randn(g, N, K, dtype=DT[io], scale=K ** -0.5)
    b, r = randn(g, N), randn(g, M, N, dtype=DT[io])
    whole = erd.ssd_linear(x, w, b, "silu", r)
    for a, n in ((0, 1), (0, 2), (3, 5), (7, 16), (1, 17), (100, 33), (5, 64), (9, 65), (64, 128),
                 (33, 129), (200, 256), (11, 300), (3, 513), (1, 700), (76, 1024)):
        part = erd.ssd_linear(x[a:a + n].contiguous(), w, b, "silu", r[a:a + n].contiguous())
        assert same_bits(part, whole[a:a + n]), (a, n)
    # as do the columns
    for a, n in ((0, 1), (5, 16), (16, 17)):
        part = erd.ssd_linear(x, w[a:a + n].contiguous(), b[a:a + n].contiguous(), "silu",
                              r[:, a:a + n].contiguous())
        assert same_bits(part, whole[:, a:a + n].contiguous()), (a, n)


def test_large_tiles_match_small_ones():
    """A product large enough for every kernel, against the same rows in small
    calls and, for some of them, fp64."""
    g = gen(5)
    M, N, K = 4096 + 37, 2304 + 16, 1032
    for io in ("bf16", "f32"):
        x, w = randn(g, M, K, dtype=DT[io]), randn(g, N, K, dtype=DT[io], scale=K ** -0.5)
        whole = erd.ssd_linear(x, w, out_dtype=torch.float32)
        for a in (0, 255, 1000, 2048, M - 16):
            assert same_bits(erd.ssd_linear(x[a:a + 16].contiguous(), w,
                                            out_dtype=torch.float32), whole[a:a + 16])
        rows = torch.tensor([0, 31, 127, 128, 255, 256, 2047, M - 1], device=DEV)
        check_close(whole[rows], *linear64(x[rows], w))


@pytest.mark.parametrize("H,G,P,N,dt", [(24, 1, 64, 128, "f32"), (8, 4, 32, 64, "bf16"),
                                        (5, 1, 16, 16, "f32"), (3, 3, 64, 32, "bf16")])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 19, 300])
def test_in_proj_splits_the_columns(H, G, P, N, dt, io, M):
    sh = erd.Shape(H, G, P, N, 64, io, dt)
    g, K = gen(H + M), 200
    a, cd = H * P, erd.conv_dim(sh)
    x, w, b = randn(g, M, K, dtype=DT[io]), randn(g, a + cd + H, K, dtype=DT[io]), randn(
        g, a + cd + H)
    z, xBC, d = erd.ssd_in_proj(sh, x, w, b)
    assert z.shape == (M, H, P) and xBC.shape == (M, cd) and d.shape == (M, H)
    for part, lo, hi in ((z.view(M, a), 0, a), (xBC, a, a + cd), (d, a + cd, a + cd + H)):
        one = erd.ssd_linear(x, w[lo:hi].contiguous(), b[lo:hi].contiguous(),
                             out_dtype=part.dtype)
        assert same_bits(part, one)
        check_close(part, *linear64(x, w[lo:hi], b[lo:hi]))


def test_a_bad_row_or_column_stays_its_own():
    """NaN and infinities spread along their own row or column alone; K past
    the end is no part of the sum."""
    g = gen(3)
    for io in ("bf16", "f32"):
        for M, N in ((40, 48), (300, 272)):
            x, w = randn(g, M, 72, dtype=DT[io]), randn(g, N, 72, dtype=DT[io])
            good = erd.ssd_linear(x, w)
            x[7, 70], x[M - 1, 0], w[5, 71] = float("nan"), float("inf"), float("inf")
            bad = erd.ssd_linear(x, w)
            rows = torch.ones(M, dtype=torch.bool, device=DEV)
            rows[7] = rows[M - 1] = False
            cols = torch.ones(N, dtype=torch.bool, device=DEV)
            cols[5] = False
            assert same_bits(bad[rows][:, cols], good[rows][:, cols])
            assert bool(bad[7].isnan().all()) and not bool(bad[M - 1].isfinite().any())
            assert not bool(bad[:, 5].isfinite().any())


def test_activations_at_the_ends():
    """Values that saturate: silu and gelu go to 0 and to v, relu2 keeps NaN."""
    v = torch.tensor([-1e30, -200.0, -90.0, 0.0, 90.0, 1e18, float("inf"), float("nan")],
                     device=DEV)
    x = torch.zeros(8, 4, device=DEV)
    x[:, 0] = v
    w = torch.zeros(1, 4, device=DEV)
    w[0, 0] = 1.0
    for act, want in (("silu", [0, 0, 0, 0, 90, 1e18, float("inf")]),
                      ("gelu", [0, 0, 0, 0, 90, 1e18, float("inf")]),
                      ("relu2", [0, 0, 0, 0, 8100, 1e36, float("inf")])):
        y = erd.ssd_linear(x, w, activation=act)[:, 0].cpu()
        for got, ref in zip(y[:7].tolist(), want):
            assert got == pytest.approx(ref, rel=1e-6, abs=1e-30)
        assert bool(y[7].isnan())


def test_in_place_residual_and_given_outputs():
    g = gen(9)
    for io in ("bf16", "f32"):
        for M in (3, 200):
            x, w = randn(g, M, 64, dtype=DT[io]), randn(g, 96, 64, dtype=DT[io])
            r = randn(g, M, 96, dtype=DT[io])
            want = erd.ssd_linear(x, w, residual=r)
            assert erd.ssd_linear(x, w, residual=r, out=r) is r
            assert same_bits(r, want)
    x, w = randn(g, 2, 64, dtype=torch.bfloat16), randn(g, 8, 64, dtype=torch.bfloat16)
    r = torch.zeros(2, 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="dtype"):
        erd.ssd_linear(x, w, residual=r.float())
    with pytest.raises(ValueError, match="contiguous"):
        erd.ssd_linear(x, w.t().contiguous().t())
    with pytest.raises(ValueError, match="activation"):
        erd.ssd_linear(x, w, activation="tanh")
    with pytest.raises(erd.SsdError, match="UNSUPPORTED"):
        erd.ssd_linear(x[:, :12].contiguous(), w[:, :12].contiguous())
    # a misaligned view is refused for x and w, fine for the others
    odd = torch.zeros(17, dtype=torch.bfloat16, device=DEV)[1:].view(2, 8)
    assert same_bits(erd.ssd_linear(x, w, residual=odd, out=odd), erd.ssd_linear(x, w))
    with pytest.raises(erd.SsdError, match="ALIGN"):
        erd.ssd_linear(torch.zeros(129, dtype=torch.bfloat16, device=DEV)[1:].view(2, 64), w)
    assert erd.ssd_linear(x[:0], w).shape == (0, 8)
    assert erd.ssd_linear(x, w[:0]).shape == (2, 0)


def test_outputs_past_32_bits():
    """More than 2**31 outputs: the last rows land where they belong."""
    g = gen(2)
    M, N = 70001, 32768
    x, w = randn(g, M, 8, dtype=torch.bfloat16), randn(g, N, 8, dtype=torch.bfloat16)
    y = erd.ssd_linear(x, w)
    for a in (0, 65530, M - 5):
        assert same_bits(y[a:a + 5], erd.ssd_linear(x[a:a + 5].contiguous(), w))


def test_other_stream():
    g = gen(4)
    x, w = randn(g, 300, 512, dtype=torch.bfloat16), randn(g, 640, 512, dtype=torch.bfloat16)
    want = erd.ssd_linear(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = erd.ssd_linear(x, w, stream=s)
    s.synchronize()
    assert same_bits(y, want)


@pytest.mark.parametrize("M,N,K", [(140000, 24, 16384), (70000, 65544, 8)])
def test_rows_past_32_bits(M, N, K):
    """x of more than 2**31 elements, and an output of more than 2**32."""
    g = gen(K)
    x = torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
    for a in range(0, M, 20000):
        x[a:a + 20000] = randn(g, *x[a:a + 20000].shape)
    w = randn(g, N, K, dtype=torch.bfloat16)
    y = erd.ssd_linear(x, w, activation="relu2")
    for a in (0, M // 2, M - 3):
        assert same_bits(y[a:a + 3], erd.ssd_linear(x[a:a + 3], w, activation="relu2"))


@pytest.mark.parametrize("M,N", [(2 ** 29 - 3, 8), (8, 2 ** 29 - 8)])
def test_the_most_rows_and_columns(M, N):
    """One dimension at the limit of a launch: rows (columns) far apart, the
    last ones among them, against a call of their own."""
    g = gen(N % 97)
    x = torch.zeros(M, 8, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(N, 8, dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, 1, 12345678, 2 ** 28 + 77, 2 ** 29 - 9], device=DEV)
    few, many = (w, x) if M > N else (x, w)
    few.copy_(randn(g, 8, 8))
    many[at] = randn(g, 5, 8, dtype=torch.bfloat16)
    y = erd.ssd_linear(x, w)
    part = erd.ssd_linear(x[at], w) if M > N else erd.ssd_linear(x, w[at])
    assert same_bits(y[at] if M > N else y[:, at].contiguous(), part)
    assert int((y.view(-1).view(torch.int32) != 0).sum()) <= 5 * 8
