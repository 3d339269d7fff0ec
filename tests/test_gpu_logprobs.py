"""ssd_token_logprobs on the GPU against fp64.

Tolerances, from the arithmetic (fp32): on its way an element passes at most
n = 32 ceil(chunks / 16) additions in its lane, 6 in the wave's tree and 16
between streams, each 2**-24 relative to a sum of positive terms, and exp2 of
a rounded product, (1.5 |x - m| + 4) 2**-24 of its term, the mean of |x - m|
under p being below ln V + 1. So log s is off by (n + 22 + 1.5 (ln V + 1) + 4 +
2 |log s|) 2**-24 and a log probability by that and two roundings of values
up to |lp|, 2**-23 |lp|; u / s by (n + 30) 2**-24 (ln V + 1) more."""
import math

import pytest
import torch

import exact_replay_decode_amd as erd
from gpu_cases import same_bits
from step_cases import DEV, DT, gen, randn

pytestmark = pytest.mark.gpu
INF = float("inf")


def plain(x, tok, k):
    """fp64 on the host; order by value descending, then index ascending."""
    x = x.cpu().double()
    tok = tok.cpu().long()
    T, V = x.shape
    m = x.max(1, keepdim=True).values
    none = (m == -INF)
    e = torch.exp(torch.where(none, 0.0, x - torch.where(none, 0.0, m)))
    e = torch.where(none, 0.0, e)
    z = e.sum(1, keepdim=True)
    lz = torch.where(none, 0.0, torch.log(torch.where(none, 1.0, z)))
    lp = torch.where(none, -INF, x - torch.where(none, 0.0, m) - lz)
    p = lp.exp()
    ent = -torch.where(p > 0, p * lp, 0.0).sum(1)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    place = torch.empty_like(order)
    place.scatter_(1, order, torch.arange(V).expand(T, V).contiguous())
    at = tok.clamp(0, V - 1)[:, None]
    ok = (tok >= 0) & (tok < V)
    logprob = torch.where(ok, lp.gather(1, at)[:, 0], float("nan"))
    rank = torch.where(ok, place.gather(1, at)[:, 0], -1)
    return logprob, ent, rank, order[:, :k], lp.gather(1, order[:, :k])


def check(x, tok, k):
    V = x.shape[1]
    r = erd.ssd_token_logprobs(x, tok, top_k=k)
    lp, ent, rank, ids, tlp = plain(x, tok, k)
    n = 32 * math.ceil(math.ceil(V / 2048) / 16)
    u = 2.0 ** -24
    base = (n + 22 + 1.5 * (math.log(V) + 1) + 4 + 2 * (math.log(V) + 1)) * u

    def close(a, b, tol):
        a, b = a.cpu().double(), b
        assert torch.equal(a.isnan(), b.isnan())
        inf = b.isinf()
        assert torch.equal(a[inf], b[inf])
        f = ~inf & ~b.isnan()
        d = (a[f] - b[f]).abs()
        lim = tol + 2 * u * b[f].abs()
        assert bool((d <= lim).all()), float((d / lim).max())

    close(r.logprob, lp, base)
    close(r.entropy, ent, base + (n + 30) * u * (math.log(V) + 1))
    assert torch.equal(r.rank.cpu().long(), rank)
    if k:
        assert torch.equal(r.top_ids.cpu().long(), ids)
        close(r.top_logprobs, tlp, base)
    else:
        assert r.top_ids is None and r.top_logprobs is None
    return r


@pytest.mark.parametrize("V", [1, 2, 7, 8, 63, 500, 2047, 2048, 2049, 5001, 32768, 50257, 70000])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_matches_fp64(V, io):
    g = gen(V)
    for T, k in ((3, 5), (300, 20), (5, 64), (2, 1), (4, 0)):
        T = min(T, max(1, 2 ** 22 // V))
        x = randn(g, T, V, dtype=DT[io], scale=3.0)
        tok = torch.randint(0, V, (T,), generator=g, device=DEV, dtype=torch.int32)
        check(x, tok, min(k, V))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [4, 300, 600])
def test_ties_masks_and_orders(io, T):
    """Equal values (index decides), rows in ascending and descending order,
    masks that leave few, one or no token, whole chunks masked."""
    V, k = 9001, 32
    g = gen(T)
    up = torch.arange(V, device=DEV, dtype=torch.float32)
    rows = [torch.full((V,), 1.5), torch.zeros(V), -0.0 * torch.ones(V),
            up / V * 8, -up / V * 8, torch.full((V,), -INF), (up % 2) - 3, (up % 5 == 0) * 4.0]
    few = torch.full((V,), -INF)
    few[[5, 77, 4500, 9000]] = torch.tensor([1.0, 3.0, 1.0, -2.0])
    one = torch.full((V,), -INF)
    one[8999] = -7.0
    half = torch.randn(V)
    half[:4096] = -INF
    low = torch.full((V,), torch.finfo(DT[io]).min)     # the type's lowest value is no mask
    low[3] = 0.0
    signs = torch.where(up.cpu() % 3 == 0, 0.0, -0.0)   # +0 and -0 are equal
    rows += [few, one, half, low, signs]
    x = torch.stack([r.to(DEV) for r in rows]).to(DT[io])
    x = x[torch.arange(T, device=DEV) % len(rows)].contiguous()
    for seed in range(3):
        tok = torch.randint(0, V, (T,), generator=g, device=DEV, dtype=torch.int32)
        tok[:min(T, 13)] = torch.tensor([0, 9000, 77, 5, 8999, 4500, 4096, 4095, 1, 3, 2, 8192,
                                         4], device=DEV, dtype=torch.int32)[:min(T, 13)].roll(seed)
        check(x, tok, k)
    check(x[:, :40].contiguous(), tok % 40, 40)


def test_a_wave_list_that_overflows():
    """Many equal best values in every chunk, best values last, and top_k at
    its limit: the lists are cut many times."""
    V, k = 40000, 64
    g = gen(8)
    x = randn(g, 6, V)
    x[0, :30000] = 5.0
    x[1] = torch.arange(V, device=DEV) // 700
    x[2, 2048:4096] = 9.0
    x[3] = torch.arange(V, 0, -1, device=DEV) // 900
    x[4, ::3] = 4.0
    tok = torch.tensor([29999, 39999, 3000, 899, 6, 0], dtype=torch.int32, device=DEV)
    for io in ("bf16", "f32"):
        for T in (6, 600):
            check(x.to(DT[io])[torch.arange(T, device=DEV) % 6].contiguous(),
                  tok[torch.arange(T, device=DEV) % 6].contiguous(), k)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_rows_that_are_no_distribution(io):
    g = gen(2)
    x = randn(g, 6, 5000, dtype=DT[io])
    x[0, 17] = float("nan")
    x[1, 4999] = INF
    x[2] = float("nan")
    x[3] = -INF
    x[3, 9] = float("nan")
    x[4, 100:200] = INF
    tok = torch.tensor([17, 3, 4, 9, 150, 7], dtype=torch.int32, device=DEV)
    for T in (6, 600):
        xx = x[torch.arange(T, device=DEV) % 6].contiguous()
        tt = tok[torch.arange(T, device=DEV) % 6].contiguous()
        r = erd.ssd_token_logprobs(xx, tt, top_k=7)
        bad = torch.arange(T, device=DEV) % 6 < 5
        for v in (r.logprob, r.entropy, r.top_logprobs):
            assert bool(v[bad].isnan().all()) and bool(v[~bad].isfinite().all())
        assert bool((r.rank[bad] == -1).all()) and bool((r.top_ids[bad] == -1).all())
    check(x[5:], tok[5:], 7)


def test_tokens_out_of_range():
    g = gen(3)
    x = randn(g, 4, 100)
    tok = torch.tensor([-1, 100, 2 ** 31 - 1, 50], dtype=torch.int32, device=DEV)
    check(x, tok, 5)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("V", [777, 50257, 131073])
def test_rows_do_not_depend_on_the_call(io, V):
    g = gen(V)
    x = randn(g, 700, V, dtype=DT[io], scale=2.0)
    tok = torch.randint(0, V, (700,), generator=g, device=DEV, dtype=torch.int32)
    whole = erd.ssd_token_logprobs(x, tok, top_k=6)
    for a, n in ((0, 1), (1, 3), (40, 256), (3, 257), (99, 600)):
        part = erd.ssd_token_logprobs(x[a:a + n], tok[a:a + n], top_k=6)
        for p, w in zip(part, whole):
            assert same_bits(p.contiguous(), w[a:a + n].contiguous())
    # the alternatives do not change the sums
    none = erd.ssd_token_logprobs(x, tok)
    assert same_bits(none.logprob, whole.logprob) and same_bits(none.entropy, whole.entropy)
    assert same_bits(none.rank, whole.rank)


def test_logits_past_32_bits():
    """More than 2**31 logits, rows that start at odd addresses."""
    g = gen(1)
    T, V = 43000, 50257
    x = torch.empty(T, V, dtype=torch.bfloat16, device=DEV)
    x[:] = randn(g, 1, V, dtype=torch.bfloat16)
    last = randn(g, 3, V, dtype=torch.bfloat16)
    x[-3:] = last
    tok = torch.full((T,), 50256, dtype=torch.int32, device=DEV)
    r = erd.ssd_token_logprobs(x, tok, top_k=4)
    p = erd.ssd_token_logprobs(last, tok[:3], top_k=4)
    for a, b in zip(r, p):
        assert same_bits(a[-3:].contiguous(), b)
    check(last, tok[:3], 4)


def test_refusals_and_empty():
    x = torch.zeros(3, 10, device=DEV)
    tok = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert erd.ssd_token_logprobs(x[:0], tok[:0]).logprob.shape == (0,)
    with pytest.raises(erd.SsdError, match="SHAPE"):
        erd.ssd_token_logprobs(x, tok, top_k=11)
    with pytest.raises(ValueError, match="dtype"):
        erd.ssd_token_logprobs(x, tok.long())
    with pytest.raises(ValueError, match="not bfloat16 or float32"):
        erd.ssd_token_logprobs(x.half(), tok)
    with pytest.raises(ValueError, match="contiguous"):
        erd.ssd_token_logprobs(torch.zeros(10, 3, device=DEV).t(), tok)


def test_the_most_rows():
    """As many rows as a launch takes."""
    T, V = 16777208, 3
    g = gen(11)
    x = randn(g, T, V, dtype=torch.bfloat16)
    tok = torch.randint(0, V, (T,), generator=g, device=DEV, dtype=torch.int32)
    r = erd.ssd_token_logprobs(x, tok, top_k=2)
    for a in (0, T // 2 + 1, T - 700):
        part = erd.ssd_token_logprobs(x[a:a + 700], tok[a:a + 700], top_k=2)
        for p, w in zip(part, r):
            assert same_bits(p, w[a:a + 700])
    want = torch.log_softmax(x[-700:].double(), 1).gather(1, tok[-700:, None].long())[:, 0]
    # (two chunks' worth of roundings bound three terms: 16 * 2**-24 and 2**-23 |lp|)
    assert bool(((r.logprob[-700:].double() - want).abs()
                 <= 16 * 2.0 ** -24 + 2.0 ** -23 * want.abs()).all())
    with pytest.raises(erd.SsdError, match="UNSUPPORTED"):
        erd.ssd_token_logprobs(torch.zeros(T + 1, 1, device=DEV),
                               torch.zeros(T + 1, dtype=torch.int32, device=DEV))
