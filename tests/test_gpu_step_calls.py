"""How the operators around the scan are called, on the GPU: captured into
graphs, on two streams at once, on a stream of the caller's, and with outputs
of the caller's."""
import pytest
import torch

import exact_replay_decode_amd as erd
from gpu_cases import same_bits
from step_cases import DEV, gen, randn

pytestmark = pytest.mark.gpu


class Calls:
    """One call of every operator that computes rows, over buffers of its own.
    fill() gives the buffers new inputs, run() returns the results."""

    def __init__(self, io="bf16", rows=37):
        self.sh = erd.Shape(8, 2, 32, 64, 64, io, "f32")
        t = self.sh.io
        self.cols = 2 * 8 * 32 + 2 * 2 * 64 + 8
        g = gen(rows)
        self.w = randn(g, self.cols, 200, dtype=t, scale=0.07)
        self.w2 = randn(g, 144, 256, dtype=t, scale=0.06)
        self.head = randn(g, 5003, 144, dtype=t, scale=0.1)
        self.nw = randn(g, 256) + 1
        self.u = torch.zeros(rows, 200, dtype=t, device=DEV)
        self.tok = torch.zeros(rows, dtype=torch.int32, device=DEV)

    def fill(self, seed):
        g = gen(seed)
        self.u.copy_(randn(g, *self.u.shape))
        self.tok.copy_(torch.randint(0, 5003, self.tok.shape, generator=g, device=DEV))
        return self

    def run(self, stream=None):
        z, xBC, dt = erd.ssd_in_proj(self.sh, self.u, self.w, stream=stream)
        y = xBC[:, :256].contiguous().view(z.shape) if stream is None else z
        h = erd.ssd_gated_norm(self.sh, y, self.nw, z=z, stream=stream)
        o = erd.ssd_linear(h.view(-1, 256), self.w2, activation="silu", stream=stream)
        logits = erd.ssd_linear(o, self.head, out_dtype=torch.float32, stream=stream)
        return (z, xBC, dt, h, o, logits,
                *erd.ssd_token_logprobs(logits, self.tok, top_k=5, stream=stream))


def same(a, b):
    return all(same_bits(x, y) for x, y in zip(a, b, strict=True))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 37, 300])
def test_captured_calls_equal_eager_ones(io, rows):
    graph, eager = Calls(io, rows), Calls(io, rows)
    graph.fill(0)
    graph.run()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = graph.run()
    for seed in range(5):
        want = eager.fill(seed).run()
        graph.fill(seed)
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert same(out, want), seed


def test_two_graphs_and_an_eager_run_side_by_side():
    """Two captured graphs replayed on two streams while an eager run works on
    the current one: nothing is shared between calls."""
    a, b, c = (Calls("bf16", r) for r in (64, 300, 5))
    want = [x.fill(i).run() for i, x in enumerate((a, b, c))]
    torch.cuda.synchronize()
    graphs = []
    for x in (a, b):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = x.run()
        graphs.append((gr, out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for gr, _, s in graphs:
            with torch.cuda.stream(s):
                gr.replay()
        got = c.run()
        torch.cuda.synchronize()
        assert same(got, want[2])
        for (_, out, _), w in zip(graphs, want):
            assert same(out, w)


def test_calls_on_a_stream_given():
    """Outputs are allocated for and written on the stream of the call."""
    a = Calls("bf16", 100).fill(1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for seed in (1, 2):
        a.fill(seed)
        s.wait_stream(torch.cuda.current_stream())
        got = a.run(stream=s)
        s.synchronize()
        with torch.cuda.stream(s):
            y = a.run(stream=s)
        s.synchronize()
        assert same(got, y)


def _cache(seed, S=6, pt=16, pool=40):
    sh = erd.Shape(4, 2, 32, 32, 64, "bf16", "f32")
    c = erd.ReplayCache(sh, S, DEV, page_tokens=pt, num_pages=pool)
    g = gen(seed)
    for b in (c.state, c.state_bf, c.buf_x, c.buf_dt, c.buf_B):
        b.copy_(randn(g, *b.shape))
    c.buf_len.copy_(torch.tensor([0, 1, 17, 33, 63, 48], dtype=torch.int32)[:S])
    c.boundary_pos.copy_(torch.arange(S) * 64)
    # pages scattered over the pool; slot 0 holds two that it does not need
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((S, 4), -1, dtype=torch.int32)
    for s, n in enumerate((2, 1, 2, 3, 4, 3)[:S]):
        for i in range(n):
            table[s, i] = order.pop()
    c.buf_pages.copy_(table)
    return sh, c


def _arrays(c):
    return (c.state, c.state_bf, c.buf_x, c.buf_dt, c.buf_B, c.buf_len, c.boundary_pos,
            c.buf_pages)


def _round(sh, c, lists, granted, used, copied, work):
    """Every page and slot call on one cache."""
    ends, forks, like = lists
    erd.ssd_replay_cache_free(sh, c, slot_idx=ends)
    erd.ssd_replay_pages_reserve(sh, c, 1, slot_idx=forks, like_idx=like, granted=granted)
    erd.ssd_replay_cache_copy(sh, c, c, forks, like, copied=copied)
    erd.ssd_replay_pages_trim(sh, c)
    erd.ssd_replay_pages_compact(sh, c, used=used, workspace=work)


def test_captured_page_calls_equal_eager_ones():
    """Slots ended, forked, trimmed and compacted in one graph, replayed over
    different contents with eager work between."""
    i32 = dict(dtype=torch.int32, device=DEV)
    lists = (torch.tensor([0, 1], **i32), torch.tensor([1, 0], **i32),
             torch.tensor([4, 2], **i32))
    (sh, g), (_, e) = _cache(0), _cache(0)
    outs = [[torch.zeros(n, **i32) for n in (2, 1, 2, 42)] for _ in range(2)]
    _round(sh, _cache(9)[1], lists, *outs[0])   # (loads the kernels)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        _round(sh, g, lists, *outs[0])
    for seed in range(6):
        src = _cache(seed)[1]
        for c in (g, e):
            for to, frm in zip(_arrays(c), _arrays(src)):
                to.copy_(frm)
        _round(sh, e, lists, *outs[1])
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert bool(outs[1][0].all()) and bool(outs[1][2].all())
        assert all(same_bits(x, y) for x, y in zip(outs[0][:3], outs[1][:3]))
        assert all(same_bits(x, y) for x, y in zip(_arrays(g), _arrays(e))), seed


def test_two_caches_on_two_streams():
    """Rounds over two caches at the same time, against the same one by one."""
    i32 = dict(dtype=torch.int32, device=DEV)
    lists = (torch.tensor([0, 1], **i32), torch.tensor([1, 0], **i32),
             torch.tensor([4, 2], **i32))
    both = [_cache(s) for s in (1, 2)]
    alone = [_cache(s) for s in (1, 2)]
    outs = [[torch.zeros(n, **i32) for n in (2, 1, 2, 42)] for _ in range(4)]
    for (sh, c), o in zip(alone, outs):
        _round(sh, c, lists, *o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    for (sh, c), o, s in zip(both, outs[2:], streams):
        with torch.cuda.stream(s):
            _round(sh, c, lists, *o)
    torch.cuda.synchronize()
    for k in range(2):
        assert all(same_bits(x, y) for x, y in zip(outs[k][:3], outs[2 + k][:3]))
        assert all(same_bits(x, y) for x, y in zip(_arrays(alone[k][1]), _arrays(both[k][1])))


def test_one_table_for_the_caches_of_two_layers():
    """Reserve and trim through one of the caches serves both; copies of each
    find the pages."""
    (sh, a), (_, b) = _cache(3), _cache(4)
    b.buf_pages = a.buf_pages
    i32 = dict(dtype=torch.int32, device=DEV)
    dst, src = torch.tensor([0, 1], **i32), torch.tensor([4, 4], **i32)
    assert bool(erd.ssd_replay_pages_reserve(sh, a, 0, slot_idx=dst, like_idx=src).all())
    for c in (a, b):
        ok = torch.zeros(2, **i32)
        erd.ssd_replay_cache_copy(sh, c, c, dst, src, copied=ok)
        assert bool(ok.all())
    erd.ssd_replay_pages_trim(sh, b)
    held = a.buf_pages[a.buf_pages >= 0]
    assert held.unique().numel() == held.numel() == 4 + 4 + 2 + 3 + 4 + 3
    for c in (a, b):
        rows = c.buf_x.view(-1, *c.buf_x.shape[-2:])
        for k in (0, 1):
            for row in (0, 15, 16, 47, 48, 62):
                p, q = (int(c.buf_pages[s, row // 16]) * 16 + row % 16 for s in (k, 4))
                assert p != q and same_bits(rows[p], rows[q])


def test_pages_that_two_slots_share():
    """A page that two table entries name is used once, is not handed out, and
    both entries follow it when the pool is compacted."""
    sh, c = _cache(6)
    c.buf_pages[2, :2] = c.buf_pages[4, :2]        # slot 2 reads slot 4's first pages
    rows = c.buf_x.view(-1, *c.buf_x.shape[-2:])
    pages = c.buf_pages.cpu()
    held = {int(p) for p in pages.flatten() if p >= 0}
    want = [rows[int(p) * 16:int(p) * 16 + 16].clone() if p >= 0 else None
            for p in pages.flatten()]
    used = erd.ssd_replay_pages_compact(sh, c)
    assert int(used) == len(held) and int(c.buf_pages.max()) == len(held) - 1
    assert same_bits(c.buf_pages[2, :2], c.buf_pages[4, :2])
    for p, w in zip(c.buf_pages.cpu().flatten().tolist(), want):
        assert (p < 0) == (w is None)
        if w is not None:
            assert same_bits(rows[p * 16:p * 16 + 16], w)
    free = 40 - len(held)
    i32 = dict(dtype=torch.int32, device=DEV)
    got = erd.ssd_replay_pages_reserve(sh, c, 64, slot_idx=torch.tensor([0, 1, 3], **i32))
    lack = [4 - 2, 4 - 1, 4 - 3]
    assert sum(lack) <= free and bool(got.all())
    new = sorted(set(c.buf_pages.flatten().tolist()) - {-1})
    assert new == list(range(len(held) + sum(lack)))


def test_lists_with_skipped_and_empty_entries():
    """An empty list does nothing; entries out of range are skipped in every
    call, and the rest is served."""
    i32 = dict(dtype=torch.int32, device=DEV)
    sh, c = _cache(5)
    before = [t.clone() for t in _arrays(c)]
    none = torch.empty(0, **i32)
    assert erd.ssd_replay_pages_reserve(sh, c, 1, slot_idx=none).shape == (0,)
    erd.ssd_replay_pages_trim(sh, c, slot_idx=none)
    erd.ssd_replay_cache_free(sh, c, slot_idx=none)
    erd.ssd_replay_cache_copy(sh, c, c, none, none)
    out = torch.tensor([-1, 6, 2 ** 31 - 1, -2 ** 31], **i32)
    ok = torch.ones(4, **i32)
    assert not bool(erd.ssd_replay_pages_reserve(sh, c, 64, slot_idx=out).any())
    assert not bool(erd.ssd_replay_pages_reserve(sh, c, 64, slot_idx=torch.arange(4, **i32),
                                                 like_idx=out).any())
    erd.ssd_replay_pages_trim(sh, c, slot_idx=out)
    erd.ssd_replay_cache_free(sh, c, slot_idx=out)
    erd.ssd_replay_cache_copy(sh, c, c, out, torch.arange(4, **i32), copied=ok)
    assert not bool(ok.any())
    erd.ssd_replay_cache_copy(sh, c, c, torch.arange(4, **i32), out, copied=ok)
    assert not bool(ok.any())
    assert all(same_bits(x, y) for x, y in zip(_arrays(c), before))


def test_the_longest_lists():
    """As many entries as a launch takes, all but a few out of range."""
    i32 = dict(dtype=torch.int32, device=DEV)
    n = 16777208
    (sh, c), (_, d) = _cache(7), _cache(7)
    at = torch.tensor([5, n // 2, n - 1], device=DEV)
    src, dst = torch.full((n,), -1, **i32), torch.full((n,), 9, **i32)
    src[at], dst[at] = torch.tensor([2, 3, 5], **i32), torch.tensor([0, 1, 4], **i32)
    small = [t[at].contiguous() for t in (src, dst)]
    copied = torch.ones(n, **i32)
    for k, (s, t), got in ((c, (src, dst), copied), (d, small, None)):
        erd.ssd_replay_cache_free(sh, k, slot_idx=t)
        ok = erd.ssd_replay_pages_reserve(sh, k, 1, slot_idx=t, like_idx=s)
        assert int(ok.sum()) == 3
        erd.ssd_replay_cache_copy(sh, k, k, t, s, copied=got)
        erd.ssd_replay_pages_trim(sh, k, slot_idx=t)
    assert int(copied.sum()) == 3 and bool(copied[at].all())
    assert all(same_bits(x, y) for x, y in zip(_arrays(c), _arrays(d)))


def test_outputs_given():
    a = Calls("f32", 20).fill(3)
    z, xBC, dt, h, o, logits, *score = a.run()
    g = erd.ssd_in_proj(a.sh, a.u, a.w, out=tuple(torch.zeros_like(t) for t in (z, xBC, dt)))
    assert same(g, (z, xBC, dt))
    y = xBC[:, :256].contiguous().view(z.shape)
    assert same_bits(erd.ssd_gated_norm(a.sh, y, a.nw, z=z, out=torch.zeros_like(h)), h)
    assert same_bits(erd.ssd_linear(o, a.head, out=torch.zeros_like(logits)), logits)
    got = erd.ssd_token_logprobs(logits, a.tok, 5,
                                 out=erd.TokenLogprobs(*(torch.zeros_like(t) for t in score)))
    assert same(got, score)
    # only what is asked for is written
    some = erd.TokenLogprobs(torch.zeros(20, device=DEV), None, None, None, None)
    assert same_bits(erd.ssd_token_logprobs(logits, a.tok, out=some).logprob, score[0])
