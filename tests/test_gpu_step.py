"""A model step around the scan, as a serving program runs it: in-projection,
conv, scan or replay decode on a paged cache, gated norm, out-projection onto
the residual stream, the head's logits and the tokens' log probabilities, with
pages reserved and trimmed around every step.

The prompt in one call, the prompt in pieces and token-by-token decode give
the same bits all the way to the log probabilities (vLLM RFC "Mamba2:
exact-replay decode so that prefill, chunked prefill and decode produce
identical bits"), eagerly and from a captured graph."""
import numpy as np
import pytest
import torch

import exact_replay_decode_amd as erd
from exact_replay_decode_amd import synth
from gpu_cases import same_bits
from step_cases import DEV, DT, gen, randn

pytestmark = pytest.mark.gpu


class Model:
    """Two mixer layers and a head, random weights."""

    def __init__(self, H=8, G=2, P=64, N=128, Q=64, d=256, V=5003, io="bf16", layers=2, seed=0):
        self.shape = erd.Shape(H, G, P, N, Q, io, "f32")
        self.d, self.V, self.io = d, V, DT[io]
        g = gen(seed)
        cd = erd.conv_dim(self.shape)
        n = H * P + cd + H
        self.layers = []
        for li in range(layers):
            hp = synth.make_head_params(H, seed + li)
            self.layers.append(dict(
                w_in=randn(g, n, d, dtype=self.io, scale=d ** -0.5),
                w_out=randn(g, d, H * P, dtype=self.io, scale=(H * P) ** -0.5),
                conv_w=randn(g, cd, 4, scale=0.5), conv_b=randn(g, cd, scale=0.1),
                norm=randn(g, H * P, scale=0.1) + 1.0,
                prm=tuple(torch.from_numpy(v).to(DEV) for v in (hp.A, hp.D, hp.dt_bias))))
        self.head = randn(g, V, d, dtype=self.io, scale=d ** -0.5)
        self.emb = randn(g, V, d, dtype=self.io)

    def caches(self, slots, pt=16):
        Q = self.shape.chunk_size
        out = []
        for _ in self.layers:
            c = erd.ReplayCache(self.shape, slots, DEV, page_tokens=pt,
                                num_pages=slots * (Q // pt))
            c.buf_x.normal_()
            out.append((c, torch.zeros(slots, erd.conv_dim(self.shape), 3, dtype=self.io,
                                       device=DEV)))
        return out

    def logits(self, h, y, z, L):
        T = h.shape[0]
        v = erd.ssd_gated_norm(self.shape, y, L["norm"], z=z)
        return erd.ssd_linear(v.view(T, -1), L["w_out"], residual=h)

    def prefill(self, ids, cu, state, slots):
        h = self.emb[ids]
        for L, (c, conv) in zip(self.layers, state):
            n = torch.from_numpy(np.diff(cu).astype(np.int32)).to(DEV)
            assert bool(erd.ssd_replay_pages_reserve(self.shape, c, n, slot_idx=slots).all())
            z, xBC, dt = erd.ssd_in_proj(self.shape, h, L["w_in"])
            x, B, C = erd.ssd_conv1d_varlen(self.shape, cu, xBC, L["conv_w"], L["conv_b"],
                                            conv_state=conv, slot_idx=slots)
            A, D, bias = L["prm"]
            y = erd.ssd_replay_prefill(self.shape, c, cu, x, dt, B, C, A, D, bias, slot_idx=slots)
            erd.ssd_replay_pages_trim(self.shape, c, slot_idx=slots)
            h = self.logits(h, y, z, L)
        return erd.ssd_linear(h, self.head, out_dtype=torch.float32)

    def decode(self, ids, state, slots):
        h = self.emb[ids]
        for L, (c, conv) in zip(self.layers, state):
            erd.ssd_replay_pages_reserve(self.shape, c, 1, slot_idx=slots)
            z, xBC, dt = erd.ssd_in_proj(self.shape, h, L["w_in"])
            A, D, bias = L["prm"]
            y, _ = erd.ssd_replay_decode_conv(self.shape, c, xBC, L["conv_w"], conv, dt, A, D, bias,
                                              bias=L["conv_b"], slot_idx=slots)
            erd.ssd_replay_pages_trim(self.shape, c, slot_idx=slots)
            h = self.logits(h, y, z, L)
        return erd.ssd_linear(h, self.head, out_dtype=torch.float32)


def same_scores(a, b):
    return all(same_bits(p.contiguous(), q.contiguous()) for p, q in zip(a, b))


@pytest.mark.parametrize("io,kw", [("bf16", {}), ("f32", dict(H=4, G=1, P=16, N=16, Q=32, d=64,
                                                              V=777))])
def test_prompt_pieces_and_decode_score_alike(io, kw):
    m = Model(io=io, **kw)
    g = gen(1)
    lengths = [150, 97, 201]
    cu = synth.cu_seqlens(lengths)
    T = int(cu[-1])
    ids = torch.randint(0, m.V, (T,), generator=g, device=DEV)
    nxt = torch.randint(0, m.V, (T,), generator=g, device=DEV, dtype=torch.int32)
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV)
    whole = m.prefill(ids, cu, m.caches(3), slots)
    score = erd.ssd_token_logprobs(whole, nxt, top_k=5)

    # each sequence alone, in pieces that cross the chunk end
    for s in range(3):
        st, a = m.caches(4), int(cu[s])
        sl = torch.tensor([3], dtype=torch.int32, device=DEV)
        for n in (1, 40, lengths[s] - 41):
            part = m.prefill(ids[a:a + n], synth.cu_seqlens([n]), st, sl)
            assert same_bits(part, whole[a:a + n])
            a += n

    # a short prompt, then all three token by token, until the shortest ends
    st, pre = m.caches(3), 20
    at = torch.tensor([int(c) for c in cu[:-1]], device=DEV)
    ip = torch.cat([torch.arange(int(c), int(c) + pre) for c in cu[:-1]]).to(DEV)
    assert same_bits(m.prefill(ids[ip], synth.cu_seqlens([pre] * 3), st, slots), whole[ip])
    for t in range(pre, min(lengths)):
        it = at + t
        y = m.decode(ids[it], st, slots)
        assert same_bits(y, whole[it]), t
        r = erd.ssd_token_logprobs(y, nxt[it], top_k=5)
        assert same_scores(r, [v[it] for v in score])


def test_captured_steps_equal_eager_ones():
    """One decode step of the whole model with its page traffic and scoring,
    captured once and replayed 70 times (past a chunk end), with the eager run
    and synchronizations between the replays."""
    m = Model()
    g = gen(2)
    S, steps = 3, 70
    ids = torch.randint(0, m.V, (S, 30 + steps + 1), generator=g, device=DEV)
    slots = torch.arange(S, dtype=torch.int32, device=DEV)
    eager, graph = m.caches(S), m.caches(S)
    for st in (eager, graph):
        m.prefill(ids[:, :30].reshape(-1), synth.cu_seqlens([30] * S), st, slots)
    stream = torch.cuda.Stream()
    tok_in = ids[:, 30].clone()
    nxt = ids[:, 31].to(torch.int32).contiguous()
    saved = [(c.clone(), v.clone()) for c, v in graph]
    stream.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=stream):
        out = erd.ssd_token_logprobs(m.decode(tok_in, graph, slots), nxt, top_k=3)
    torch.cuda.synchronize()
    for (c, v), (c0, v0) in zip(graph, saved):
        c.copy_from(c0)
        v.copy_(v0)
    for t in range(30, 30 + steps):
        want = erd.ssd_token_logprobs(m.decode(ids[:, t].contiguous(), eager, slots),
                                      ids[:, t + 1].to(torch.int32).contiguous(), top_k=3)
        tok_in.copy_(ids[:, t])
        nxt.copy_(ids[:, t + 1])
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert same_scores(out, want), t
    for (c, v), (ce, ve) in zip(graph, eager):
        assert same_bits(c.state, ce.state) and same_bits(c.buf_pages, ce.buf_pages)
        assert same_bits(v, ve)


def test_forked_samples_score_their_own_tokens():
    """Best of four: a prompt prefilled once and forked, each sample decodes its
    own tokens and scores what a prefill of the whole sample scores; then the
    losers end and the pool is compacted, and the winner goes on."""
    m = Model(seed=3)
    g = gen(3)
    pre, steps, S = 75, 30, 5
    prompt = torch.randint(0, m.V, (pre,), generator=g, device=DEV)
    tails = torch.randint(0, m.V, (4, steps + 12), generator=g, device=DEV)
    st = m.caches(S)
    first = torch.tensor([0], dtype=torch.int32, device=DEV)
    m.prefill(prompt, synth.cu_seqlens([pre]), st, first)
    src = torch.zeros(4, dtype=torch.int32, device=DEV)
    dst = torch.arange(1, 5, dtype=torch.int32, device=DEV)
    for c, conv in st:
        assert bool(erd.ssd_replay_pages_reserve(m.shape, c, 0, slot_idx=dst, like_idx=src).all())
        erd.ssd_replay_cache_copy(m.shape, c, c, dst, src)
        conv[1:] = conv[0]
        erd.ssd_replay_cache_free(m.shape, c, slot_idx=first)
    got = [m.decode(tails[:, t].contiguous(), st, dst) for t in range(steps)]
    lose, win = dst[[0, 1, 3]].contiguous(), dst[2:3].contiguous()
    for c, _ in st:
        erd.ssd_replay_cache_free(m.shape, c, slot_idx=lose)
        used = erd.ssd_replay_pages_compact(m.shape, c)
        assert int(used) == int((c.buf_pages >= 0).sum()) and int(c.buf_pages.max()) < int(used)
    more = [m.decode(tails[2:3, t].contiguous(), st, win) for t in range(steps, steps + 12)]
    for i in range(4):
        n = steps + (12 if i == 2 else 0)
        whole = m.prefill(torch.cat([prompt, tails[i, :n]]), synth.cu_seqlens([pre + n]),
                          m.caches(1), first)
        for t in range(steps):
            assert same_bits(got[t][i], whole[pre + t]), (i, t)
        if i == 2:
            for t in range(12):
                assert same_bits(more[t][0], whole[pre + steps + t]), t
