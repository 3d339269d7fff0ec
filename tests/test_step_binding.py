"""The binding's own checks (exact_replay_decode_amd/step.py) on the host: host
tensors stand in for the GPU's, and a library that records what would have
been launched for the real one."""
import ctypes

import pytest
import torch

import exact_replay_decode_amd as erd
from exact_replay_decode_amd import _lib, step

SH = erd.Shape(4, 2, 16, 16, 64)
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Recorder:
    """Every entry point of the library: notes its name, returns SSD_OK."""

    def __init__(self):
        self.calls = []

    def ssd_replay_pages_compact_workspace_bytes(self, cache):
        return (ctypes.cast(cache, ctypes.POINTER(_lib.ssd_replay_cache))[0].num_pages + 2) * 4

    def __getattr__(self, name):
        return lambda *args: self.calls.append(name) or 0


@pytest.fixture
def lib(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(step, "_dev", lambda t, name: t.device)
    monkeypatch.setattr(step, "_here", lambda device, stream: True)
    monkeypatch.setattr(step, "_raw_stream", lambda index: None)
    monkeypatch.setattr(step._lib, "load", lambda: rec)
    return rec


def refused(lib, match, fn, *args, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)
    assert lib.calls == []


def served(lib, fn, *args, **kw):
    fn(*args, **kw)
    assert lib.calls.pop() == fn.__name__ and lib.calls == []


def test_linear_out_shares_no_memory(lib):
    pool = torch.zeros(4096, dtype=BF)
    x, w, o = (pool[a:a + 256].view(16, 16) for a in (0, 512, 1024))
    r, b = pool[2048:2304].view(16, 16), torch.zeros(16)
    served(lib, erd.ssd_linear, x, w, b, out=o, residual=r)
    served(lib, erd.ssd_linear, x, w, b, out=r, residual=r)          # in place
    served(lib, erd.ssd_linear, x, x, out=o)                         # inputs may be one
    for bad, name in ((x, "x"), (w, "weight"), (pool[8:264].view(16, 16), "x"),
                      (pool[767:1023].view(16, 16), "weight"),
                      (pool[2056:2312].view(16, 16), "residual"),    # beside itself
                      (pool[1793:2049].view(16, 16), "residual")):
        refused(lib, f"out shares memory with {name}", erd.ssd_linear, x, w, b, residual=r,
                out=bad)
    refused(lib, "out shares memory with residual", erd.ssd_linear, x, w, residual=r,
            out=pool[2048:2560].view(F32).view(16, 16))
    # the last byte before and the first after are free
    served(lib, erd.ssd_linear, x, w, out=pool[256:512].view(16, 16))
    served(lib, erd.ssd_linear, x[:0], w, out=o[:0])


def test_linear_out_is_not_the_bias(lib):
    b = torch.zeros(16)
    x, w = torch.zeros(1, 8), torch.zeros(16, 8)
    refused(lib, "out shares memory with bias", erd.ssd_linear, x, w, b, out=b.view(1, 16))


def test_in_proj_parts_share_no_memory(lib):
    sh = erd.Shape(4, 2, 16, 16, 64, "f32", "f32")
    cd = erd.conv_dim(sh)
    pool = torch.zeros(20000)
    u, w = pool[:32].view(2, 16), pool[64:64 + 16 * (64 + cd + 4)].view(64 + cd + 4, 16)
    z, xBC, dt = pool[8000:8128].view(2, 4, 16), pool[8128:8128 + 2 * cd].view(2, cd), \
        pool[9000:9008].view(2, 4)
    served(lib, erd.ssd_in_proj, sh, u, w, out=(z, xBC, dt))
    refused(lib, "z and xBC share", erd.ssd_in_proj, sh, u, w,
            out=(pool[8001:8129].view(2, 4, 16), xBC, dt))
    refused(lib, "xBC and dt share", erd.ssd_in_proj, sh, u, w,
            out=(z, xBC, pool[8130:8138].view(2, 4)))
    refused(lib, "dt shares memory with u", erd.ssd_in_proj, sh, u, w,
            out=(z, xBC, pool[31:39].view(2, 4)))
    refused(lib, "z shares memory with weight", erd.ssd_in_proj, sh, u, w,
            out=(pool[64:192].view(2, 4, 16), xBC, dt))


def test_norm_out_is_an_input_or_apart(lib):
    sh = erd.Shape(4, 2, 16, 16, 64, "f32", "f32")
    pool = torch.zeros(4096)
    y, z, w = pool[:128].view(2, 4, 16), pool[256:384].view(2, 4, 16), pool[512:576]
    for out in (y, z, pool[128:256].view(2, 4, 16)):
        served(lib, erd.ssd_gated_norm, sh, y, w, z=z, out=out)
    served(lib, erd.ssd_gated_norm, sh, y, w, z=y, out=y)
    for at, name in ((4, "y"), (252, "z"), (512, "weight"), (575, "weight")):
        refused(lib, f"out shares memory with {name}", erd.ssd_gated_norm, sh, y, w, z=z,
                out=pool[at:at + 128].view(2, 4, 16))


def test_logprob_outputs_share_no_memory(lib):
    pool = torch.zeros(4096)
    logits, tok = pool[:400].view(4, 100), pool[400:404].view(I32)
    lp, ent, rank = pool[500:504], pool[504:508], pool[508:512].view(I32)
    ids, tlp = pool[512:524].view(I32).view(4, 3), pool[524:536].view(4, 3)
    good = erd.TokenLogprobs(lp, ent, rank, ids, tlp)
    served(lib, erd.ssd_token_logprobs, logits, tok, 3, out=good)
    served(lib, erd.ssd_token_logprobs, logits, tok, 0,
           out=erd.TokenLogprobs(lp, None, None, None, None))
    # (what a call does not write is not looked at)
    served(lib, erd.ssd_token_logprobs, logits, tok, 0, out=good._replace(top_ids=lp))
    for kw, match in ((dict(entropy=lp), "logprob and entropy"),
                      (dict(rank=pool[503:507].view(I32)), "share memory"),
                      (dict(top_logprobs=ids.view(F32)), "top_ids and top_logprobs"),
                      (dict(logprob=logits[0, :4]), "logprob shares memory with logits"),
                      (dict(rank=tok), "rank shares memory with tokens")):
        refused(lib, match, erd.ssd_token_logprobs, logits, tok, 3, out=good._replace(**kw))


def test_page_calls_write_no_list(lib):
    c = erd.ReplayCache(SH, 3, "cpu", page_tokens=16, num_pages=12)
    a, b, n, g = (torch.zeros(2, dtype=I32) for _ in range(4))
    reserve, copy, compact = (erd.ssd_replay_pages_reserve, erd.ssd_replay_cache_copy,
                              erd.ssd_replay_pages_compact)
    served(lib, reserve, SH, c, n, slot_idx=a, like_idx=b, granted=g)
    served(lib, reserve, SH, c, n, slot_idx=a, like_idx=a, granted=g)
    for bad, name in ((a, "slot_idx"), (b, "like_idx"), (n, "tokens"),
                      (c.buf_pages.view(-1)[2:4], "buf_pages"), (c.buf_len[1:], "buf_len")):
        refused(lib, f"granted shares memory with {name}", reserve, SH, c, n, slot_idx=a,
                like_idx=b, granted=bad)
    served(lib, copy, SH, c, c, a, b, copied=g)
    for bad, name in ((a, "dst_idx"), (b, "src_idx"), (c.buf_len[:2], "dst.buf_len")):
        refused(lib, f"copied shares memory with {name}", copy, SH, c, c, a, b, copied=bad)
    work = torch.zeros(20, dtype=I32)
    served(lib, compact, SH, c)
    served(lib, compact, SH, c, used=work[14:15], workspace=work[:14])
    refused(lib, "used and workspace share", compact, SH, c, used=work[13:14],
            workspace=work[:14])
    refused(lib, "used shares memory with buf_pages", compact, SH, c,
            used=c.buf_pages.view(-1)[:1])


def test_counts_past_32_bits_are_refused(lib):
    sh = erd.Shape(4, 2, 16, 16, 64, "f32", "f32")
    y, w = torch.zeros(2, 4, 16), torch.zeros(64)
    served(lib, erd.ssd_gated_norm, sh, y, w, groups=2)
    refused(lib, "32 bits", erd.ssd_gated_norm, sh, y, w, groups=2 ** 32 + 2)
    logits, tok = torch.zeros(1, 8), torch.zeros(1, dtype=I32)
    served(lib, erd.ssd_token_logprobs, logits, tok, 1)
    for k in (2 ** 32 + 1, -2 ** 32 + 1):
        refused(lib, "32 bits", erd.ssd_token_logprobs, logits, tok, k)
    c = erd.ReplayCache(SH, 3, "cpu")
    long = torch.zeros(1, dtype=I32).expand(2 ** 32 + 1)      # (takes no memory)
    refused(lib, "32 bits", erd.ssd_replay_cache_free, SH, c, slot_idx=long)
    refused(lib, "32 bits", erd.ssd_replay_cache_copy, SH, c, c, long, long)
