"""Python binding of the operators around the scan in a model step
(include/ssd_step.h): the mixer's projections, its gated norm, the log
probabilities of tokens, and the pages and slots of a replay cache.

As in api.py this is argument marshalling only: tensors are checked for
device, dtype, layout and size, and outputs that the caller passes for memory
of their own; then their data pointers and a HIP stream are handed to the
library. Calls run on the stream given, or on the current stream
of their tensors' device. Outputs that the caller does not pass are allocated
on that stream. No call records gradients.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple

import torch

from . import _lib
from .api import ReplayCache, Shape, _need, conv_dim

_CODE = {torch.float32: _lib.SSD_F32, torch.bfloat16: _lib.SSD_BF16}
_raw_stream = torch._C._cuda_getCurrentRawStream
_new = torch.empty_strided   # (1.2 us where torch.empty takes 1.6)


@contextlib.contextmanager
def _elsewhere(device, stream):
    """Makes `device` and `stream` (None: the device's current one) current,
    so that outputs are allocated for the stream that writes them."""
    if stream is not None and stream.device != device:
        raise ValueError(f"stream on {stream.device}, tensors on {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _here(device, stream):
    """Whether a call on `device` can run on the current stream as it is."""
    return stream is None and device.index == torch._C._cuda_getDevice()


def _dev(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: on {t.device}, expected a GPU")
    return t.device


def _chk(t, name, shape, dtype, device):
    """api._need, whose messages it leaves to it: these calls are short enough
    for the checks to count."""
    if (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype
            and t.get_device() == device.index and t.is_contiguous()):
        return t
    return _need(t, name, shape, dtype, device)


def _apart(outs, ins, same=()):
    """Refuses outputs that share memory with one another or with what the
    call reads (names with tensors; None and empty ones pass). same: names of
    inputs that the output (of the same size then) may be itself."""
    seen = []
    for name, t in outs:
        if t is None:
            continue
        a = t.data_ptr()
        b = a + t.nbytes
        for c, d, other in seen:
            if a < d and c < b and a < b:
                raise ValueError(f"{other} and {name} share memory")
        if a < b:
            seen.append((a, b, name))
    for name, t in ins:
        if t is None:
            continue
        a = t.data_ptr()
        b = a + t.nbytes
        for c, d, other in seen:
            if a < d and c < b and a < b and not (a == c and b == d and name in same):
                raise ValueError(f"{other} shares memory with {name}")


def _io(t, name):
    if t.dtype not in _CODE:
        raise ValueError(f"{name}: dtype {t.dtype} is not bfloat16 or float32")
    return _CODE[t.dtype]


def _i32(v, name):
    """A count for an int32 argument, which ctypes would cut to 32 bits."""
    v = int(v)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name}: {v} does not fit 32 bits")
    return v


def _p(t):
    return None if t is None else t.data_ptr()


def _shape(shape):
    """The C struct of a Shape by reference, made once per object."""
    c = shape.__dict__.get("_c")
    if c is None:
        c = shape.c()   # (no field: not compared, not hashed; copied and pickled as the rest)
        object.__setattr__(shape, "_c", c)
    return ctypes.byref(c)


def ssd_linear(x, weight, bias=None, activation="none", residual=None, out=None, out_dtype=None,
               stream=None):
    """act(x @ weight.T + bias) + residual, fused: x [M, K], weight [N, K],
    residual [M, N] of one dtype (bf16 or fp32), bias [N] fp32; K a
    multiple of 8 (bf16) or 4 (fp32). activation: none, silu, gelu (tanh form)
    or relu2. out [M, N] in out_dtype (x's by default; bf16 or fp32); out may
    be the residual. A row's bits do not depend on M."""
    dev = _dev(x, "x")
    if not _here(dev, stream):
        with _elsewhere(dev, stream):
            return ssd_linear(x, weight, bias, activation, residual, out, out_dtype)
    io = _io(x, "x")
    if x.dim() != 2 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("x and weight must be [M, K] and [N, K]")
    (M, K), N = x.shape, weight.shape[0]
    _chk(x, "x", (M, K), x.dtype, dev)
    _chk(weight, "weight", (N, K), x.dtype, dev)
    if bias is not None:
        _chk(bias, "bias", (N,), torch.float32, dev)
    if residual is not None:
        _chk(residual, "residual", (M, N), x.dtype, dev)
    if activation not in _lib.ACTIVATIONS:
        raise ValueError(f"activation {activation!r} is not one of {sorted(_lib.ACTIVATIONS)}")
    if out_dtype is None:
        out_dtype = x.dtype if out is None else out.dtype
    if out_dtype not in _CODE:
        raise ValueError(f"out_dtype {out_dtype} is not bfloat16 or float32")
    if out is None:
        out = _new((M, N), (N, 1), dtype=out_dtype, device=dev)
    else:
        _chk(out, "out", (M, N), out_dtype, dev)
        _apart((("out", out),), (("x", x), ("weight", weight), ("bias", bias),
                                 ("residual", residual)), ("residual",))
    rc = _lib.load().ssd_linear(M, N, K, io, _CODE[out_dtype], _lib.ACTIVATIONS[activation],
                                x.data_ptr(), weight.data_ptr(), _p(bias), _p(residual),
                                out.data_ptr(), _raw_stream(dev.index))
    _lib.check(rc, "ssd_linear")
    return out


def ssd_in_proj(shape: Shape, u, weight, bias=None, out=None, stream=None):
    """The mixer's in-projection: u [M, d_model] with weight
    [2*H*P + 2*G*N + H, d_model] (bias fp32 or None). Returns z [M, H, P], xBC
    [M, conv_dim] and raw dt [M, H], the arrays the gate, the conv and the
    scan take; out: the three to write into."""
    dev = _dev(u, "u")
    if not _here(dev, stream):
        with _elsewhere(dev, stream):
            return ssd_in_proj(shape, u, weight, bias, out)
    if u.dim() != 2:
        raise ValueError("u must be [M, d_model]")
    M, K = u.shape
    H, P, io, dtt = shape.H, shape.P, shape.io, shape.dtt
    cd = conv_dim(shape)
    N = H * P + cd + H
    _chk(u, "u", (M, K), io, dev)
    _chk(weight, "weight", (N, K), io, dev)
    if bias is not None:
        _chk(bias, "bias", (N,), torch.float32, dev)
    if out is None:
        z = _new((M, H, P), (H * P, P, 1), dtype=io, device=dev)
        xBC = _new((M, cd), (cd, 1), dtype=io, device=dev)
        dt = _new((M, H), (H, 1), dtype=dtt, device=dev)
    else:
        z, xBC, dt = out
        _chk(z, "z", (M, H, P), io, dev)
        _chk(xBC, "xBC", (M, cd), io, dev)
        _chk(dt, "dt", (M, H), dtt, dev)
        _apart((("z", z), ("xBC", xBC), ("dt", dt)),
               (("u", u), ("weight", weight), ("bias", bias)))
    rc = _lib.load().ssd_in_proj(_shape(shape), M, K, u.data_ptr(), weight.data_ptr(), _p(bias),
                                 z.data_ptr(), xBC.data_ptr(), dt.data_ptr(),
                                 _raw_stream(dev.index))
    _lib.check(rc, "ssd_in_proj")
    return z, xBC, dt


def ssd_gated_norm(shape: Shape, y, weight, z=None, groups=None, eps=1e-5,
                   norm_before_gate=False, out=None, stream=None):
    """RMS norm of y [T, H, P] over `groups` groups of whole heads (shape.G by
    default), scaled by weight [H*P] fp32 and gated by silu(z) before the norm
    (or after it, norm_before_gate); z None: no gate. out may be y or z."""
    dev = _dev(y, "y")
    if not _here(dev, stream):
        with _elsewhere(dev, stream):
            return ssd_gated_norm(shape, y, weight, z, groups, eps, norm_before_gate, out)
    io = shape.io
    full = (y.shape[0], shape.H, shape.P)
    _chk(y, "y", full, io, dev)
    _chk(weight, "weight", (shape.H * shape.P,), torch.float32, dev)
    if z is not None:
        _chk(z, "z", full, io, dev)
    if out is None:
        out = torch.empty_like(y)
    else:
        _chk(out, "out", full, io, dev)
        _apart((("out", out),), (("y", y), ("z", z), ("weight", weight)), ("y", "z"))
    rc = _lib.load().ssd_gated_norm(_shape(shape), full[0],
                                    shape.G if groups is None else _i32(groups, "groups"),
                                    float(eps), int(bool(norm_before_gate)), y.data_ptr(), _p(z),
                                    weight.data_ptr(), out.data_ptr(), _raw_stream(dev.index))
    _lib.check(rc, "ssd_gated_norm")
    return out


class TokenLogprobs(NamedTuple):
    """Results of ssd_token_logprobs, one row each (top_* None for top_k 0)."""
    logprob: torch.Tensor
    entropy: torch.Tensor
    rank: torch.Tensor
    top_ids: torch.Tensor | None
    top_logprobs: torch.Tensor | None


def ssd_token_logprobs(logits, tokens, top_k=0, out: TokenLogprobs | None = None, stream=None):
    """Log probability of tokens [T] (int32) under the softmax of logits [T, V]
    (bf16 or fp32), with the entropy, the token's rank (0 = greedy choice) and
    the top_k best tokens by value, ties to the lower index. -inf logits are
    masked tokens; a token outside [0, V) gets NaN and rank -1; a row with a
    NaN or +inf gets NaN, rank and ids -1."""
    dev = _dev(logits, "logits")
    if not _here(dev, stream):
        with _elsewhere(dev, stream):
            return ssd_token_logprobs(logits, tokens, top_k, out)
    if logits.dim() != 2:
        raise ValueError("logits must be [T, V]")
    T, V = logits.shape
    code = _io(logits, "logits")
    _chk(logits, "logits", (T, V), logits.dtype, dev)
    _chk(tokens, "tokens", (T,), torch.int32, dev)
    k = _i32(top_k, "top_k")
    if out is None:
        f, i = torch.float32, torch.int32
        out = TokenLogprobs(
            _new((T,), (1,), dtype=f, device=dev), _new((T,), (1,), dtype=f, device=dev),
            _new((T,), (1,), dtype=i, device=dev),
            _new((T, k), (k, 1), dtype=i, device=dev) if k > 0 else None,
            _new((T, k), (k, 1), dtype=f, device=dev) if k > 0 else None)
    else:
        _chk(out.logprob, "logprob", (T,), torch.float32, dev)
        if out.entropy is not None:
            _chk(out.entropy, "entropy", (T,), torch.float32, dev)
        if out.rank is not None:
            _chk(out.rank, "rank", (T,), torch.int32, dev)
        if k > 0:
            _chk(out.top_ids, "top_ids", (T, k), torch.int32, dev)
            _chk(out.top_logprobs, "top_logprobs", (T, k), torch.float32, dev)
        _apart(zip(out._fields, out[:5 if k > 0 else 3]),
               (("logits", logits), ("tokens", tokens)))
    rc = _lib.load().ssd_token_logprobs(
        T, V, code, logits.data_ptr(), tokens.data_ptr(), k, out.logprob.data_ptr(),
        _p(out.entropy), _p(out.rank), _p(out.top_ids), _p(out.top_logprobs),
        _raw_stream(dev.index))
    _lib.check(rc, "ssd_token_logprobs")
    return out


def _cache(cache, shape, name="cache"):
    """(device, C struct by reference) of a cache made for this shape."""
    if cache.shape is not shape and cache.shape != shape:
        raise ValueError(f"{name} was made for another shape")
    return cache.state.device, ctypes.byref(cache.struct())


def _list(slot_idx, cache, device):
    """(entries, slot list) of a call over slot_idx (None: every slot)."""
    if slot_idx is None:
        return cache.num_slots, None
    n = _i32(slot_idx.shape[0], "slot_idx")
    return n, _chk(slot_idx, "slot_idx", (n,), torch.int32, device).data_ptr()


def ssd_replay_pages_reserve(shape: Shape, cache: ReplayCache, tokens, slot_idx=None,
                             like_idx=None, granted=None, stream=None):
    """Hands out pages of a paged cache so that each listed slot (all of them
    by default) can take tokens[b] more tokens (an int, or an int32 tensor with
    one count per entry); like_idx: the slots whose buffered length counts, for
    slots about to be copied from them. Lowest free page first, in list order,
    all of a slot's pages or none. Returns granted [n] int32 (1: has them
    all)."""
    dev, cs = _cache(cache, shape)
    if not _here(dev, stream):
        with _elsewhere(dev, stream):
            return ssd_replay_pages_reserve(shape, cache, tokens, slot_idx, like_idx, granted)
    n, sl = _list(slot_idx, cache, dev)
    like = None if like_idx is None else _chk(like_idx, "like_idx", (n,), torch.int32, dev)
    if isinstance(tokens, torch.Tensor):
        tok, every = _chk(tokens, "tokens", (n,), torch.int32, dev).data_ptr(), 0
    else:
        tok, every = None, max(0, min(int(tokens), shape.chunk_size))
    if granted is None:
        granted = _new((n,), (1,), dtype=torch.int32, device=dev)
    else:
        _chk(granted, "granted", (n,), torch.int32, dev)
        _apart((("granted", granted),),
               (("tokens", None if tok is None else tokens), ("slot_idx", slot_idx),
                ("like_idx", like_idx), ("buf_pages", cache.buf_pages),
                ("buf_len", cache.buf_len)))
    rc = _lib.load().ssd_replay_pages_reserve(_shape(shape), cs, n, sl, _p(like), tok, every,
                                              granted.data_ptr(), _raw_stream(dev.index))
    _lib.check(rc, "ssd_replay_pages_reserve")
    return granted


def ssd_replay_pages_trim(shape: Shape, cache: ReplayCache, slot_idx=None, stream=None):
    """Returns the pages past the buffered tokens of the listed slots (all of
    them by default)."""
    dev, cs = _cache(cache, shape)
    if not _here(dev, stream):
        with _elsewhere(dev, stream):
            return ssd_replay_pages_trim(shape, cache, slot_idx)
    n, sl = _list(slot_idx, cache, dev)
    rc = _lib.load().ssd_replay_pages_trim(_shape(shape), cs, n, sl, _raw_stream(dev.index))
    _lib.check(rc, "ssd_replay_pages_trim")


def ssd_replay_cache_free(shape: Shape, cache: ReplayCache, slot_idx=None, stream=None):
    """Ends the listed slots (all of them by default): they become fresh, and
    a paged cache gets their pages back."""
    dev, cs = _cache(cache, shape)
    if not _here(dev, stream):
        with _elsewhere(dev, stream):
            return ssd_replay_cache_free(shape, cache, slot_idx)
    n, sl = _list(slot_idx, cache, dev)
    rc = _lib.load().ssd_replay_cache_free(_shape(shape), cs, n, sl, _raw_stream(dev.index))
    _lib.check(rc, "ssd_replay_cache_free")


def ssd_replay_cache_copy(shape: Shape, dst: ReplayCache, src: ReplayCache, dst_idx, src_idx,
                          copied=None, stream=None):
    """Slots dst_idx of dst become what slots src_idx of src are (sources may
    repeat: a fork). dst and src may be one cache or two that differ in slots,
    pages or layout; a paged dst needs pages first (ssd_replay_pages_reserve
    with like_idx). copied [n] int32, if given, tells which entries were."""
    dev, cd = _cache(dst, shape, "dst")
    sdev, cs = _cache(src, shape, "src")
    if sdev != dev:
        raise ValueError(f"src on {sdev}, expected {dev}")
    if not _here(dev, stream):
        with _elsewhere(dev, stream):
            return ssd_replay_cache_copy(shape, dst, src, dst_idx, src_idx, copied)
    n = _i32(dst_idx.shape[0], "dst_idx")
    _chk(dst_idx, "dst_idx", (n,), torch.int32, dev)
    _chk(src_idx, "src_idx", (n,), torch.int32, dev)
    if copied is not None:
        _chk(copied, "copied", (n,), torch.int32, dev)
        _apart((("copied", copied),),
               (("dst_idx", dst_idx), ("src_idx", src_idx), ("dst.buf_pages", dst.buf_pages),
                ("src.buf_pages", src.buf_pages), ("dst.buf_len", dst.buf_len),
                ("src.buf_len", src.buf_len)))
    rc = _lib.load().ssd_replay_cache_copy(_shape(shape), cd, cs, n, dst_idx.data_ptr(),
                                           src_idx.data_ptr(), _p(copied),
                                           _raw_stream(dev.index))
    _lib.check(rc, "ssd_replay_cache_copy")


def ssd_replay_pages_compact(shape: Shape, cache: ReplayCache, used=None, workspace=None,
                             stream=None):
    """Moves the pages in use to the front of the pool (pages 0..U-1) and the
    table with them. Returns used [1] int32, U on the device. workspace: an
    int32 tensor of num_pages + 2 words, if not to be allocated here."""
    dev, cs = _cache(cache, shape)
    if not _here(dev, stream):
        with _elsewhere(dev, stream):
            return ssd_replay_pages_compact(shape, cache, used, workspace)
    lib = _lib.load()
    words = lib.ssd_replay_pages_compact_workspace_bytes(cs) // 4
    given = used is not None or workspace is not None
    used = _new((1,), (1,), dtype=torch.int32, device=dev) if used is None else \
        _chk(used, "used", (1,), torch.int32, dev)
    if workspace is None:
        workspace = _new((words,), (1,), dtype=torch.int32, device=dev)
    else:
        _chk(workspace, "workspace", (words,), torch.int32, dev)
    if given:
        _apart((("used", used), ("workspace", workspace)), (("buf_pages", cache.buf_pages),))
    rc = lib.ssd_replay_pages_compact(_shape(shape), cs, used.data_ptr(), workspace.data_ptr(),
                                      4 * words, _raw_stream(dev.index))
    _lib.check(rc, "ssd_replay_pages_compact")
    return used
