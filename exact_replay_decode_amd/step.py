"""Python binding of the operators around the scan in a model step
(include/ssd_step.h): the mixer's projections, its gated norm, the log
probabilities of tokens, and the pages and slots of a replay cache.

As in api.py this is argument marshalling only: tensors are checked for
device, dtype, layout and size, then their data pointers and a HIP stream are
handed to the library. Calls run on the stream given, or on the current stream
of their tensors' device. Outputs that the caller does not pass are allocated
on that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple

import torch

from . import _lib
from .api import ReplayCache, Shape, _need, _opt, _slots, conv_dim

_CODE = {torch.float32: _lib.SSD_F32, torch.bfloat16: _lib.SSD_BF16}


@contextlib.contextmanager
def _other(device, stream):
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _on(device, stream):
    """(context, raw stream) of a call on `device`: the context makes the
    device and the stream current where they are not yet, so that outputs are
    allocated for the stream that writes them."""
    cur = torch.cuda.current_stream(device)
    if device.index == torch.cuda.current_device() and (stream is None or stream == cur):
        return contextlib.nullcontext(), cur.cuda_stream
    s = cur if stream is None else stream
    if s.device != device:
        raise ValueError(f"stream on {s.device}, tensors on {device}")
    return _other(device, s), s.cuda_stream


def _dev(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: on {t.device}, expected a GPU")
    return t.device


def _io(t, name):
    if t.dtype not in _CODE:
        raise ValueError(f"{name}: dtype {t.dtype} is not bfloat16 or float32")
    return _CODE[t.dtype]


def _p(t):
    return None if t is None else t.data_ptr()


def ssd_linear(x, weight, bias=None, activation="none", residual=None, out=None, out_dtype=None,
               stream=None):
    """act(x @ weight.T + bias) + residual in one launch: x [M, K], weight
    [N, K], residual [M, N] of one dtype (bf16 or fp32), bias [N] fp32; K a
    multiple of 8 (bf16) or 4 (fp32). activation: none, silu, gelu (tanh form)
    or relu2. out [M, N] in out_dtype (x's by default; bf16 or fp32); out may
    be the residual. A row's bits do not depend on M."""
    dev = _dev(x, "x")
    io = _io(x, "x")
    if x.dim() != 2 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("x and weight must be [M, K] and [N, K]")
    (M, K), N = x.shape, weight.shape[0]
    _need(x, "x", (M, K), x.dtype, dev)
    _need(weight, "weight", (N, K), x.dtype, dev)
    _opt(bias, "bias", (N,), torch.float32, dev)
    _opt(residual, "residual", (M, N), x.dtype, dev)
    if activation not in _lib.ACTIVATIONS:
        raise ValueError(f"activation {activation!r} is not one of {sorted(_lib.ACTIVATIONS)}")
    if out_dtype is None:
        out_dtype = x.dtype if out is None else out.dtype
    if out_dtype not in _CODE:
        raise ValueError(f"out_dtype {out_dtype} is not bfloat16 or float32")
    ctx, st = _on(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty((M, N), dtype=out_dtype, device=dev)
        else:
            _need(out, "out", (M, N), out_dtype, dev)
        rc = _lib.load().ssd_linear(M, N, K, io, _CODE[out_dtype], _lib.ACTIVATIONS[activation],
                                    x.data_ptr(), weight.data_ptr(), _p(bias), _p(residual),
                                    out.data_ptr(), st)
    _lib.check(rc, "ssd_linear")
    return out


def ssd_in_proj(shape: Shape, u, weight, bias=None, out=None, stream=None):
    """The mixer's in-projection in one launch: u [M, d_model] with weight
    [2*H*P + 2*G*N + H, d_model] (bias fp32 or None). Returns z [M, H, P], xBC
    [M, conv_dim] and raw dt [M, H], the arrays the gate, the conv and the
    scan take; out: the three to write into."""
    dev = _dev(u, "u")
    if u.dim() != 2:
        raise ValueError("u must be [M, d_model]")
    M, K = u.shape
    cd = conv_dim(shape)
    N = shape.H * shape.P + cd + shape.H
    _need(u, "u", (M, K), shape.io, dev)
    _need(weight, "weight", (N, K), shape.io, dev)
    _opt(bias, "bias", (N,), torch.float32, dev)
    sh = shape.c()
    ctx, st = _on(dev, stream)
    with ctx:
        if out is None:
            z = torch.empty((M, shape.H, shape.P), dtype=shape.io, device=dev)
            xBC = torch.empty((M, cd), dtype=shape.io, device=dev)
            dt = torch.empty((M, shape.H), dtype=shape.dtt, device=dev)
        else:
            z, xBC, dt = out
            _need(z, "z", (M, shape.H, shape.P), shape.io, dev)
            _need(xBC, "xBC", (M, cd), shape.io, dev)
            _need(dt, "dt", (M, shape.H), shape.dtt, dev)
        rc = _lib.load().ssd_in_proj(ctypes.byref(sh), M, K, u.data_ptr(), weight.data_ptr(),
                                     _p(bias), z.data_ptr(), xBC.data_ptr(), dt.data_ptr(), st)
    _lib.check(rc, "ssd_in_proj")
    return z, xBC, dt


def ssd_gated_norm(shape: Shape, y, weight, z=None, groups=None, eps=1e-5,
                   norm_before_gate=False, out=None, stream=None):
    """RMS norm of y [T, H, P] over `groups` groups of whole heads (shape.G by
    default), scaled by weight [H*P] fp32 and gated by silu(z) before the norm
    (or after it, norm_before_gate); z None: no gate. out may be y or z."""
    dev = _dev(y, "y")
    T = int(y.shape[0])
    full = (T, shape.H, shape.P)
    _need(y, "y", full, shape.io, dev)
    _need(weight, "weight", (shape.H * shape.P,), torch.float32, dev)
    _opt(z, "z", full, shape.io, dev)
    sh = shape.c()
    ctx, st = _on(dev, stream)
    with ctx:
        out = torch.empty_like(y) if out is None else _need(out, "out", full, shape.io, dev)
        rc = _lib.load().ssd_gated_norm(ctypes.byref(sh), T,
                                        shape.G if groups is None else int(groups), float(eps),
                                        int(bool(norm_before_gate)), y.data_ptr(), _p(z),
                                        weight.data_ptr(), out.data_ptr(), st)
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
    if logits.dim() != 2:
        raise ValueError("logits must be [T, V]")
    T, V = logits.shape
    code = _io(logits, "logits")
    _need(logits, "logits", (T, V), logits.dtype, dev)
    _need(tokens, "tokens", (T,), torch.int32, dev)
    k = int(top_k)
    ctx, st = _on(dev, stream)
    with ctx:
        if out is None:
            f = torch.empty((2, T), dtype=torch.float32, device=dev)
            out = TokenLogprobs(
                f[0], f[1], torch.empty((T,), dtype=torch.int32, device=dev),
                torch.empty((T, k), dtype=torch.int32, device=dev) if k > 0 else None,
                torch.empty((T, k), dtype=torch.float32, device=dev) if k > 0 else None)
        else:
            _need(out.logprob, "logprob", (T,), torch.float32, dev)
            _opt(out.entropy, "entropy", (T,), torch.float32, dev)
            _opt(out.rank, "rank", (T,), torch.int32, dev)
            if k > 0:
                _need(out.top_ids, "top_ids", (T, k), torch.int32, dev)
                _need(out.top_logprobs, "top_logprobs", (T, k), torch.float32, dev)
        rc = _lib.load().ssd_token_logprobs(
            T, V, code, logits.data_ptr(), tokens.data_ptr(), k, out.logprob.data_ptr(),
            _p(out.entropy), _p(out.rank), _p(out.top_ids), _p(out.top_logprobs), st)
    _lib.check(rc, "ssd_token_logprobs")
    return out


def _list(slot_idx, cache):
    """(entries, slot list) of a call over slot_idx (None: every slot)."""
    if slot_idx is None:
        return cache.num_slots, None
    return int(slot_idx.shape[0]), _slots(slot_idx, int(slot_idx.shape[0]), cache.device)


def _device_of(cache, shape, name="cache"):
    if cache.shape != shape:
        raise ValueError(f"{name} was made for another shape")
    return cache.state.device


def ssd_replay_pages_reserve(shape: Shape, cache: ReplayCache, tokens, slot_idx=None,
                             like_idx=None, granted=None, stream=None):
    """Hands out pages of a paged cache so that each listed slot (all of them
    by default) can take tokens[b] more tokens (an int, or an int32 tensor with
    one count per entry); like_idx: the slots whose buffered length counts, for
    slots about to be copied from them. Lowest free page first, in list order,
    all of a slot's pages or none. Returns granted [n] int32 (1: has them
    all)."""
    dev = _device_of(cache, shape)
    n, sl = _list(slot_idx, cache)
    like = _slots(like_idx, n, dev)
    tok, every = (None, int(tokens)) if not isinstance(tokens, torch.Tensor) else \
        (_need(tokens, "tokens", (n,), torch.int32, dev), 0)
    every = max(min(every, shape.chunk_size), 0)
    sh, cs = shape.c(), cache.struct()
    ctx, st = _on(dev, stream)
    with ctx:
        granted = torch.empty((n,), dtype=torch.int32, device=dev) if granted is None else \
            _need(granted, "granted", (n,), torch.int32, dev)
        rc = _lib.load().ssd_replay_pages_reserve(ctypes.byref(sh), ctypes.byref(cs), n, _p(sl),
                                                  _p(like), _p(tok), every, granted.data_ptr(),
                                                  st)
    _lib.check(rc, "ssd_replay_pages_reserve")
    return granted


def ssd_replay_pages_trim(shape: Shape, cache: ReplayCache, slot_idx=None, stream=None):
    """Returns the pages past the buffered tokens of the listed slots (all of
    them by default)."""
    n, sl = _list(slot_idx, cache)
    sh, cs = shape.c(), cache.struct()
    ctx, st = _on(_device_of(cache, shape), stream)
    with ctx:
        rc = _lib.load().ssd_replay_pages_trim(ctypes.byref(sh), ctypes.byref(cs), n, _p(sl), st)
    _lib.check(rc, "ssd_replay_pages_trim")


def ssd_replay_cache_free(shape: Shape, cache: ReplayCache, slot_idx=None, stream=None):
    """Ends the listed slots (all of them by default): they become fresh, and
    a paged cache gets their pages back."""
    n, sl = _list(slot_idx, cache)
    sh, cs = shape.c(), cache.struct()
    ctx, st = _on(_device_of(cache, shape), stream)
    with ctx:
        rc = _lib.load().ssd_replay_cache_free(ctypes.byref(sh), ctypes.byref(cs), n, _p(sl), st)
    _lib.check(rc, "ssd_replay_cache_free")


def ssd_replay_cache_copy(shape: Shape, dst: ReplayCache, src: ReplayCache, dst_idx, src_idx,
                          copied=None, stream=None):
    """Slots dst_idx of dst become what slots src_idx of src are (sources may
    repeat: a fork). dst and src may be one cache or two that differ in slots,
    pages or layout; a paged dst needs pages first (ssd_replay_pages_reserve
    with like_idx). copied [n] int32, if given, tells which entries were."""
    dev = _device_of(dst, shape, "dst")
    n = int(dst_idx.shape[0])
    d, s = _slots(dst_idx, n, dev), _slots(src_idx, n, dev)
    if _device_of(src, shape, "src") != dev:
        raise ValueError(f"src on {src.state.device}, expected {dev}")
    _opt(copied, "copied", (n,), torch.int32, dev)
    sh, cd, cs = shape.c(), dst.struct(), src.struct()
    ctx, st = _on(dev, stream)
    with ctx:
        rc = _lib.load().ssd_replay_cache_copy(ctypes.byref(sh), ctypes.byref(cd),
                                               ctypes.byref(cs), n, _p(d), _p(s), _p(copied), st)
    _lib.check(rc, "ssd_replay_cache_copy")


def ssd_replay_pages_compact(shape: Shape, cache: ReplayCache, used=None, workspace=None,
                             stream=None):
    """Moves the pages in use to the front of the pool (pages 0..U-1) and the
    table with them. Returns used [1] int32, U on the device."""
    dev = _device_of(cache, shape)
    sh, cs = shape.c(), cache.struct()
    lib = _lib.load()
    need = lib.ssd_replay_pages_compact_workspace_bytes(ctypes.byref(cs))
    ctx, st = _on(dev, stream)
    with ctx:
        used = torch.empty((1,), dtype=torch.int32, device=dev) if used is None else \
            _need(used, "used", (1,), torch.int32, dev)
        if workspace is None:
            workspace = torch.empty((need // 4,), dtype=torch.int32, device=dev)
        size = workspace.numel() * workspace.element_size()
        rc = lib.ssd_replay_pages_compact(ctypes.byref(sh), ctypes.byref(cs), used.data_ptr(),
                                          workspace.data_ptr(), size, st)
    _lib.check(rc, "ssd_replay_pages_compact")
    return used
