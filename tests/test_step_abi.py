"""The operators around the scan (include/ssd_step.h) on the host: the
library exports what the header declares, and bad arguments are refused with
the documented status before anything is launched (fake device pointers; no
GPU needed). An accepted call would need one, so every call here is refused
or has nothing to do."""
import copy
import ctypes
import dataclasses
import os
import pickle
import re

import pytest
import torch

import exact_replay_decode_amd as erd
from exact_replay_decode_amd import _lib

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "include", "ssd_step.h")
OK, NULL, SHAPE, DTYPE, STATE, CHUNK, WORK, UNSUP, _, ALIGN = (0, -1, -2, -3, -4, -5, -6, -7, -8,
                                                               -9)
A = 0x1000          # an aligned fake address
BF16, F32 = _lib.SSD_BF16, _lib.SSD_F32


def shape(**kw):
    base = dict(H=4, G=2, P=16, N=16, chunk_size=64, io_dtype=1, dt_dtype=1, state_dtype=0,
                dt_softplus=1)
    base.update(kw)
    return _lib.ssd_shape(**base)


def cache(**kw):
    base = dict(state=A, state_bf=A, buf_x=A, buf_dt=A, buf_B=A, buf_C=None, buf_len=A,
                boundary_pos=A, work=None, num_slots=3, chunk_size=64, state_dtype=0,
                buf_pages=A, page_tokens=16, num_pages=12)
    base.update(kw)
    return _lib.ssd_replay_cache(**base)


def test_header_and_exports_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(ss\w+)\s*\(", text, flags=re.M))
    assert names == set(_lib.STEP_EXPORTS)
    lib = _lib.load()
    for name in names:
        assert hasattr(lib, name), name


def linear(M=4, N=8, K=16, io=BF16, out=BF16, act=0, x=A, w=A, bias=None, res=None, o=A):
    return _lib.load().ssd_linear(M, N, K, io, out, act, x, w, bias, res, o, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=0), SHAPE), (dict(K=-8), SHAPE),
    (dict(K=12), UNSUP), (dict(io=F32, out=F32, K=6), UNSUP), (dict(K=4), UNSUP),
    (dict(M=2 ** 31), UNSUP), (dict(N=2 ** 31), UNSUP), (dict(M=2 ** 30, N=2 ** 30), UNSUP),
    (dict(M=2 ** 18, N=2 ** 18 + 1), UNSUP), (dict(N=2 ** 29 + 1), UNSUP),
    (dict(K=2 ** 20 + 8), UNSUP), (dict(io=2), DTYPE), (dict(out=-1), DTYPE),
    (dict(act=4), UNSUP), (dict(act=-1), UNSUP), (dict(x=None), NULL), (dict(w=None), NULL),
    (dict(o=None), NULL), (dict(x=A + 8), ALIGN), (dict(w=A + 2), ALIGN),
    (dict(bias=A + 2), ALIGN), (dict(res=A + 1), ALIGN), (dict(o=A + 1), ALIGN),
    (dict(o=A + 2, out=F32), ALIGN),
    (dict(res=A, o=A, out=F32), DTYPE),   # in place with another dtype
    (dict(M=0, x=None, o=None), OK), (dict(N=0, w=None, o=None), OK)])
def test_linear_refusals(kw, code):
    assert linear(**kw) == code


@pytest.mark.parametrize("kw,skw,code", [
    (dict(M=-1), {}, SHAPE), (dict(K=0), {}, SHAPE), (dict(K=20), {}, UNSUP),
    (dict(u=None), {}, NULL), (dict(z=None), {}, NULL), (dict(dt=None), {}, NULL),
    (dict(x=None), {}, NULL), (dict(x=A + 1), {}, ALIGN), (dict(u=A + 8), {}, ALIGN),
    (dict(dt=A + 1), {}, ALIGN),
    ({}, dict(H=3), SHAPE), ({}, dict(P=24), UNSUP), ({}, dict(io_dtype=5), DTYPE),
    ({}, dict(state_dtype=1), STATE), (dict(M=0, u=None), {}, OK)])
def test_in_proj_refusals(kw, skw, code):
    a = dict(M=4, K=16, u=A, w=A, bias=None, z=A, x=A, dt=A)
    a.update(kw)
    assert _lib.load().ssd_in_proj(ctypes.byref(shape(**skw)), a["M"], a["K"], a["u"], a["w"],
                                   a["bias"], a["z"], a["x"], a["dt"], None) == code


@pytest.mark.parametrize("kw,skw,code", [
    (dict(T=-1), {}, SHAPE), (dict(groups=0), {}, SHAPE), (dict(groups=3), {}, SHAPE),
    (dict(eps=-1.0), {}, SHAPE), (dict(eps=float("nan")), {}, SHAPE),
    (dict(eps=float("inf")), {}, SHAPE), (dict(y=None), {}, NULL), (dict(w=None), {}, NULL),
    (dict(o=None), {}, NULL), (dict(z=A + 8), {}, ALIGN), (dict(w=A + 4), {}, ALIGN),
    (dict(groups=1), dict(H=512, G=1, P=128), UNSUP),    # a group of 65536 channels
    (dict(T=2 ** 31), {}, UNSUP), (dict(T=2 ** 28 + 1), {}, UNSUP), (dict(T=0, y=None), {}, OK)])
def test_gated_norm_refusals(kw, skw, code):
    a = dict(T=4, groups=2, eps=1e-5, y=A, z=None, w=A, o=A)
    a.update(kw)
    assert _lib.load().ssd_gated_norm(ctypes.byref(shape(**skw)), a["T"], a["groups"], a["eps"],
                                      0, a["y"], a["z"], a["w"], a["o"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), SHAPE), (dict(V=0), SHAPE), (dict(k=-1), SHAPE), (dict(k=11), SHAPE),
    (dict(V=100, k=65), UNSUP), (dict(V=2 ** 31 - 1), UNSUP), (dict(T=2 ** 31), UNSUP),
    (dict(T=2 ** 24 - 7), UNSUP), (dict(dt=3), DTYPE), (dict(x=None), NULL),
    (dict(tok=None), NULL), (dict(lp=None), NULL),
    (dict(k=1, ids=None), NULL), (dict(k=1, tlp=None), NULL), (dict(x=A + 1), ALIGN),
    (dict(x=A + 2, dt=F32), ALIGN), (dict(T=0, x=None), OK)])
def test_token_logprobs_refusals(kw, code):
    a = dict(T=4, V=10, dt=BF16, x=A, tok=A, k=0, lp=A, ent=None, rank=None, ids=A, tlp=A)
    a.update(kw)
    assert _lib.load().ssd_token_logprobs(a["T"], a["V"], a["dt"], a["x"], a["tok"], a["k"],
                                          a["lp"], a["ent"], a["rank"], a["ids"], a["tlp"],
                                          None) == code


BAD_CACHES = [
    (dict(state=None), NULL), (dict(buf_len=None), NULL), (dict(boundary_pos=None), NULL),
    (dict(num_slots=0), SHAPE), (dict(page_tokens=8), SHAPE), (dict(page_tokens=24), SHAPE),
    (dict(page_tokens=128), SHAPE), (dict(num_pages=0), SHAPE), (dict(chunk_size=32), CHUNK),
    (dict(state_dtype=1), STATE), (dict(buf_x=A + 8), ALIGN), (dict(num_pages=2 ** 20 + 1), UNSUP),
    (dict(num_slots=2 ** 29), UNSUP)]


@pytest.mark.parametrize("ckw,code", BAD_CACHES)
def test_page_calls_refuse_bad_caches(ckw, code):
    lib, sh, c = _lib.load(), ctypes.byref(shape()), ctypes.byref(cache(**ckw))
    good = ctypes.byref(cache())
    assert lib.ssd_replay_pages_reserve(sh, c, 1, A, None, None, 1, None, None) == code
    assert lib.ssd_replay_pages_trim(sh, c, 1, A, None) == code
    assert lib.ssd_replay_cache_free(sh, c, 1, A, None) == code
    assert lib.ssd_replay_cache_copy(sh, c, good, 1, A, A, None, None) == code
    assert lib.ssd_replay_cache_copy(sh, good, c, 1, A, A, None, None) == code
    assert lib.ssd_replay_pages_compact(sh, c, A, A, 1 << 30, None) == code


def test_page_calls_refuse_bad_arguments():
    lib, sh, c = _lib.load(), ctypes.byref(shape()), ctypes.byref(cache())
    flat = ctypes.byref(cache(buf_pages=None))
    assert lib.ssd_replay_pages_reserve(sh, flat, 1, A, None, None, 1, None, None) == NULL
    assert lib.ssd_replay_pages_trim(sh, flat, 1, A, None) == NULL
    assert lib.ssd_replay_pages_compact(sh, flat, A, A, 1 << 30, None) == NULL
    for n, code in ((-1, SHAPE), (4, SHAPE), (0, OK)):     # 3 slots, no list
        assert lib.ssd_replay_pages_reserve(sh, c, n, None, None, None, 1, None, None) == code
        assert lib.ssd_replay_pages_trim(sh, c, n, None, None) == code
        assert lib.ssd_replay_cache_free(sh, c, n, None, None) == code
        assert lib.ssd_replay_cache_free(sh, flat, n, None, None) == code
    assert lib.ssd_replay_cache_copy(sh, c, c, -1, A, A, None, None) == SHAPE
    assert lib.ssd_replay_cache_copy(sh, c, c, 1, None, A, None, None) == NULL
    assert lib.ssd_replay_cache_copy(sh, c, c, 1, A, None, None, None) == NULL
    with_c = ctypes.byref(cache(buf_C=A))
    assert lib.ssd_replay_cache_copy(sh, with_c, c, 1, A, A, None, None) == NULL
    assert lib.ssd_replay_cache_copy(sh, c, c, 0, None, None, None, None) == OK
    need = lib.ssd_replay_pages_compact_workspace_bytes(c)
    assert need == (12 + 2) * 4
    assert lib.ssd_replay_pages_compact_workspace_bytes(flat) == 0
    assert lib.ssd_replay_pages_compact(sh, c, None, A, need, None) == NULL
    assert lib.ssd_replay_pages_compact(sh, c, A, None, need, None) == WORK
    assert lib.ssd_replay_pages_compact(sh, c, A, A, need - 1, None) == WORK
    assert lib.ssd_replay_pages_compact(sh, c, A, A + 2, need, None) == ALIGN


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 8)
    sh = erd.Shape(4, 2, 16, 16, 64)
    with pytest.raises(ValueError, match="expected a GPU"):
        erd.ssd_linear(x, x)
    with pytest.raises(ValueError, match="expected a GPU"):
        erd.ssd_in_proj(sh, x, x)
    with pytest.raises(ValueError, match="expected a GPU"):
        erd.ssd_gated_norm(sh, x, x)
    with pytest.raises(ValueError, match="expected a GPU"):
        erd.ssd_token_logprobs(x, x)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        erd.ssd_linear(None, x)


def test_lists_too_long_for_a_launch_are_refused():
    lib, sh, c = _lib.load(), ctypes.byref(shape()), ctypes.byref(cache())
    n = 2 ** 24 - 7
    assert lib.ssd_replay_cache_free(sh, c, n, A, None) == UNSUP
    assert lib.ssd_replay_cache_copy(sh, c, c, n, A, A, None, None) == UNSUP


def test_a_shape_that_was_used_still_copies_and_pickles():
    """What the binding keeps with a Shape is no part of its value."""
    from exact_replay_decode_amd import step
    sh = erd.Shape(4, 2, 16, 16, 64)
    step._shape(sh)
    for other in (copy.copy(sh), copy.deepcopy(sh), pickle.loads(pickle.dumps(sh)),
                  dataclasses.replace(sh)):
        assert other == sh and hash(other) == hash(sh) and repr(other) == repr(sh)
        assert bytes(step._shape(other)._obj) == bytes(sh.c())
    more = dataclasses.replace(sh, H=8)
    assert more != sh and step._shape(more)._obj.H == 8
