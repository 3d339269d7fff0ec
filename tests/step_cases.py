"""Plain 64-bit implementations of the operators around the scan, and shared
helpers of their GPU tests."""
from __future__ import annotations

import math

import numpy as np
import torch

DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# half a step of the stored type, relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return torch.randn(*shape, generator=g, device=DEV).mul_(scale).to(dtype)


def activate64(v, act):
    if act == "silu":
        return v * torch.special.expit(v)
    if act == "gelu":
        return v * torch.special.expit(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    if act == "relu2":
        return torch.clamp(v, min=0) ** 2
    return v


def linear64(x, w, bias=None, act="none", residual=None):
    """(value, bound on the fp32 error before the last rounding) in fp64, on
    the host. The chain: K additions, each off by at most an ulp, 2**-23 of
    the partial sums' magnitude, itself at most mag = sum |x w| + |bias|; the
    bias adds one. An activation passes errors on at its slope (silu, gelu:
    at most 1.13; relu2: 2|v| + the error itself) and adds its own: exp2 of a
    rounded product, a reciprocal and a product, at most 4e-6 of the value
    plus 2e-6. The residual's addition rounds once more."""
    x, w = x.cpu().double(), w.cpu().double()
    v, mag = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        v, mag = v + bias.cpu().double(), mag + bias.cpu().double().abs()
    err = (x.shape[1] + 2) * 2.0 ** -23 * mag
    a = activate64(v, act)
    if act == "relu2":
        err = err * (2 * v.abs() + err) + 2.0 ** -23 * a
    elif act != "none":
        err = 1.13 * err + 4e-6 * a.abs() + 2e-6
    if residual is not None:
        a = a + residual.cpu().double()
        err = err + 2.0 ** -23 * a.abs()
    return a, err


def check_close(y, ref, err, what=""):
    """|y - ref| <= err plus half a step of y's type."""
    h = HALF[y.dtype]
    d = (y.cpu().double() - ref).abs()
    bound = err * (1 + h) + h * ref.abs() + 1e-37
    bad = ~(d <= bound)
    assert not bool(bad.any()), (what, float((d / bound).max()), int(bad.sum()))


# ---- pages and slots, on the host --------------------------------------------

class HostPages:
    """The page table of a cache as Python lists."""

    def __init__(self, table, lens, num_pages, Q, pt):
        self.t = [list(map(int, r)) for r in table]
        self.lens = [int(v) for v in lens]
        self.num_pages, self.Q, self.pt = num_pages, Q, pt

    def ok(self, p):
        return 0 <= p < self.num_pages

    def free(self):
        taken = {p for row in self.t for p in row if self.ok(p)}
        return [p for p in range(self.num_pages) if p not in taken]

    def reserve(self, slots, tokens, like=None):
        pool = self.free()
        room, asked, got = len(pool), 0, []
        for b, s in enumerate(slots):
            k = s if like is None else like[b]
            if not (0 <= s < len(self.t) and 0 <= k < len(self.t)
                    and 0 <= self.lens[k] < self.Q):
                got.append(0)
                continue
            n = -(-min(self.lens[k] + max(tokens[b], 0), self.Q) // self.pt)
            lack = [i for i in range(n) if not self.ok(self.t[s][i])]
            asked += len(lack)
            got.append(int(not lack or asked <= room))
            if got[-1]:
                for i in lack:
                    self.t[s][i] = pool.pop(0)
        return got

    def trim(self, slots):
        for s in slots:
            if 0 <= s < len(self.t) and self.lens[s] >= 0:
                self.t[s] = [p if i * self.pt < self.lens[s] else -1
                             for i, p in enumerate(self.t[s])]

    def compact(self):
        """Moves {from: to}; the table follows."""
        used = sorted({p for row in self.t for p in row if self.ok(p)})
        to = dict(zip([p for p in used if p >= len(used)], self.free()))
        self.t = [[to.get(p, p) for p in row] for row in self.t]
        return to, len(used)

    def table(self):
        return np.array(self.t, dtype=np.int32)
