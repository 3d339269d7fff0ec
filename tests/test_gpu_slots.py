"""Pages and slots of the replay cache on the GPU: tables against a host-side
page table in plain Python (step_cases.HostPages), copies against the source's
bytes, and decode going on with the same bits from forked, moved and
compacted slots."""
import numpy as np
import pytest
import torch

import exact_replay_decode_amd as erd
from gpu_cases import DEV, make_problem, same_bits
from step_cases import HostPages

pytestmark = pytest.mark.gpu

NAMES = ("state", "state_bf", "buf_x", "buf_dt", "buf_B", "buf_C", "buf_len", "boundary_pos",
         "buf_pages")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def random_cache(slots, Q, pt, num_pages, seed, H=3, G=1, P=16, N=16, io="bf16", dt="bf16",
                 with_C=False, fill=0.6):
    """A cache with random contents and a random table: some slots full, some
    empty, entries that are no pages among them."""
    sh = erd.Shape(H, G, P, N, Q, io, dt)
    rng = np.random.default_rng(seed)
    c = erd.ReplayCache(sh, slots, DEV, with_C, page_tokens=pt, num_pages=num_pages)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    for name in NAMES[:6]:
        t = getattr(c, name)
        if t is not None:
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
    lens = rng.integers(0, Q, slots)
    lens[:3] = [0, Q - 1, 1][:slots]
    c.buf_len.copy_(torch.from_numpy(lens.astype(np.int32)))
    c.boundary_pos.copy_(torch.from_numpy(Q * rng.integers(0, 9, slots)))
    npp = Q // pt
    table = np.full((slots, npp), -1, dtype=np.int32)
    pool = rng.permutation(num_pages).tolist()
    for s in range(slots):
        for i in range(npp):
            if pool and rng.random() < fill:
                table[s, i] = pool.pop()
            elif rng.random() < 0.2:
                table[s, i] = rng.choice([num_pages, num_pages + 7, -5, 2 ** 31 - 1, -2 ** 31])
    c.buf_pages.copy_(torch.from_numpy(table))
    return sh, c, HostPages(table, lens, num_pages, Q, pt), rng


SIZES = [(1, 16, 16, 1), (3, 64, 16, 12), (7, 64, 16, 33), (40, 256, 16, 700), (40, 256, 64, 100),
         (50, 128, 16, 300), (70, 256, 32, 400), (300, 256, 16, 4000), (1500, 32, 16, 2600),
         (2100, 64, 16, 40000)]


@pytest.mark.parametrize("slots,Q,pt,num_pages", SIZES)
def test_reserve_and_trim_match_the_host_table(slots, Q, pt, num_pages):
    for seed in range(4):
        sh, c, h, rng = random_cache(slots, Q, pt, num_pages, seed, fill=(0.2, 0.6, 0.9, 0.5)[seed])
        before = c.clone()
        n = int(rng.integers(1, slots + 1))
        pick = rng.permutation(slots)[:n].tolist()
        if n > 3:
            pick[1], pick[2] = -1, slots + 3        # skipped entries
        tok = rng.integers(-2, Q + 9, n).tolist()
        like = rng.integers(0, slots, n).tolist()
        if n > 5:
            like[4] = slots
        got = erd.ssd_replay_pages_reserve(sh, c, i32(tok), slot_idx=i32(pick))
        want = h.reserve(pick, tok)
        assert got.cpu().tolist() == want
        assert np.array_equal(c.buf_pages.cpu().numpy(), h.table())
        got = erd.ssd_replay_pages_reserve(sh, c, 0, slot_idx=i32(pick), like_idx=i32(like))
        assert got.cpu().tolist() == h.reserve(pick, [0] * n, like)
        assert np.array_equal(c.buf_pages.cpu().numpy(), h.table())
        erd.ssd_replay_pages_trim(sh, c, slot_idx=i32(pick))
        h.trim(pick)
        assert np.array_equal(c.buf_pages.cpu().numpy(), h.table())
        got = erd.ssd_replay_pages_reserve(sh, c, 1)
        assert got.cpu().tolist() == h.reserve(range(slots), [1] * slots)
        erd.ssd_replay_pages_trim(sh, c)
        h.trim(range(slots))
        assert np.array_equal(c.buf_pages.cpu().numpy(), h.table())
        for name in NAMES[:-1]:
            if getattr(c, name) is not None:
                assert same_bits(getattr(c, name), getattr(before, name)), name


def test_reserve_serves_in_order_until_the_pool_is_out():
    """Page counts written out by hand: 6 pages, needs 2, 3, 2, 1 and 0."""
    sh = erd.Shape(1, 1, 16, 16, 64)
    c = erd.ReplayCache(sh, 6, DEV, page_tokens=16, num_pages=7)
    c.buf_pages[5, 0] = 2                       # taken: free are 0 1 3 4 5 6
    c.buf_len.copy_(i32([20, 33, 31, 0, 5, 0]))
    got = erd.ssd_replay_pages_reserve(sh, c, i32([1, 1, 1, 1, 0]), slot_idx=i32([0, 1, 2, 3, 4]))
    # 0: 21 tokens, 2 pages; 1: 34, 3 pages; 2: 32, 2 pages (7 asked: too many); 3: 1 page (8
    # asked); 4: 5 tokens, 1 page (9 asked)
    assert got.tolist() == [1, 1, 0, 0, 0]
    assert c.buf_pages.tolist() == [[0, 1, -1, -1], [3, 4, 5, -1], [-1] * 4, [-1] * 4, [-1] * 4,
                                    [2, -1, -1, -1]]
    got = erd.ssd_replay_pages_reserve(sh, c, 1, slot_idx=i32([0, 3]))
    assert got.tolist() == [1, 1] and c.buf_pages[3, 0].item() == 6
    # a buffered length that is none is not served
    c.buf_len[4] = 64
    assert erd.ssd_replay_pages_reserve(sh, c, 0, slot_idx=i32([4, 0])).tolist() == [0, 1]


@pytest.mark.parametrize("slots,Q,pt,num_pages", SIZES)
@pytest.mark.parametrize("io,dt,with_C", [("bf16", "bf16", True), ("f32", "f32", False)])
def test_compact_matches_the_host_table(slots, Q, pt, num_pages, io, dt, with_C):
    for seed in range(3):
        sh, c, h, _ = random_cache(slots, Q, pt, num_pages, seed, io=io, dt=dt, with_C=with_C,
                                   fill=(0.05, 0.5, 1.0)[seed])
        before = c.clone()
        used = erd.ssd_replay_pages_compact(sh, c)
        moves, n = h.compact()
        assert used.tolist() == [n]
        assert np.array_equal(c.buf_pages.cpu().numpy(), h.table())
        a, b = (torch.tensor(v, dtype=torch.long, device=DEV) for v in
                (list(moves), list(moves.values())))
        for name in NAMES[2:6]:
            if getattr(c, name) is not None:
                want = getattr(before, name).clone()
                want[b] = want[a]
                assert same_bits(getattr(c, name), want), name
        for name in ("state", "state_bf", "buf_len", "boundary_pos"):
            assert same_bits(getattr(c, name), getattr(before, name)), name
        again = erd.ssd_replay_pages_compact(sh, c)
        assert again.tolist() == [n] and np.array_equal(c.buf_pages.cpu().numpy(), h.table())


def test_a_pool_of_the_largest_size():
    """1048576 pages (a 128 KB bitmap): the last ones are handed out and
    compacted away."""
    n = 1 << 20
    sh = erd.Shape(1, 1, 16, 16, 16)
    c = erd.ReplayCache(sh, 3, DEV, page_tokens=16, num_pages=n)
    c.buf_pages.copy_(i32([[n - 1], [-1], [31]]))
    c.buf_len.copy_(i32([4, 0, 3]))
    c.buf_x[n - 1] = 7.0
    assert erd.ssd_replay_pages_reserve(sh, c, 1, slot_idx=i32([1])).tolist() == [1]
    assert c.buf_pages.tolist() == [[n - 1], [0], [31]]
    assert erd.ssd_replay_pages_compact(sh, c).tolist() == [3]
    assert c.buf_pages.tolist() == [[2], [0], [1]]
    assert bool((c.buf_x[2] == 7.0).all())


def by_slot(c):
    """Buffers by slot with the rows past buf_len zeroed."""
    out = []
    live = torch.arange(c.shape.chunk_size, device=DEV)[None] < c.buf_len[:, None]
    for t in c.buffers_by_slot():
        out.append(None if t is None else
                   torch.where(live.reshape(live.shape + (1,) * (t.dim() - 2)), t, 0))
    return out


# (source pages, destination pages): contiguous, paged, other page sizes
@pytest.mark.parametrize("spt,dpt", [(None, None), (16, 16), (None, 32), (64, None), (16, 64),
                                     (64, 16)])
@pytest.mark.parametrize("H,P,N,io,dt", [(3, 16, 16, "bf16", "bf16"), (5, 32, 64, "f32", "bf16"),
                                         (32, 64, 128, "bf16", "f32")])
def test_copy_between_caches_and_layouts(spt, dpt, H, P, N, io, dt):
    Q = 64
    sh = erd.Shape(H, 1, P, N, Q, io, dt)
    g = torch.Generator(device=DEV)
    g.manual_seed(H)

    def make(slots, pt, with_C):
        c = erd.ReplayCache(sh, slots, DEV, with_C, page_tokens=pt,
                            num_pages=slots * (Q // pt) + 3 if pt else None)
        for name in NAMES[:6]:
            t = getattr(c, name)
            if t is not None:
                t.copy_(torch.randn(t.shape, generator=g, device=DEV))
        c.buf_len.copy_(torch.randint(0, Q, (slots,), generator=g, device=DEV))
        c.buf_len[:4] = i32([0, 1, Q - 1, 16])
        c.boundary_pos.copy_(Q * torch.randint(1, 9, (slots,), generator=g, device=DEV))
        if pt:
            perm = torch.randperm(c.num_pages, generator=g, device=DEV)
            c.buf_pages.copy_(perm[:slots * (Q // pt)].view(slots, -1))
        return c

    src, dst = make(9, spt, True), make(11, dpt, True)
    before, src_before = dst.clone(), src.clone()
    s, d = [0, 1, 2, 3, 2, 2, 8, 9, 4, -1, 5], [10, 0, 3, 7, 1, 2, 8, 4, 11, 5, 9]
    if spt:
        src.buf_pages[5, 0] = -1                # a page that slot 5 needs is missing
        src.buf_len[5] = 3
        src_before = src.clone()
    done = i32([7] * len(s))
    erd.ssd_replay_cache_copy(sh, dst, src, i32(d), i32(s), copied=done)
    ok = [int(0 <= a < 9 and 0 <= b < 11 and not (spt and a == 5)) for a, b in zip(s, d)]
    assert done.tolist() == ok
    want = before.clone()
    sb, db = by_slot(src), by_slot(dst)
    wb = by_slot(before)
    for a, b, o in zip(s, d, ok):
        if o:
            for name in ("state", "state_bf", "buf_len", "boundary_pos"):
                getattr(want, name)[b] = getattr(src, name)[a]
            for w, v in zip(wb, sb):
                w[b] = v[a]
    for name in ("state", "state_bf", "buf_len", "boundary_pos"):
        assert same_bits(getattr(dst, name), getattr(want, name)), name
    for x, y in zip(db, wb):
        assert same_bits(x, y)
    for name in NAMES:
        if getattr(src, name) is not None:
            assert same_bits(getattr(src, name), getattr(src_before, name)), name
    # rows past the copied ones, and pages of other slots, are left as they were
    live = torch.arange(Q, device=DEV)[None] < dst.buf_len[:, None]
    touched = torch.zeros(11, dtype=torch.bool, device=DEV)
    touched[[b for b, o in zip(d, ok) if o]] = True
    keep = ~(live & touched[:, None])
    for x, y in zip(dst.buffers_by_slot(), before.buffers_by_slot()):
        assert same_bits(x[keep], y[keep])


def test_copy_skips_a_destination_without_pages_and_a_slot_itself():
    sh, c, h, _ = random_cache(6, 64, 16, 40, 1)
    c.buf_pages.fill_(-1)
    c.buf_pages[0] = i32([0, 1, 2, 3])
    c.buf_pages[1] = i32([4, 5, -1, 41])
    c.buf_len.copy_(i32([40, 7, 0, 64, -1, 3]))
    before = c.clone()
    done = i32([9] * 4)
    # 1 lacks the third page; 2 needs none; 3 and 4 hold no length; 0 is itself
    erd.ssd_replay_cache_copy(sh, c, c, i32([1, 4, 5, 0]), i32([0, 2, 3, 0]), copied=done)
    assert done.tolist() == [0, 1, 0, 1]
    for s in (0, 1, 5):
        assert same_bits(c.state[s], before.state[s]) and c.buf_len[s] == before.buf_len[s]
    assert same_bits(c.state[4], before.state[2]) and int(c.buf_len[4]) == 0
    assert same_bits(c.buf_x, before.buf_x)
    with pytest.raises(ValueError, match="another shape"):
        erd.ssd_replay_cache_copy(erd.Shape(4, 1, 16, 16, 64), c, c, i32([1]), i32([0]))
    with pytest.raises(ValueError, match="dtype"):
        erd.ssd_replay_cache_copy(sh, c, c, i32([1]).long(), i32([0]))


@pytest.mark.parametrize("pt", [None, 16])
def test_free_makes_a_fresh_slot(pt):
    H, Q = 6, 64
    sh = erd.Shape(H, 2, 32, 64, Q)
    c = erd.ReplayCache(sh, 5, DEV, page_tokens=pt, num_pages=20 if pt else None)
    for name in NAMES[:5]:
        getattr(c, name).normal_()
    c.buf_len.fill_(9)
    c.boundary_pos.fill_(128)
    if pt:
        c.buf_pages.copy_(torch.arange(20, dtype=torch.int32, device=DEV).view(5, 4))
    before = c.clone()
    erd.ssd_replay_cache_free(sh, c, slot_idx=i32([3, -1, 1, 5]))
    for s in range(5):
        gone = s in (1, 3)
        for name in ("state", "state_bf", "buf_len", "boundary_pos"):
            got, was = getattr(c, name)[s], getattr(before, name)[s]
            assert bool((got == 0).all()) if gone else same_bits(got, was), (name, s)
        if pt:
            assert c.buf_pages[s].tolist() == ([-1] * 4 if gone else
                                               before.buf_pages[s].tolist())
    for name in NAMES[2:5]:
        assert same_bits(getattr(c, name), getattr(before, name))
    erd.ssd_replay_cache_free(sh, c)
    assert not bool(c.state.any()) and not bool(c.buf_len.any())


def test_state_past_4_gib():
    """Slots whose states lie past 32-bit byte offsets."""
    sh = erd.Shape(64, 1, 128, 128, 16)
    c = erd.ReplayCache(sh, 1040, DEV)
    c.state[1].fill_(2.0)
    c.state_bf[1].fill_(3.0)
    erd.ssd_replay_cache_copy(sh, c, c, i32([1039, 1030]), i32([1, 1]))
    for s in (1039, 1030):
        assert bool((c.state[s] == 2.0).all()) and bool((c.state_bf[s] == 3.0).all())
    erd.ssd_replay_cache_free(sh, c, slot_idx=i32([1039]))
    assert not bool(c.state[1039].any()) and bool((c.state[1030] == 2.0).all())
    assert not bool(c.state[1038].any())


@pytest.mark.parametrize("H,G,P,N,Q,io,pt", [(8, 2, 64, 128, 64, "bf16", 16),
                                             (4, 1, 16, 16, 32, "f32", 16)])
def test_forked_moved_and_compacted_slots_decode_on(H, G, P, N, Q, io, pt):
    """One prompt forked into three slots, one of them moved to a contiguous
    cache, the pool compacted half way: every copy decodes on with the bits of
    the single-shot prefill of the whole sequence."""
    L, pre = 3 * Q + 11, Q + Q // 2 + 3
    pr = make_problem([L], H=H, G=G, P=P, N=N, Q=Q, io=io, seed=4)
    x, dt, B, C = pr.dev(None)
    y_ss, _, _ = erd.ssd_prefill_varlen(pr.shape, pr.cu, x, dt, pr.A, B, C, pr.D, pr.bias)
    sh = pr.shape
    c = erd.ReplayCache(sh, 6, DEV, page_tokens=pt, num_pages=6 * (Q // pt))
    c.buf_x.normal_()
    c.buf_B.normal_()
    # slot 5 holds the front of the pool for a while
    assert erd.ssd_replay_pages_reserve(sh, c, Q, slot_idx=i32([5])).tolist() == [1]
    assert erd.ssd_replay_pages_reserve(sh, c, pre, slot_idx=i32([2])).tolist() == [1]
    erd.ssd_replay_prefill(sh, c, [0, pre], x[:pre], dt[:pre], B[:pre], C[:pre], pr.A, pr.D,
                           pr.bias, slot_idx=i32([2]))
    erd.ssd_replay_pages_trim(sh, c, slot_idx=i32([2]))
    dst, src = i32([0, 4, 1]), i32([2, 2, 2])
    assert erd.ssd_replay_pages_reserve(sh, c, 0, slot_idx=dst, like_idx=src).tolist() == [1] * 3
    erd.ssd_replay_cache_copy(sh, c, c, dst, src)
    flat = erd.ReplayCache(sh, 2, DEV)
    erd.ssd_replay_cache_copy(sh, flat, c, i32([1]), i32([4]))
    erd.ssd_replay_cache_free(sh, c, slot_idx=i32([4, 5]))
    slots = i32([2, 0, 1])
    for t in range(pre, L):
        if t == pre + 2:
            used = erd.ssd_replay_pages_compact(sh, c)
            assert int(c.buf_pages.max()) == int(used) - 1
        assert erd.ssd_replay_pages_reserve(sh, c, 1, slot_idx=slots).tolist() == [1] * 3
        rep = lambda v: v[t:t + 1].expand(3, *v.shape[1:]).contiguous()  # noqa: E731
        y = erd.ssd_replay_decode(sh, c, rep(x), rep(dt), rep(B), rep(C), pr.A, pr.D, pr.bias,
                                  slot_idx=slots)
        yf = erd.ssd_replay_decode(sh, flat, x[t:t + 1], dt[t:t + 1], B[t:t + 1], C[t:t + 1],
                                   pr.A, pr.D, pr.bias, slot_idx=i32([1]))
        erd.ssd_replay_pages_trim(sh, c, slot_idx=slots)
        for row in (*y, *yf):
            assert same_bits(row, y_ss[t]), t
