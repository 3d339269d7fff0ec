"""The stream argument of the operators around the scan, made visible: the
stream given is the one that a graph captures, the current one is another. What
is launched on the stream given becomes part of the graph and runs on each
replay, over that replay's inputs; what is launched on the current stream runs
once, at the call, and the replays' outputs would be stale."""
import pytest
import torch

import exact_replay_decode_amd as erd
from gpu_cases import same_bits
from step_cases import DEV
from test_gpu_step_calls import Calls, _arrays, _cache, same

pytestmark = pytest.mark.gpu


def capture(call):
    """(graph, results) of call(stream) on the capturing stream, another one
    being current."""
    graph, given, other = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=given):
        with torch.cuda.stream(other):
            out = call(given)
            assert torch.cuda.current_stream() == other
    torch.cuda.synchronize()
    return graph, out


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 100])
def test_rows_are_computed_on_the_stream_given(io, rows):
    a, eager = Calls(io, rows).fill(0), Calls(io, rows)
    a.run(stream=torch.cuda.Stream())   # (loads the kernels)
    graph, out = capture(lambda s: a.run(stream=s))
    for seed in (1, 2, 3):
        a.fill(seed)
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        # (the same calls, so the same inputs for the norm: a stream of their own)
        want = eager.fill(seed).run(stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert same(out, want), seed


def test_pages_and_slots_change_on_the_stream_given():
    i32 = dict(dtype=torch.int32, device=DEV)
    ends, forks, like, five, three = (torch.tensor(v, **i32)
                                      for v in ([0, 1], [1, 0], [4, 2], [5], [3]))
    copied = [torch.zeros(2, **i32) for _ in range(2)]

    def calls(sh, c, ok, s):
        erd.ssd_replay_cache_free(sh, c, slot_idx=ends, stream=s)
        granted = erd.ssd_replay_pages_reserve(sh, c, 1, slot_idx=forks, like_idx=like, stream=s)
        erd.ssd_replay_cache_copy(sh, c, c, forks, like, copied=ok, stream=s)
        erd.ssd_replay_pages_trim(sh, c, stream=s)
        return granted, erd.ssd_replay_pages_compact(sh, c, stream=s)

    one = {  # each alone, so that none hides behind another
        "free": lambda sh, c, s: erd.ssd_replay_cache_free(sh, c, slot_idx=ends, stream=s),
        "reserve": lambda sh, c, s: erd.ssd_replay_pages_reserve(sh, c, 40, stream=s),
        "trim": lambda sh, c, s: erd.ssd_replay_pages_trim(sh, c, stream=s),
        "copy": lambda sh, c, s: erd.ssd_replay_cache_copy(sh, c, c, five, three, stream=s),
        "compact": lambda sh, c, s: erd.ssd_replay_pages_compact(sh, c, stream=s)}
    (sh, g), (_, e) = _cache(0), _cache(0)
    calls(sh, _cache(9)[1], copied[0], torch.cuda.Stream())   # (loads the kernels)
    torch.cuda.synchronize()
    graph, out = capture(lambda s: calls(sh, g, copied[0], s))
    graphs = {name: capture(lambda s: call(sh, g, s)) for name, call in one.items()}
    for seed in range(4):
        src = _cache(seed)[1]

        def reset():
            for c in (g, e):
                for to, frm in zip(_arrays(c), _arrays(src)):
                    to.copy_(frm)
            torch.cuda.synchronize()

        reset()
        graph.replay()
        want = calls(sh, e, copied[1], None)
        torch.cuda.synchronize()
        assert bool(want[0].all()) and same_bits(copied[0], copied[1])
        assert all(same_bits(x, y) for x, y in zip(out, want))
        assert all(same_bits(x, y) for x, y in zip(_arrays(g), _arrays(e))), seed
        for name, call in one.items():
            reset()
            graphs[name][0].replay()
            call(sh, e, None)
            torch.cuda.synchronize()
            assert all(same_bits(x, y) for x, y in zip(_arrays(g), _arrays(e))), (seed, name)
            assert not all(same_bits(x, y) for x, y in zip(_arrays(e), _arrays(src))), name
