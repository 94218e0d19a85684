"""The cache's table calls in place, as captured steps repeat them: prompts of many tokens (two
kernels), tables that are slices of wider ones, pages given back."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from oracle import serving as os_
from test_gpu_kv_tables import I32, ints, state

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [2048, 2049, 7000])
def test_steps_of_many_tokens_and_releases(tokens):
    b, wide = 5, 40
    lens = [126, 0, 300, 5, 0]
    table, free, pages = state(lens, wide, 150, seed=tokens)
    free, count = free + [-9] * (pages - len(free)), len(free)
    outer = torch.full((b, wide + 7), -3, dtype=I32, device="cuda")
    dt = outer[:, 2:wide + 2]
    dt.copy_(ints(table))
    dl, df, dc, dn = ints(lens), ints(free), ints([count]), ints([0] * b)
    done = torch.zeros(b, dtype=torch.bool, device="cuda")
    start = ints([0, 10, 20, 30, 40])
    outs = dict(seq_lens_out=dl, free_count_out=dc, cu_tokens=ints([0] * (b + 1)),
                positions=ints([0] * tokens), slots=ints([0] * tokens, torch.int64))

    def step():
        api.nvfp4_kv_extend(dn, dl, dt, df, dc, tokens=tokens, start=start, **outs)
        api.nvfp4_kv_release(done, dl, dt, df, dc, dl, dc)

    step()  # nothing new, nothing done
    assert dl.tolist() == lens and dc.tolist() == [count]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for i, (new, ended) in enumerate([
            ([1000, 1, 0, 500, 2], [0, 0, 0, 0, 0]), ([3, 1000, 900, 0, 140], [1, 0, 0, 0, 1]),
            ([1500, 1, 1, 1, 128], [0, 1, 1, 1, 1]), ([0, 0, 0, 0, 0], [1, 0, 1, 0, 0])]):
        dn.copy_(ints(new))
        done.copy_(ints(ended, torch.bool))
        graph.replay()
        lens, count, cu, positions, slots, table = os_.extend(new, lens, table, free, count, tokens,
                                                              start.tolist())
        lens, count, free = os_.release(ended, lens, table, free, count)
        assert dl.tolist() == lens and dc.tolist() == [count] and dt.tolist() == table, i
        assert df.tolist() == free and outs["cu_tokens"].tolist() == cu
        assert outs["positions"].tolist() == positions and outs["slots"].tolist() == slots
    assert bool((outer[:, :2] == -3).all()) and bool((outer[:, wide + 2:] == -3).all())
    assert api.device_status() == 0


def test_a_refused_step_in_place_stays_as_it_was():
    lens, new = [100, 128, -5], [3000, 1, 4]
    table, free, pages = state(lens, 30, 10, seed=2)
    dl, dt, dc = ints(lens), ints(table), ints([10])
    got = api.nvfp4_kv_extend(ints(new), dl, dt, ints(free + [-9] * (pages - 10)), dc, tokens=4000,
                              seq_lens_out=dl, free_count_out=dc)
    assert api.device_status() == 1
    assert dl.tolist() == lens and dc.tolist() == [10] and dt.tolist() == table
    assert got.cu_tokens.tolist() == [0] * 4 and bool((got.slots == -1).all())
    assert bool((got.positions == -1).all())
