"""Steps of a server whose sequences share prefixes and see an encoder's states: pages and places
for the new tokens (nvfp4_kv_extend), positions, the append, single tokens behind the shared
prefixes (attn_qat_decode_prefix), all tokens to the encoder's keys (attn_qat_cross), and the
pages of ended sequences back (nvfp4_kv_release), against oracle/serving.py.  Tables, places and
records are equal; outputs keep the bounds of test_gpu_kv_cache.py."""
import pytest
import torch

from nvfp4_fake_quant_gb300 import api
from oracle import serving as os_
from test_gpu_cross import ints, offsets, vmax_of
from test_gpu_kv_cache import BF16, PAGE, check_decode, make_pool

pytestmark = pytest.mark.gpu
GROUPS, SHARED, STATES = [0, 3, 4], [200, 0], [300, 5, 0, 129]


class Server:
    def __init__(self, h, hkv, d, pages=40, wide=6):
        self.h, self.hkv, self.d, self.b = h, hkv, d, 4
        g = torch.Generator().manual_seed(h + d)
        self.g = g
        self.pool = make_pool(pages, hkv, d, g).cuda()
        perm = torch.randperm(pages, generator=g).tolist()
        take = [perm.pop() for _ in range(2)]
        self.prefix = ints([take, [-1, -1]])
        self.states = ints([[perm.pop() if i * PAGE < n else -1 for i in range(3)] for n in STATES])
        self.shared, self.state_lens, self.groups = ints(SHARED), ints(STATES), ints(GROUPS)
        starts = [SHARED[0]] * 3 + [SHARED[1]]
        self.start = ints(starts)
        self.freq = api.rope_inv_freq(d, device="cuda")[0]
        # the oracle's tables
        self.o_lens, self.o_free, self.o_count = [0] * 4, perm + [-9] * (pages - len(perm)), len(perm)
        self.o_table, self.o_start = [[-7] * wide for _ in range(4)], starts
        self.lens, self.count = ints(self.o_lens), ints([self.o_count])
        self.table, self.free = ints(self.o_table), ints(self.o_free)

    def step(self, qkv, new, single):
        """One step of qkv bf16 [T, H + 2 Hkv, D] and new int32 [B]; ``single``: a token each."""
        step = api.nvfp4_kv_extend(new, self.lens, self.table, self.free, self.count,
                                   tokens=qkv.shape[0], start=self.start, seq_lens_out=self.lens,
                                   free_count_out=self.count)
        q, k = api.rope_apply(qkv[:, :self.h], qkv[:, self.h:self.h + self.hkv], step.positions,
                              self.freq)
        api.nvfp4_kv_append_slots(k, qkv[:, self.h + self.hkv:], step.slots, self.pool)
        got = (step, q, k)
        if single:
            got += api.attn_qat_decode_prefix(q, self.pool, self.table, self.lens, self.prefix,
                                              self.shared, self.groups)
        return got + api.attn_qat_cross(q, self.pool, self.states, self.state_lens,
                                        step.cu_tokens)

    def check(self, qkv, new, got, single):
        step, q, k, *outs = got
        t = qkv.shape[0]
        after, self.o_count, cu, positions, slots, self.o_table = os_.extend(
            new, self.o_lens, self.o_table, self.o_free, self.o_count, t, self.o_start)
        self.o_lens = after
        assert api.device_status() == 0
        assert self.lens.tolist() == after and self.count.tolist() == [self.o_count]
        assert self.table.tolist() == self.o_table and step.cu_tokens.tolist() == cu
        assert step.positions.tolist() == positions and step.slots.tolist() == slots
        want = api.rope_apply(qkv[:, :self.h], qkv[:, self.h:self.h + self.hkv], ints(positions),
                              self.freq)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
        there = torch.tensor(slots[:cu[-1]], dtype=torch.long)
        parts = os_.record_parts(self.pool, self.d)
        for x, at in ((k, 0), (qkv[:, self.h + self.hkv:], 1)):
            for part, packed in zip(parts[at::2], os_.pack(x[:cu[-1]].cpu())):
                assert torch.equal(part[there // PAGE, :, there % PAGE], packed)
        pool, vmax, scale = self.pool.cpu(), vmax_of(self.pool, self.d), self.d ** -0.5
        q = q.cpu()
        if single:
            refs = []
            for b in range(self.b):
                s = 0 if b < GROUPS[1] else 1
                spans = [(self.prefix[s], SHARED[s]), (torch.tensor(self.o_table[b]), after[b])]
                refs.append(os_.attend(q[b:b + 1], pool, spans, scale))
            ref = tuple(torch.cat(x) for x in zip(*refs))
            check_decode(*outs[:2], ref, max(after) + max(SHARED), vmax)
        o, lse = outs[-2:]
        for b, n in enumerate(STATES):
            r = slice(cu[b], cu[b + 1])
            ref = os_.attend(q[r], pool, [(self.states[b], n)], scale)
            check_decode(o[r], lse[r], ref, n, vmax)
        assert not bool(o[cu[-1]:].any()) and bool((lse[cu[-1]:] == -float("inf")).all())

    def release(self, done):
        api.nvfp4_kv_release(torch.tensor(done, device="cuda"), self.lens, self.table, self.free,
                             self.count, self.lens, self.count)
        self.o_lens, self.o_count, self.o_free = os_.release(done, self.o_lens, self.o_table,
                                                             self.o_free, self.o_count)
        assert self.lens.tolist() == self.o_lens and self.count.tolist() == [self.o_count]
        assert self.free.tolist() == self.o_free and api.device_status() == 0

    def rows(self, t):
        return torch.randn(t, self.h + 2 * self.hkv, self.d, generator=self.g).to(BF16).cuda()


@pytest.mark.parametrize("h,hkv,d", [(8, 2, 128), (4, 4, 64)])
def test_prompts_then_captured_single_tokens(h, hkv, d):
    server = Server(h, hkv, d)
    # prompts of several lengths, one sequence without, rows behind the last token
    new = [126, 0, 255, 3]
    x = server.rows(sum(new) + 2)
    server.check(x, new, server.step(x, ints(new), False), False)
    # single tokens: once, then as replays of a captured step
    ones, x = ints([1] * 4), server.rows(4)
    server.check(x, [1] * 4, server.step(x, ones, True), True)
    state = [t.clone() for t in (server.lens, server.count, server.table, server.pool)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = server.step(x, ones, True)
    for t, v in zip((server.lens, server.count, server.table, server.pool), state):
        assert torch.equal(t, v)  # the capture ran nothing
    for i in range(4):  # over a page's end, and through an ended sequence that begins again
        x.copy_(server.rows(4))
        graph.replay()
        server.check(x, [1] * 4, got, True)
        if i == 1:
            server.release([True, False, False, True])


def test_a_step_that_does_not_fit_writes_nothing_and_is_reported():
    server = Server(4, 4, 64, pages=11)
    new = [128] * 4  # four pages of the three that are free
    assert server.o_count == 3
    x, before = server.rows(512), [t.clone() for t in (server.lens, server.count, server.table,
                                                       server.pool)]
    step, _, _, o, lse = server.step(x, ints(new), False)
    assert api.device_status() == 1
    for t, v in zip((server.lens, server.count, server.table, server.pool), before):
        assert torch.equal(t, v)
    assert step.slots.tolist() == [-1] * 512 and step.cu_tokens.tolist() == offsets([0] * 4)
    assert not bool(o.any()) and bool((lse == -float("inf")).all())


def test_the_timing_files_each_call_under_its_kind():
    server = Server(4, 2, 64)
    x, ones = server.rows(4), ints([1] * 4)
    server.step(x, ones, True)
    api.timing_enable(True)
    try:
        server.step(x, ones, True)
        api.nvfp4_kv_release(torch.zeros(4, dtype=torch.bool, device="cuda"), server.lens,
                             server.table, server.free, server.count)
        got = {k: n for k, (n, _) in api.timing_read().items() if n}
    finally:
        api.timing_enable(False)
    # the prefix part is timed as cross attention, the fold as a decode
    assert got == {"kv_tables": 2, "rope": 1, "kv_append": 1, "cross": 2, "decode": 1}
    assert api.device_status() == 0
