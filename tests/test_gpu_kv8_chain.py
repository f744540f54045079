"""Calls that follow one another on a stream with nothing in between.  Every
kernel of the rotary positions and of the 8-bit cache starts beside its
predecessor and waits for it on the device, so each call here reads or
overwrites what the call just before it writes or reads; the same calls with
the device idle between them say what has to come out, bit for bit."""
import os
import subprocess
import sys

import pytest
import torch

import sparse_long_context_02_b200 as dsa

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


def _pools(P, page, Hkv, d):
    return [torch.zeros((P, page, Hkv, d), dtype=torch.uint8, device="cuda") for _ in "kv"] + [
        torch.zeros((P, Hkv), device="cuda") for _ in "kv"]


class Steps:
    """`steps` tokens for each of B sequences: rope, append, attend over every
    key, attend over selected ones; the attention's output is the next step's
    query, and the cache grows under the eyes of the next call."""

    def __init__(self, B, Hq, Hkv, d, page, start, steps, seed):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.Hq, self.Hkv, self.d, self.steps = B, Hq, Hkv, d, steps
        need = -(-(max(start) + steps) // page)
        self.x = torch.randn((steps, B, Hq + 2 * Hkv, d), generator=g, device="cuda").to(BF)
        self.cache = _pools(B * need, page, Hkv, d)
        order = torch.randperm(B * need, generator=g, device="cuda").int()
        self.table = order.reshape(B, need).contiguous()
        self.lens = [torch.tensor([n + s for n in start], dtype=torch.int32, device="cuda")
                     for s in range(steps + 1)]
        self.pos = [n.long() for n in self.lens]
        self.freqs = dsa.rope_freqs(d, 1e4)[0]
        first = torch.randn((max(sum(start), 1), Hkv, d), generator=g, device="cuda").to(BF)
        off = torch.tensor([sum(start[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
        if sum(start):
            dsa.kv8_append(first, first, *self.cache, self.table, torch.zeros_like(self.lens[0]),
                           off)
        self.begin = [t.clone() for t in self.cache]
        self.idx = torch.stack([torch.randperm(min(start) + 1, generator=g, device="cuda")[:16]
                                for _ in range(B)]).int().contiguous()

    def reset(self):
        for t, b in zip(self.cache, self.begin):
            t.copy_(b)

    def fresh_inputs(self):
        self.x.copy_(torch.randn(self.x.shape, generator=self.g, device="cuda"))

    def run(self, between=lambda: None):
        out = []
        O = None
        for s in range(self.steps):
            x = self.x[s]
            q0 = x[:, :self.Hq] if O is None else O
            q, k = dsa.rope(q0, x[:, self.Hq:self.Hq + self.Hkv], self.pos[s], self.freqs)
            between()
            dsa.kv8_append(k, x[:, self.Hq + self.Hkv:], *self.cache, self.table, self.lens[s])
            between()
            O = dsa.attn_kv8(q, *self.cache, self.table, self.lens[s + 1], 0.125)
            between()
            S = dsa.sparse_attn_kv8(O, *self.cache, self.table, self.lens[s + 1], self.idx, 0.125)
            between()
            out += [O, S]
            O = S
        return out


@pytest.mark.parametrize("B,Hq,Hkv,d,page,start", [
    (1, 32, 4, 128, 64, [700]), (3, 8, 2, 64, 16, [40, 15, 100]),
    (2, 32, 4, 128, 64, [30000, 17]), (64, 32, 4, 128, 16, [30 + b for b in range(64)]),
    (200, 8, 2, 64, 32, [31] * 200)])
def test_steps_in_a_graph_and_on_a_stream(B, Hq, Hkv, d, page, start):
    c = Steps(B, Hq, Hkv, d, page, start, 6, B)
    c.run()  # warm
    g = torch.cuda.CUDAGraph()
    c.reset()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        held = c.run()
    for _ in range(4):
        c.fresh_inputs()
        c.reset()
        want = c.run(torch.cuda.synchronize)
        cache = [t.clone() for t in c.cache]
        c.reset()
        got = c.run()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert all(torch.equal(a, b) for a, b in zip(cache, c.cache))
        c.reset()
        for t in held:
            t.fill_(7)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, held))
        assert all(torch.equal(a, b) for a, b in zip(cache, c.cache))
    assert dsa.device_error() == dsa.DEVERR_NONE


@pytest.mark.parametrize("B,n,kk", [(4, 900, 64), (2, 9000, 2048), (16, 300, 256)])
def test_attention_straight_behind_the_selection(B, n, kk):
    """The selection releases its successor at its start and then writes the
    index rows that the attention reads."""
    HI, dI, Hq, Hkv, d, page = 64, 128, 32, 4, 128, 64
    g = torch.Generator(device="cuda").manual_seed(n)

    def randn(*s):
        return torch.randn(s, generator=g, device="cuda")

    need = -(-n // page)
    cache = _pools(B * need, page, Hkv, d)
    table = torch.randperm(B * need, generator=g, device="cuda").int().reshape(B, need).contiguous()
    off = torch.arange(B + 1, device="cuda") * n
    x = randn(B * n, Hkv, d).to(BF)
    dsa.kv8_append(x, x, *cache, table, torch.zeros(B, dtype=torch.int32, device="cuda"), off.int())
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    kI = randn(B * n, dI).to(torch.float8_e4m3fn)
    qI, wI, Q = (torch.empty((B, HI, dI), dtype=torch.float8_e4m3fn, device="cuda"),
                 torch.empty((B, HI), device="cuda"), torch.empty((B, Hq, d), dtype=BF, device="cuda"))

    def fresh():
        qI.copy_(randn(B, HI, dI).to(torch.float8_e4m3fn))
        wI.copy_(randn(B, HI).abs())
        Q.copy_(randn(B, Hq, d))

    def run(between=lambda: None):
        _, idx = dsa.decode_select_shard(qI, wI, kI, off, kk)
        between()
        O = dsa.sparse_attn_kv8(Q, *cache, table, lens, idx, d ** -0.5)
        between()
        return idx, O

    fresh()
    run()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = [run() for _ in range(3)]
    for _ in range(10):
        fresh()
        want = run(torch.cuda.synchronize)
        assert int((want[0] >= 0).sum()) == B * min(kk, n)
        for pair in [run() for _ in range(3)]:
            assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])
        for idx, O in held:
            idx.fill_(-1)
        graph.replay()
        for idx, O in held:
            assert torch.equal(idx, want[0]) and torch.equal(O, want[1])
    assert dsa.device_error() == dsa.DEVERR_NONE


FIRST = """
import torch
import sparse_long_context_02_b200 as dsa
g = torch.Generator(device="cuda").manual_seed(1)
B, Hq, Hkv, d, page, M = 3, 32, 4, 128, 64, {pages}
q = torch.randn((B, Hq, d), generator=g, device="cuda").bfloat16()
x = torch.randn((B, Hkv, d), generator=g, device="cuda").bfloat16()
cache = [torch.zeros((B * M, page, Hkv, d), dtype=torch.uint8, device="cuda") for _ in "kv"]
cache += [torch.zeros((B * M, Hkv), device="cuda") for _ in "kv"]
table = torch.arange(B * M, dtype=torch.int32, device="cuda").reshape(B, M)
lens = torch.zeros(B, dtype=torch.int32, device="cuda")
one = torch.ones(B, dtype=torch.int32, device="cuda")
idx = torch.zeros((B, 8), dtype=torch.int32, device="cuda")
pos = torch.arange(B, device="cuda")
f = dsa.rope_freqs(d)[0]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):  # the process's first call of each
    rq, rk = dsa.rope(q, x, pos, f)
    dsa.kv8_append(rk, x, *cache, table, lens)
    O = dsa.attn_kv8(rq, *cache, table, one, 0.1)
    S = dsa.sparse_attn_kv8(rq, *cache, table, one, idx[:, :1].contiguous(), 0.1)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(O, dsa.attn_kv8(rq, *cache, table, one, 0.1)) and torch.equal(O, S)
v = (cache[1].view(torch.float8_e4m3fn).float() * cache[3][:, None, :, None])[::M, 0]
assert torch.equal(O, v.repeat_interleave(Hq // Hkv, 1).bfloat16())
assert dsa.device_error() == 0
print("captured")
"""


@pytest.mark.parametrize("pages", [2, 2000])
def test_the_first_calls_of_a_process_may_be_captured(pages):
    r = subprocess.run([sys.executable, "-c", FIRST.replace("{pages}", str(pages))], cwd=ROOT,
                       capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
