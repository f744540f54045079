"""GPU parity of the attention over the paged 8-bit cache
(dsa_sparse_attn_kv8, dsa_attn_kv8) against the float64 oracle
(oracle/kv8.py) on the stored rows.

Tolerance.  A score is an exact product of fp16 values summed in fp32, 16 at a
time: with up to 8 partial sums, truncated, and three fp32 products after
them it is off by less than E = 2^-19 scale sum_c |q_c k_c| (nats); a softmax
weight then by exp(2 E) - 1 with the normaliser's share, plus 2^-11 for its
rounding to fp16, 2^-18 for the exponentials and the fp32 sums.  Weights below
2^-29 of the largest (weight times scale of V) are off by 2^-40 of it in
absolute terms, times codes of up to 448, for each of n keys: n 2^-31 max(p
v_scale).  The output is rounded to bf16 (2^-8 by finfo.eps / 2), lse is off
by E, the sum's 2^-18 and its own fp32 rounding."""
import numpy as np
import pytest
import torch

import oracle.kv8 as KV
import sparse_long_context_02_b200 as dsa

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(x):
    t = torch.from_numpy(np.asarray(x, np.float32)).bfloat16()
    return t.double().numpy(), t.cuda()


class Case:
    """Random codes in a fragmented pool; slots past a sequence hold NaN."""

    def __init__(self, lens, page, Hq, Hkv, d, seed=0, rows=None, codes=None, extra=0):
        r = self.r = np.random.default_rng(seed)
        self.lens, self.page, self.Hq, self.Hkv, self.d = lens, page, Hq, Hkv, d
        need = [-(-max(n, 0) // page) for n in lens]
        P = sum(need) + 2
        order = r.permutation(P)
        M, at = max(need + [1]) + extra, 0
        self.table = np.full((len(lens), M), -1, np.int32)
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        self.pools = []
        for _ in "kv":
            x = KV.encode(r.normal(size=(P, page, Hkv, d)) * 64)
            for p in order[at:]:
                x[p] = 127
            for b, n in enumerate(lens):
                if n > 0 and n % page:
                    x[self.table[b, n // page], n % page:] = 127
            self.pools.append(x)
        self.scales = [2.0 ** r.integers(-8, -3, (P, Hkv)) for _ in "kv"]
        self.row_off = None if rows is None else np.concatenate([[0], np.cumsum(rows)])
        self.T = len(lens) if rows is None else int(self.row_off[-1])
        self.seq = (np.arange(len(lens)) if rows is None
                    else np.repeat(np.arange(len(lens)), rows))
        self.seen = [max(lens[b], 0) for b in self.seq]
        if rows is not None:
            for t in range(self.T):
                b = self.seq[t]
                self.seen[t] = max(0, lens[b] - (int(self.row_off[b + 1]) - 1 - t))
        self.scale = d ** -0.5
        self.set_q(r.normal(size=(self.T, Hq, d)) * 2.0 ** r.uniform(-1, 2, (self.T, Hq, 1)))

    def set_q(self, q, tail=0):
        if tail:
            q = np.concatenate([q, np.ones((tail, self.Hq, self.d))])
        self.Q, self.Qt = bf16(q)
        self.Q = self.Q[:self.T]

    def cache(self):
        return (dev(self.pools[0]), dev(self.pools[1]), dev(self.scales[0].astype(np.float32)),
                dev(self.scales[1].astype(np.float32)), dev(self.table),
                dev(np.asarray(self.lens, np.int32)))

    def select(self, k, holes=True):
        idx = np.full((self.T, k), -1, np.int32)
        for t in range(self.T):
            m = min(k, self.seen[t])
            idx[t, :m] = np.sort(self.r.choice(self.seen[t], m, replace=False)) if m else 0
            if holes and m > 2 and t % 3 == 1:
                idx[t, self.r.integers(0, m)] = -1
                idx[t, 0] = idx[t, 1]
        return idx

    def run(self, idx=None, **kw):
        ro = None if self.row_off is None else dev(self.row_off.astype(np.int32))
        lse = torch.full(self.Qt.shape[:2], 77.0, device="cuda")
        O = torch.full_like(self.Qt, 55.0)
        if idx is None:
            dsa.attn_kv8(self.Qt, *self.cache(), self.scale, row_off=ro, O=O, lse=lse, **kw)
        else:
            dsa.sparse_attn_kv8(self.Qt, *self.cache(), dev(idx), self.scale, row_off=ro, O=O,
                                lse=lse, **kw)
        return O, lse

    def keys(self, idx=None):
        if idx is None:
            return [np.arange(n) for n in self.seen]
        return [[s for s in row if 0 <= s < max(self.lens[b], 0)]
                for row, b in zip(idx, self.seq)]

    def check(self, O, lse, idx=None):
        keys = self.keys(idx)
        ref, rl, mag, big, top = KV.attention(self.Q, *self.pools, *self.scales, self.table,
                                              self.seq, keys, self.scale)
        O = O.double().cpu().numpy()
        assert np.all(O[self.T:] == 55.0) and torch.all(lse[self.T:] == 77.0)
        lse = lse.double().cpu().numpy()[:self.T]
        E = 2.0 ** -19 * big
        n = np.array([len(s) for s in keys])[:, None]
        tol = (mag * (np.expm1(2 * E) + 2.0 ** -11 + 2.0 ** -18)[..., None] +
               (n * 2.0 ** -31 * top)[..., None])
        tol = tol + (np.abs(ref) + tol) * 2.0 ** -8
        err = np.abs(O[:self.T] - ref)
        assert np.all(err <= tol), (np.argwhere(~(err <= tol))[:4], np.nanmax(err / (tol + 1e-30)))
        dead = n[:, 0] == 0
        assert np.all(lse[dead] == -np.inf) and np.all(O[:self.T][dead] == 0)
        ltol = (E + 2.0 ** -18)[~dead] + np.abs(rl[~dead]) * 2.0 ** -22
        assert np.all(np.abs(lse[~dead] - rl[~dead]) <= ltol)
        assert dsa.device_error() == dsa.DEVERR_NONE


SHAPES = [(32, 4, 128), (8, 2, 64), (7, 1, 128), (3, 3, 64), (5, 1, 64), (16, 2, 128), (64, 64, 64),
          (6, 2, 128)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
def test_dense_single_tokens(Hq, Hkv, d, page):
    c = Case([1, 0, page, 300, -1, 2, page + 1, 777, 15, 16, 17], page, Hq, Hkv, d, page + d)
    c.check(*c.run())


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
@pytest.mark.parametrize("k", [1, 16, 100, 513])
def test_sparse_single_tokens(Hq, Hkv, d, page, k):
    c = Case([1, 0, page, 700, -1, 2, 1000], page, Hq, Hkv, d, page + d)
    idx = c.select(k)
    idx[3] = -1
    c.check(*c.run(idx), idx)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("Hq,Hkv,d", [(32, 4, 128), (8, 2, 64), (5, 1, 128)])
def test_chunks_and_several_tokens_each(Hq, Hkv, d, page):
    """Rows of ragged chunks, sequences without rows or keys, a chunk longer
    than its sequence (its first rows see nothing), rows behind the last."""
    rows = [37, 0, 4, 1, 0, 9, 2]
    lens = [200, 50, 4, 333, 0, 5, -1]
    c = Case(lens, page, Hq, Hkv, d, 5, rows)
    c.set_q(c.r.normal(size=(c.T, Hq, d)) * 2, tail=3)
    c.check(*c.run())
    idx = c.select(48)
    tail = np.full((3, 48), 1 << 30, np.int32)
    c.check(*c.run(np.concatenate([idx, tail])), idx)


@pytest.mark.parametrize("Hq,Hkv,d", [(32, 4, 128), (8, 2, 64)])
def test_long_rows_in_slices(Hq, Hkv, d):
    """One to three rows over tens of thousands of keys: split over the whole
    GPU and joined."""
    c = Case([40000, 3, 70001], 64, Hq, Hkv, d, 7)
    c.check(*c.run())
    idx = c.select(2048, holes=False)
    c.check(*c.run(idx), idx)
    c = Case([33333], 128, Hq, Hkv, d, 8, extra=5)
    c.check(*c.run())
    again = c.run()
    assert all(torch.equal(a, b) for a, b in zip(c.run(), again))


def test_many_rows():
    c = Case([3000], 64, 32, 4, 128, 9, rows=[800])
    idx = c.select(130)
    got = c.run(idx)
    c.T, c.Q, c.seq, c.seen = 800, c.Q, c.seq, c.seen
    c.check(*got, idx)


@pytest.mark.parametrize("T,Hq,Hkv,d,longest,k", [
    (1, 32, 4, 128, 4000, 0), (1, 32, 4, 128, 30, 0), (2, 8, 2, 64, 5000, 300),
    (20, 32, 4, 128, 900, 257), (74, 32, 4, 128, 300, 64), (75, 8, 4, 64, 300, 64),
    (148, 8, 4, 128, 200, 33), (149, 8, 4, 128, 200, 33), (148, 3, 3, 64, 200, 0),
    (300, 8, 2, 64, 120, 0), (512, 4, 1, 128, 90, 0), (513, 4, 1, 128, 90, 0),
    (600, 8, 4, 64, 70, 0), (600, 6, 2, 128, 70, 20), (9, 64, 64, 64, 700, 0),
    (5, 63, 63, 64, 200, 100)])
def test_numbers_of_rows(T, Hq, Hkv, d, longest, k):
    """Every way of dividing a launch: clusters of 8 to 1 CTAs per row, rows cut
    into equal ranges (fewer and more rows than CTAs), whole rows."""
    r = np.random.default_rng(T)
    c = Case([int(n) for n in r.integers(0, longest + 1, T)], 16, Hq, Hkv, d, T)
    idx = c.select(k) if k else None
    c.check(*c.run(idx), idx)


def test_long_chunks():
    """600 rows of one sequence over every key (causal), and 200 rows of three."""
    c = Case([650], 32, 8, 2, 64, 19, rows=[600])
    c.check(*c.run())
    c = Case([300, 40, 500], 16, 4, 1, 128, 20, rows=[100, 40, 60])
    c.check(*c.run())


def test_a_long_tail_of_small_weights():
    """One key far ahead of 60000: their sum is half the output."""
    n, d = 60000, 64
    c = Case([n], 64, 8, 1, d, 10)
    c.pools[0][:] = 0
    t, q = c.table[0, 12345 // 64], np.zeros((1, 8, d))
    c.pools[0][t, 12345 % 64, 0, 0] = KV.encode(256.0)
    c.scales[0][:] = 2.0 ** -8
    for h in range(8):  # weights of 1 / n (1 ... 2^-14) each
        q[0, h, 0] = (np.log(n) + h * 1.39) * 8
    c.pools[1][:] = KV.encode(1.0)
    c.pools[1][t, 12345 % 64] = KV.encode(-1.0)
    c.scales[1][:] = 1.0
    c.set_q(q)
    c.check(*c.run())


def test_scales_far_apart():
    """Pages of one row whose scales differ by 2^40 and more, a page of zeros
    at the smallest scale, queries from 1e-30 to 1e30."""
    c = Case([160, 160, 160], 16, 8, 2, 64, 11)
    for i in range(2):
        c.scales[i][:] = 2.0 ** c.r.integers(-30, 20, c.scales[i].shape)
    c.scales[0][:] = 2.0 ** -9
    p = c.table[0, 3]
    c.pools[1][p], c.scales[1][p] = 0, 2.0 ** -120
    c.check(*c.run())
    c = Case([160, 160], 16, 8, 2, 64, 12)
    q = c.r.normal(size=(2, 8, 64))
    q[0] *= 1e30
    c.scales[0][c.table[0]] = 2.0 ** -108
    q[1] *= 1e-30
    c.scales[0][c.table[1]] = 2.0 ** 92
    c.set_q(q)
    c.check(*c.run())
    q[0] *= 0
    c.set_q(q)
    c.check(*c.run())


def test_no_rows_and_a_workspace_that_is_too_small():
    c = Case([39000], 64, 32, 4, 128, 21)
    cache = c.cache()
    empty = [t[:0].contiguous() for t in cache[4:]]
    assert dsa.attn_kv8(c.Qt[:0], *cache[:4], *empty, c.scale).shape == (0, 32, 128)
    idx = torch.zeros((0, 5), dtype=torch.int32, device="cuda")
    assert dsa.sparse_attn_kv8(c.Qt[:0], *cache[:4], *empty, idx, c.scale).shape == (0, 32, 128)
    with pytest.raises(dsa.DSAError, match="workspace"):
        dsa.attn_kv8(c.Qt, *cache, c.scale, workspace=torch.empty(64, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        dsa.attn_kv8(c.Qt.transpose(0, 1).expand(32, 2, 128).transpose(0, 1), *cache, c.scale)
    with pytest.raises(ValueError, match="idx"):
        dsa.sparse_attn_kv8(c.Qt, *cache, None, c.scale)
    with pytest.raises(ValueError, match="stream"):
        dsa.attn_kv8(c.Qt, *cache, c.scale, stream="current")
    assert dsa.attn_kv8(c.Qt, *cache, c.scale, stream=0).shape == (1, 32, 128)
    torch.cuda.synchronize()


def test_nan_and_infinity_stay_in_their_rows():
    c = Case([100, 100, 100], 16, 8, 2, 64, 13)
    c.pools[1][c.table[1, 2], 3, 0, 7] = 127
    q = c.Q.copy()
    q[2, 5, 0] = np.inf
    c.set_q(q)
    O, lse = c.run()
    bad = torch.isnan(O).cpu().numpy()
    assert not bad[0].any() and bad[1, :4, 7].all() and bad[1].sum() == 4
    assert bad[2, 5].all() and bad[2].sum() == 64
    idx = np.tile(np.arange(100, dtype=np.int32), (3, 1))
    idx[1, 35] = -1  # the NaN's key is masked
    O, _ = c.run(idx)
    assert not torch.isnan(O[:2]).any()


def test_keys_outside_the_sequence_are_left_out():
    c = Case([50, 20], 16, 8, 2, 64, 14)
    idx = c.select(24, holes=False)
    good = idx.copy()
    idx[0, 5], idx[1, 7], idx[1, 9] = 50, 1 << 30, -7
    err = dsa.error_word()
    got = c.run(idx, err=err)
    assert dsa.device_error(err=err) == dsa.DEVERR_INDEX
    c.check(*got, idx)
    c.lens = [50, 500]  # longer than the table and past its entries
    got = c.run(err=err)
    assert dsa.device_error(err=err) == dsa.DEVERR_INDEX
    ref = KV.attention(c.Q[1:], *c.pools, *c.scales, c.table, [1], [np.arange(32)], c.scale)
    assert dsa.device_error() == dsa.DEVERR_NONE
    c.table[0, 1] = 99
    c.run(good, err=err)
    assert dsa.device_error(err=err) == dsa.DEVERR_INDEX
    assert ref[0].shape == (1, 8, 64)


def test_row_offsets_past_the_rows_are_recorded():
    c = Case([50, 50, 50], 16, 8, 2, 64, 15, rows=[2, 2, 2])
    for off in ([0, 2, 4, 90], [0, 1 << 30, 2, 6]):
        c.row_off = np.array(off)
        err = dsa.error_word()
        c.run(err=err)
        assert dsa.device_error(err=err) == dsa.DEVERR_INDEX, off


def test_offsets_beyond_32_bits():
    """A pool of 4.4 GB per tensor: the sequence's pages lie on both sides of
    2^32 bytes."""
    page, Hkv, d = 128, 64, 128
    pages = (1 << 32) // (page * Hkv * d) + 40
    r = np.random.default_rng(16)
    k8 = torch.zeros((pages, page, Hkv, d), dtype=torch.uint8, device="cuda")
    v8 = torch.zeros((pages, page, Hkv, d), dtype=torch.uint8, device="cuda")
    use = [pages - 1, 3, pages - 25]
    k, v = (KV.encode(r.normal(size=(3, page, Hkv, d)) * 64) for _ in "kv")
    for i, p in enumerate(use):
        k8[p], v8[p] = dev(k[i]), dev(v[i])
    sc = torch.full((pages, Hkv), 2.0 ** -6, device="cuda")
    Q, Qt = bf16(r.normal(size=(1, 64, d)))
    lse = torch.empty((1, 64), device="cuda")
    O = dsa.attn_kv8(Qt, k8, v8, sc, sc, dev(np.array([use], np.int32)),
                     dev(np.array([300], np.int32)), d ** -0.5, lse=lse)
    ref, rl, mag, _, _ = KV.attention(Q, k, v, np.full((3, Hkv), 2.0 ** -6),
                                      np.full((3, Hkv), 2.0 ** -6), np.array([[0, 1, 2]]), [0],
                                      [np.arange(300)], d ** -0.5)
    idx = dev(np.arange(300, dtype=np.int32)[None])
    S = dsa.sparse_attn_kv8(Qt, k8, v8, sc, sc, dev(np.array([use], np.int32)),
                            dev(np.array([300], np.int32)), idx, d ** -0.5)
    for got in (O, S):
        err = np.abs(got.double().cpu().numpy() - ref)
        assert np.all(err <= mag * 2.0 ** -10 + np.abs(ref) * 2.0 ** -8)
    assert np.abs(lse.double().cpu().numpy() - rl).max() <= 1e-4


def test_another_stream_and_two_captured_graphs():
    """Two graphs, each with its own workspace, replayed on two streams."""
    c = Case([5000, 39000], 64, 32, 4, 128, 17)
    cache = c.cache()
    want = dsa.attn_kv8(c.Qt, *cache, c.scale)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dsa.attn_kv8(c.Qt, *cache, c.scale, stream=s)
    also = dsa.attn_kv8(c.Qt, *cache, c.scale, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(want, got) and torch.equal(want, also)
    n = dsa.attn_kv8_workspace_size(2, c.table.shape[1] * 64, 32, 4, 128)
    assert n > 0
    graphs, outs, qs = [], [], []
    for i in range(2):
        q = c.Qt * (i + 1)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = dsa.attn_kv8(q, *cache, c.scale, workspace=ws)
        graphs.append((g, ws))
        outs.append(o)
        qs.append(q)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for q, o in zip(qs, outs):
        assert torch.equal(o, dsa.attn_kv8(q, *cache, c.scale))


def test_a_serving_step_from_projection_to_output():
    """Rotary positions, the indexer's inputs, append, select and attend: two
    prompts (one in two chunks), then single tokens for both."""
    import oracle
    import oracle.rope as OR
    Hq, Hkv, d, HI, dI, page, kk = 32, 4, 128, 64, 128, 64, 64
    r = np.random.default_rng(18)
    f, m = dsa.rope_freqs(d, 1e6)
    fi, _ = dsa.rope_freqs(64, 1e6)
    P = 12
    k8, v8 = (torch.zeros((P, page, Hkv, d), dtype=torch.float8_e4m3fn, device="cuda")
              for _ in "kv")
    ks, vs = torch.zeros((P, Hkv), device="cuda"), torch.zeros((P, Hkv), device="cuda")
    table = np.array([[7, 2, 9, 0], [1, 11, 4, 3]], np.int32)
    codes = [np.zeros((P, page, Hkv, d), np.uint8) for _ in "kv"]
    scales = [np.zeros((P, Hkv)) for _ in "kv"]
    kI = [torch.zeros((0, dI), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    lens = [0, 0]
    for new in ([100, 30], [61, 0], [1, 1], [1, 1]):
        T = sum(new)
        off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        pos = dev(np.concatenate([np.arange(n, n + j) for n, j in zip(lens, new)]))
        x = torch.from_numpy(r.normal(size=(T, (Hq + 2 * Hkv) * d)).astype(np.float32)).bfloat16()
        x = x.cuda()
        q0 = x[:, :Hq * d].unflatten(1, (Hq, d))
        k0 = x[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
        V = x[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d))
        Q, K = dsa.rope(q0, k0, pos, f, m)
        w64 = OR.turns_to_frequencies(f.cpu().numpy())
        want = OR.rope(q0.double().cpu().numpy(), pos.cpu().numpy(), w64, m)
        assert np.abs(Q.double().cpu().numpy() - want).max() <= 2.0 ** -8 * np.abs(want).max()
        xi = torch.from_numpy(r.normal(size=(T, HI + 1, dI)).astype(np.float32)).bfloat16().cuda()
        qI, kn = dsa.rope(xi[:, :HI], xi[:, HI:], pos, fi, out_dtype=torch.float8_e4m3fn)
        wI = torch.rand((T, HI), device="cuda")
        dsa.kv8_append(K, V, k8, v8, ks, vs, dev(table), dev(np.array(lens, np.int32)), dev(off))
        for t, cc, ss in ((K, codes[0], scales[0]), (V, codes[1], scales[1])):
            KV.append(t.double().cpu().numpy(), cc, ss, table, lens, off)
        for b in range(2):
            kI[b] = torch.cat([kI[b].view(torch.uint8), kn[off[b]:off[b + 1], 0].view(torch.uint8)]
                              ).view(torch.float8_e4m3fn)
            lens[b] += new[b]
        assert np.array_equal(k8.view(torch.uint8).cpu().numpy(), codes[0])
        assert np.array_equal(v8.view(torch.uint8).cpu().numpy(), codes[1])
        if max(new) == 1:
            coff = dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int64))
            packed = torch.cat([t.view(torch.uint8) for t in kI]).view(torch.float8_e4m3fn)
            _, idx = dsa.decode_select_shard(qI, wI, packed, coff, kk)
            ro = None
        else:
            idx = torch.cat([dsa.index_topk_rows(qI[off[b]:off[b + 1]].contiguous(), kI[b],
                                                 wI[off[b]:off[b + 1]].contiguous(),
                                                 lens[b] - new[b], kk)
                             for b in range(2) if new[b]])
            ro = dev(off)
        O = dsa.sparse_attn_kv8(Q, k8, v8, ks, vs, dev(table), dev(np.array(lens, np.int32)), idx,
                                d ** -0.5, row_off=ro)
        assert dsa.device_error() == dsa.DEVERR_NONE
        seq = np.repeat([0, 1], new)
        keys = [row[row >= 0] for row in idx.cpu().numpy()]
        assert all(len(s) == min(kk, int(p) + 1) for s, p in zip(keys, pos.cpu()))
        ref, _, mag, big, _ = KV.attention(Q.double().cpu().numpy(), *codes, *scales, table, seq,
                                           keys, d ** -0.5)
        err = np.abs(O.double().cpu().numpy() - ref)
        tol = mag * (np.expm1(2.0 ** -18 * big) + 2.0 ** -10)[..., None]
        assert np.all(err <= tol + (np.abs(ref) + tol) * 2.0 ** -8)
