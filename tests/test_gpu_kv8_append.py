"""GPU parity of appending to the paged 8-bit cache (dsa_kv8_append) against
the oracle (oracle/kv8.py).  Scales are powers of two, quotients by them exact
and every code one rounding: codes and scales are compared bit for bit."""
import numpy as np
import pytest
import torch

import oracle.kv8 as KV
import sparse_long_context_02_b200 as dsa

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(x):
    """float64 values rounded to bf16, as (values, tensor)."""
    t = torch.from_numpy(x.astype(np.float32)).bfloat16()
    return t.double().numpy(), t.cuda()


class Cache:
    """A pool of random codes (what earlier owners left) and its mirror."""

    def __init__(self, pages, page, Hkv, d, table, seed=0):
        r = np.random.default_rng(seed)
        self.codes = [r.integers(0, 256, (pages, page, Hkv, d), dtype=np.uint8) for _ in "kv"]
        for c in self.codes:
            c[(c & 127) == 127] = 5
        self.scales = [2.0 ** r.integers(-9, 2, (pages, Hkv)) for _ in "kv"]
        self.table = np.asarray(table, np.int32)
        self.dc = [dev(c) for c in self.codes]
        self.ds = [dev(s.astype(np.float32)) for s in self.scales]
        self.dt = dev(self.table)

    def append(self, K, V, lens, off=None, **kw):
        (Kv, Kt), (Vv, Vt) = bf16(K), bf16(V)
        o = np.arange(len(lens) + 1) if off is None else off
        for i, x in enumerate((Kv, Vv)):
            KV.append(x, self.codes[i], self.scales[i], self.table, lens, o)
        dsa.kv8_append(Kt, Vt, *self.dc, *self.ds, self.dt, dev(np.asarray(lens, np.int32)),
                       None if off is None else dev(np.asarray(off, np.int32)), **kw)
        self.check()

    def check(self):
        for i in range(2):
            assert np.array_equal(self.ds[i].cpu().numpy(), self.scales[i].astype(np.float32))
            got = self.dc[i].cpu().numpy()
            bad = np.argwhere(got != self.codes[i])
            assert len(bad) == 0, (len(bad), bad[:4])


def _tables(lens, page, seed=0, extra=0):
    need = [-(-max(n, 0) // page) + extra for n in lens]
    order = np.random.default_rng(seed).permutation(sum(need) + 3)
    M, at = max(max(need), 1), 0
    t = np.full((len(lens), M), -1, np.int32)
    for b, m in enumerate(need):
        t[b, :m] = order[at:at + m]
        at += m
    return t, sum(need) + 3


def _rows(r, T, Hkv, d):
    return r.normal(size=(T, Hkv, d)) * 2.0 ** r.integers(-3, 12, (T, 1, 1))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hkv,d", [(4, 128), (2, 64), (1, 128), (3, 64), (64, 64)])
def test_one_token_each(page, Hkv, d):
    r = np.random.default_rng(page + d)
    lens = [0, 1, page - 1, page, page + 1, 3 * page - 1, -1, 2 * page + 5]
    table, pages = _tables([n + 1 for n in lens], page)
    c = Cache(pages, page, Hkv, d, table)
    for step in range(3):
        c.append(_rows(r, len(lens), Hkv, d), _rows(r, len(lens), Hkv, d), lens)
        lens = [n + 1 if 0 <= n and (n + 1) // page < -(-(n + 1) // page) else n for n in lens]
    assert dsa.device_error() == dsa.DEVERR_NONE


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hkv,d", [(4, 128), (2, 64)])
def test_ragged_prompts_and_chunks(page, Hkv, d):
    """Sequences of 0 to many new tokens behind 0 to many old ones; rows
    behind the last sequence; slots and pages of nobody stay as they were."""
    r = np.random.default_rng(page * d)
    lens = [0, 5, page, 0, 2 * page - 1, 17, 3, -1, 1]
    new = [3 * page + 2, 1, page, 0, 2, 2 * page, 0, 7, 4 * page - 1]
    off = np.concatenate([[0], np.cumsum(new)])
    table, pages = _tables([max(n, 0) + m for n, m in zip(lens, new)], page)
    c = Cache(pages, page, Hkv, d, table)
    T = int(off[-1]) + 9
    for _ in range(2):
        c.append(_rows(r, T, Hkv, d), _rows(r, T, Hkv, d), lens, off)
    assert dsa.device_error() == dsa.DEVERR_NONE


def test_many_short_sequences():
    r = np.random.default_rng(3)
    lens, new = r.integers(0, 40, 700), r.integers(0, 4, 700)
    off = np.concatenate([[0], np.cumsum(new)])
    table, pages = _tables([n + m for n, m in zip(lens, new)], 16)
    c = Cache(pages, 16, 2, 64, table)
    c.append(_rows(r, int(off[-1]), 2, 64), _rows(r, int(off[-1]), 2, 64), list(lens), off)
    assert dsa.device_error() == dsa.DEVERR_NONE


def test_special_values():
    """NaN, infinities, the largest and smallest numbers, zeros, ties and
    values next to a scale's border."""
    x = np.zeros((7, 2, 64))
    x[0, 0, :4] = [np.nan, np.inf, -np.inf, 1.0]
    x[0, 1, :3] = [448.0, -448.0, 1.0]
    x[1, 0, :2] = [450.0, 0.0]                 # bf16: the first above 448
    x[1, 1] = 0.0
    x[2, 0, :2] = [3.3e38, 1e-38]
    x[2, 1, :3] = [1e-38, 9e-41, -1e-36]       # below the smallest scale's range
    x[3, :, :8] = [1.0, 17 / 16, 19 / 16, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, -17 / 16, 448.0]
    x[4] = np.nan
    x[5, :, 0] = -0.0
    x[6, :, 0] = 2.0 ** -120 * 448
    lens = [0, 3, 0, 0, 0, 15, 0]
    table, pages = _tables([n + 1 for n in lens], 16)
    c = Cache(pages, 16, 2, 64, table)
    c.append(x, x[::-1], lens)


def test_growing_scale_keeps_the_page():
    """A page that fills token by token, each larger than the last: older
    codes shift into the subnormals and, in the end, to zero."""
    r = np.random.default_rng(4)
    c = Cache(3, 16, 2, 64, [[1]])
    for s in range(16):
        row = r.normal(size=(1, 2, 64)) * 2.0 ** (2 * s)
        c.append(row, row[::-1] * 3, [s])
    assert dsa.device_error() == dsa.DEVERR_NONE


def test_pages_outside_the_pool_are_left_out():
    """A bad table entry, and a sequence longer than its table row: recorded,
    the rest stored."""
    r = np.random.default_rng(5)
    table = np.array([[0, -1, 2], [3, 99, 4], [5, 6, 7]], np.int32)
    c = Cache(8, 16, 2, 64, table)
    err = dsa.error_word()
    off = [0, 48, 80, 130]
    c.append(_rows(r, 130, 2, 64), _rows(r, 130, 2, 64), [0, 16, 0], off, err=err)
    assert dsa.device_error(err=err) == dsa.DEVERR_INDEX
    c.append(_rows(r, 3, 2, 64), _rows(r, 3, 2, 64), [20, 20, 48], err=err)
    assert dsa.device_error(err=err) == dsa.DEVERR_INDEX
    assert dsa.device_error() == dsa.DEVERR_NONE


def test_offsets_that_run_backwards_are_left_out():
    r = np.random.default_rng(6)
    c = Cache(8, 16, 2, 64, [[0], [1], [2]])
    x = bf16(_rows(r, 4, 2, 64))[1]
    err = dsa.error_word()
    for off in ([0, 3, 1, 4], [0, 2, 3, 9], [-5, 1, 2, 4], [0, 1 << 30, 2, 4]):
        dsa.kv8_append(x, x, *c.dc, *c.ds, c.dt, dev(np.zeros(3, np.int32)),
                       dev(np.array(off, np.int32)), err=err)
        assert dsa.device_error(err=err) == dsa.DEVERR_INDEX


def test_rows_of_one_projection():
    """K and V as parts of wider rows: token strides beyond Hkv x d."""
    r = np.random.default_rng(7)
    Hkv, d, T = 4, 128, 70
    wide, t = bf16(_rows(r, T, 3 * Hkv, d))
    table, pages = _tables([T + 5], 32)
    c = Cache(pages, 32, Hkv, d, table)
    for i in range(2):
        KV.append(wide[:, (i + 1) * Hkv:(i + 2) * Hkv], c.codes[i], c.scales[i], c.table, [5],
                  [0, T])
    dsa.kv8_append(t[:, Hkv:2 * Hkv], t[:, 2 * Hkv:], *c.dc, *c.ds, c.dt,
                   dev(np.array([5], np.int32)), dev(np.array([0, T], np.int32)))
    c.check()


def test_offsets_beyond_32_bits():
    """A pool of 4.4 GB per tensor: the last pages lie past 2^32 bytes."""
    page, Hkv, d = 128, 64, 128
    pages = (1 << 32) // (page * Hkv * d) + 40
    r = np.random.default_rng(8)
    k8 = torch.empty((pages, page, Hkv, d), dtype=torch.uint8, device="cuda")
    v8 = torch.empty((pages, page, Hkv, d), dtype=torch.uint8, device="cuda")
    ks = torch.ones((pages, Hkv), device="cuda")
    vs = torch.ones((pages, Hkv), device="cuda")
    table = dev(np.array([[pages - 1], [pages - 30]], np.int32))
    (xv, x) = bf16(_rows(r, 2, Hkv, d))
    dsa.kv8_append(x, x, k8, v8, ks, vs, table, dev(np.zeros(2, np.int32)))
    for b, p in enumerate((pages - 1, pages - 30)):
        for c, s in ((k8, ks), (v8, vs)):
            for h in (0, 63):
                n = KV.need(xv[b, h])
                assert s[p, h].item() == n
                assert np.array_equal(c[p, 0, h].cpu().numpy(), KV.encode(xv[b, h] / n))


def test_another_stream_and_a_captured_graph():
    r = np.random.default_rng(9)
    lens = [3, 40]
    table, pages = _tables([8, 45], 16, extra=1)
    c = Cache(pages, 16, 2, 64, table)
    (xv, x) = bf16(_rows(r, 2, 2, 64))
    dl = dev(np.array(lens, np.int32))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dsa.kv8_append(x, x, *c.dc, *c.ds, c.dt, dl, stream=s)
    s.synchronize()
    for i in range(2):
        KV.append(xv, c.codes[i], c.scales[i], c.table, lens, [0, 1, 2])
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.kv8_append(x, x, *c.dc, *c.ds, c.dt, dl)
        dl += 1
    c.check()
    dl += 1
    lens = [n + 1 for n in lens]
    for _ in range(3):
        new, t = bf16(_rows(r, 2, 2, 64))
        x.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            KV.append(new, c.codes[i], c.scales[i], c.table, lens, [0, 1, 2])
        lens = [n + 1 for n in lens]
        c.check()


def test_no_rows():
    c = Cache(3, 16, 2, 64, [[1]])
    x = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    dsa.kv8_append(x, x, *c.dc, *c.ds, c.dt, dev(np.array([3], np.int32)), off)
    c.check()
