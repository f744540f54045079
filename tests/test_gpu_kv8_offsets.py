"""Offsets of sequences that do not ascend, lengths and tables that lead
outside the cache: what the paged 8-bit cache's calls record of them, and what
they still compute."""
import numpy as np
import pytest
import torch

import oracle.kv8 as KV
import sparse_long_context_02_b200 as dsa
from test_gpu_kv8_append import Cache, _rows, bf16, dev
from test_gpu_kv8_attn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("off", [[0, 100, 5, 120], [0, 90, 100, 60, 120], [0, 120, 121], [-1, 120],
                                 [0] + [7, 6] * 600 + [120]])
def test_append_records_offsets_that_do_not_ascend(off):
    """Also where no unit of work comes to lie on the pair that runs backwards."""
    r = np.random.default_rng(1)
    B = len(off) - 1
    c = Cache(8 * B, 16, 2, 64, np.arange(8 * B).reshape(B, 8))
    x = bf16(_rows(r, 120, 2, 64))[1]
    err = dsa.error_word()
    dsa.kv8_append(x, x, *c.dc, *c.ds, c.dt, dev(np.zeros(B, np.int32)),
                   dev(np.array(off, np.int32)), err=err)
    assert dsa.device_error(err=err) == dsa.DEVERR_INDEX
    assert dsa.device_error() == dsa.DEVERR_NONE


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("T,off", [(20, [0, 10, 5, 20]), (20, [0, 20, 21]), (600, [0, 300, 200, 600]),
                                   (40, [0] + [3, 2] * 600 + [40])])
def test_attention_records_offsets_that_do_not_ascend(T, off, sparse):
    B = len(off) - 1
    c = Case([40] * B, 16, 8, 2, 64, 2)
    c.row_off = np.array(off)
    c.set_q(c.r.normal(size=(T, 8, 64)))
    err = dsa.error_word()
    c.run(np.zeros((T, 4), np.int32) if sparse else None, err=err)
    assert dsa.device_error(err=err) == dsa.DEVERR_INDEX
    assert dsa.device_error() == dsa.DEVERR_NONE


@pytest.mark.parametrize("off,good", [([0, 3, 1, 4], [0, 2]), ([0, 2, 3, 9], [0, 1]),
                                      ([-5, 1, 2, 4], [1, 2])])
def test_append_leaves_refused_sequences_alone(off, good):
    """The others' rows are stored; the refused ones' pages, and all that
    belongs to nobody, keep every bit."""
    r = np.random.default_rng(3)
    c = Cache(8, 16, 2, 64, [[0], [1], [2]])
    xv, x = bf16(_rows(r, 4, 2, 64))
    lens = [2, 5, 0]
    for b in good:
        for i in range(2):
            part = [max(off[b], 0), max(off[b + 1], 0)]
            KV.append(xv, c.codes[i], c.scales[i], c.table[b:b + 1], lens[b:b + 1], part)
    err = dsa.error_word()
    dsa.kv8_append(x, x, *c.dc, *c.ds, c.dt, dev(np.array(lens, np.int32)),
                   dev(np.array(off, np.int32)), err=err)
    assert dsa.device_error(err=err) == dsa.DEVERR_INDEX
    c.check()


def _against(c, O, lse, rows, seq, keys):
    """Rows of O and lse against the oracle over `keys`, by the bound of
    Case.check."""
    ref, rl, mag, big, top = KV.attention(c.Q[rows], *c.pools, *c.scales, c.table, seq, keys, c.scale)
    O, lse = O.double().cpu().numpy()[rows], lse.double().cpu().numpy()[rows]
    E = 2.0 ** -19 * big
    n = np.array([len(s) for s in keys])[:, None]
    tol = (mag * (np.expm1(2 * E) + 2.0 ** -11 + 2.0 ** -18)[..., None] +
           (n * 2.0 ** -31 * top)[..., None])
    tol = tol + (np.abs(ref) + tol) * 2.0 ** -8
    assert np.all(np.abs(O - ref) <= tol)
    some = n[:, 0] > 0
    assert np.all(np.abs(lse[some] - rl[some]) <=
                  (E + 2.0 ** -18 + np.abs(rl) * 2.0 ** -22)[some])
    assert np.all(O[~some] == 0) and np.all(lse[~some] == -np.inf)


def test_attention_without_the_keys_that_cannot_be_reached():
    """A sequence longer than its table row, whose last entries are no pages:
    the keys that remain; a table entry outside the pool: all keys but its own.
    The neighbour row is as ever."""
    c = Case([50, 20], 16, 8, 2, 64, 14)
    for x in c.pools:  # the clamped sequence reaches slots that lay past it
        p = c.table[1, 1]
        x[p][(x[p] & 127) == 127] = 0x30
    c.lens = [50, 500]
    err = dsa.error_word()
    O, lse = c.run(err=err)
    assert dsa.device_error(err=err) == dsa.DEVERR_INDEX
    _against(c, O, lse, [0, 1], [0, 1], [np.arange(50), np.arange(32)])
    c.lens = [50, 20]
    idx = c.select(24, holes=False)
    c.table[0, 1] = 99
    O, lse = c.run(idx, err=err)
    assert dsa.device_error(err=err) == dsa.DEVERR_INDEX
    left = [s for s in idx[0] if 0 <= s < 16 or s >= 32]
    assert 0 < len(left) < 24
    _against(c, O, lse, [0, 1], [0, 1], [left, [s for s in idx[1] if s >= 0]])
    O, lse = c.run(err=err)
    assert dsa.device_error(err=err) == dsa.DEVERR_INDEX
    _against(c, O, lse, [0, 1], [0, 1], [np.r_[0:16, 32:50], np.arange(20)])


def test_attention_of_the_rows_that_bad_offsets_leave():
    """Offsets past the rows: the sequence that they cut off has no keys, the
    rows of the others are as ever."""
    c = Case([50, 50, 50], 16, 8, 2, 64, 15, rows=[2, 2, 2])
    c.row_off = np.array([0, 2, 4, 90])
    err = dsa.error_word()
    O, lse = c.run(err=err)
    assert dsa.device_error(err=err) == dsa.DEVERR_INDEX
    _against(c, O, lse, [0, 1, 2, 3, 4, 5], c.seq,
             [np.arange(49), np.arange(50), np.arange(49), np.arange(50), [], []])
