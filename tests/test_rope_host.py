"""Rotary positions without a GPU: the oracle's pins, the frequency table of
the library against the oracle's formulas, and the calls' refusals."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.rope as OR
import sparse_long_context_02_b200 as dsa
from sparse_long_context_02_b200 import build as dsa_build

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = 0x10000  # aligned, never dereferenced: every call below fails validation


@pytest.fixture(scope="module")
def L():
    dsa_build.build()
    return dsa.lib()


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_scores_depend_on_the_distance_only(interleaved):
    rng = np.random.default_rng(1)
    w, m = OR.frequencies(16)
    q, k = rng.normal(size=(1, 1, 20)), rng.normal(size=(1, 1, 20))

    def score(p, s):
        return float((OR.rope(q, [p], w, m, 2, interleaved) *
                      OR.rope(k, [s], w, m, 2, interleaved)).sum())

    assert abs(score(9, 4) - score(105, 100)) < 1e-12
    assert abs(score(9, 4) - score(9, 5)) > 1e-3
    assert np.array_equal(OR.rope(q, [0], w, m, 2, interleaved), q)
    y = OR.rope(q, [3], w, m, 2, interleaved)
    assert np.array_equal(y[..., :2], q[..., :2]) and np.array_equal(y[..., 18:], q[..., 18:])


def test_oracle_pairs_and_angle():
    w = np.array([np.pi / 2, np.pi])
    x = np.arange(1.0, 5.0).reshape(1, 1, 4)
    # pairs (1, 3) by a quarter turn, (2, 4) by a half
    assert np.allclose(OR.rope(x, [1], w), [[[-3, -2, 1, -4]]], atol=1e-12)
    # pairs (1, 2) and (3, 4)
    assert np.allclose(OR.rope(x, [1], w, interleaved=True), [[[-2, 1, -3, -4]]], atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_gradient_against_differences(interleaved):
    rng = np.random.default_rng(2)
    w, m = OR.frequencies(8, 100.0, "yarn", 4.0, 64.0, 8.0, 1.0)
    x, dy = rng.normal(size=(3, 2, 10)), rng.normal(size=(3, 2, 10))
    pos = [0, 5, 77]
    g = OR.rope(dy, pos, w, m, 1, interleaved, inverse=True)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1e-5
        num = ((OR.rope(x + e, pos, w, m, 1, interleaved) -
                OR.rope(x - e, pos, w, m, 1, interleaved)) * dy).sum() / 2e-5
        # the map is linear: only the difference's own rounding is left
        assert abs(num - g[i]) < 1e-9


@pytest.mark.parametrize("args", [dict(rot=128), dict(rot=2), dict(rot=64, base=1e6),
                                  dict(rot=64, scaling="linear", factor=8.0),
                                  dict(rot=128, scaling="ntk", factor=4.0),
                                  dict(rot=4, scaling="ntk", factor=1.0),
                                  dict(rot=128, base=1e6, scaling="yarn", factor=8.0,
                                       orig_len=32768.0),
                                  dict(rot=96, scaling="yarn", factor=2.5, orig_len=100.0,
                                       beta_fast=16.0, beta_slow=0.0)])
def test_frequency_table(L, args):
    f, m = dsa.rope_freqs(device="cpu", **args)
    w, m_ref = OR.frequencies(**args)
    assert f.dtype == torch.int64 and f.numel() == args["rot"] // 2
    got = OR.turns_to_frequencies(f.numpy())
    # a double's pow, a few roundings, and a unit of 2^-64 turns
    assert np.all(np.abs(got - w) <= 1e-14 * w + 4e-19)
    assert abs(m - m_ref) <= 2.0 ** -24 * m_ref


def test_frequency_table_refusals(L):
    for bad in (dict(rot=0), dict(rot=7), dict(rot=2048), dict(rot=64, base=1.0),
                dict(rot=64, base=float("nan")), dict(rot=64, scaling="linear", factor=0.5),
                dict(rot=64, scaling="linear", factor=float("inf")),
                dict(rot=2, scaling="ntk", factor=2.0),
                dict(rot=64, scaling="yarn", factor=2.0),
                dict(rot=64, scaling="yarn", factor=2.0, orig_len=10.0, beta_fast=1.0)):
        with pytest.raises(dsa.DSAError) as e:
            dsa.rope_freqs(device="cpu", **bad)
        assert e.value.status == INVALID
    with pytest.raises(ValueError, match="scaling"):
        dsa.rope_freqs(64, scaling="cubic", device="cpu")
    buf = (ctypes.c_uint64 * 32)()
    m = ctypes.c_float()
    assert L.dsa_rope_freqs(64, 1e4, 9, 1.0, 0.0, 0.0, 0.0, buf, ctypes.byref(m)) == UNSUPPORTED
    assert L.dsa_rope_freqs(64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, buf, None) == INVALID


# q, k, positions, freqs, L, Hq, Hk, d, offset, rot, interleaved, rot_scale, out_scale, in, out,
# strides (q, k, q_out, k_out), q_out, k_out, err, stream
GOOD = [FAKE] * 4 + [8, 4, 2, 64, 0, 64, 0, 1.0, 1.0, 0, 0, 256, 128, 256, 128, FAKE, FAKE, None,
                     None]


@pytest.mark.parametrize("at,value,status", [
    (0, None, INVALID), (0, FAKE + 1, INVALID), (1, None, INVALID), (2, None, INVALID),
    (2, FAKE + 4, INVALID), (3, FAKE + 4, INVALID), (4, -1, INVALID), (4, 1 << 31, INVALID),
    (5, 0, INVALID), (5, 1100, INVALID), (6, -1, INVALID), (7, 63, INVALID), (7, 2048, INVALID),
    (8, 1, INVALID), (8, 2, INVALID), (8, -2, INVALID), (9, 0, INVALID), (9, 31, INVALID),
    (9, 66, INVALID), (11, float("inf"), INVALID), (12, float("nan"), INVALID),
    (13, 2, UNSUPPORTED), (13, 7, UNSUPPORTED), (14, 3, UNSUPPORTED), (15, 255, INVALID),
    (16, 127, INVALID), (17, -256, INVALID), (18, 0, INVALID), (19, None, INVALID),
    (20, FAKE + 1, INVALID), (21, FAKE + 2, INVALID)])
def test_rope_refusals(L, at, value, status):
    a = list(GOOD)
    a[at] = value
    assert L.dsa_rope(*a) == status
    assert b"dsa_rope" in L.dsa_last_error()
    b = a[:12] + a[13:]  # no out_scale
    if at != 12:
        assert L.dsa_rope_backward(*b) == status
        assert b"dsa_rope_backward" in L.dsa_last_error()


def test_rope_empty_and_gradient_type(L):
    a = list(GOOD)
    a[4] = 0
    assert L.dsa_rope(*a) == OK
    b = GOOD[:12] + GOOD[13:]
    b[13] = 2  # e4m3 gradients
    assert L.dsa_rope_backward(*b) == UNSUPPORTED


def test_binding_checks():
    q = torch.zeros((2, 4, 8))
    pos, f = torch.zeros(2, dtype=torch.int64), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.rope(q, None, pos, f)
    with pytest.raises(ValueError, match="positions"):
        dsa.rope(q, None, pos.int(), f)
    with pytest.raises(ValueError, match="positions"):
        dsa.rope(q, None, pos[:1], f)
    with pytest.raises(ValueError, match="freqs"):
        dsa.rope(q, None, pos, f.float())
    with pytest.raises(ValueError, match="dtype"):
        dsa.rope(q.half(), None, pos, f)
    with pytest.raises(ValueError, match="out_dtype"):
        dsa.rope(q, None, pos, f, out_dtype=torch.float16)
