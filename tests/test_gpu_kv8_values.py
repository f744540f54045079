"""The attention over the paged 8-bit cache on values that its parity tests do
not meet, against the float64 oracle (oracle/kv8.py)."""
import numpy as np
import pytest
import torch

import oracle.kv8 as KV
import sparse_long_context_02_b200 as dsa
from test_gpu_kv8_append import Cache, bf16, dev
from test_gpu_kv8_attn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,k", [([1], 0), ([1, 0, 40], 0), ([300, 2], 64), ([40000], 0),
                                    ([40000, 7], 2048), ([60] * 200, 0)])
@pytest.mark.parametrize("q", [-np.inf, np.inf, np.nan])
def test_a_query_with_an_infinity_gives_nan(lens, k, q):
    """Scores that are all -inf (a query element of -inf over positive key
    elements) have no softmax: NaN, as +inf and NaN give, not the zeros of a
    row without keys.  The other heads keep their values."""
    c = Case(lens, 16, 8, 2, 64, 31)
    for x in c.pools[:1]:
        x[..., 0] = np.where((x[..., 0] & 127) == 127, x[..., 0], 0x38)  # 1.0
    clean = c.Q.copy()
    bad = clean.copy()
    bad[:, 3, 0] = q
    c.set_q(bad)
    idx = c.select(k, holes=False) if k else None
    O, lse = c.run(idx)
    c.set_q(clean)
    want, want_lse = c.run(idx)
    seen = torch.tensor([len(s) > 0 for s in c.keys(idx)], device="cuda")
    assert torch.isnan(O[seen, 3]).all() and torch.isnan(lse[seen, 3]).all()
    assert torch.all(O[~seen] == 0) and torch.all(lse[~seen] == -torch.inf)
    rest = [h for h in range(8) if h != 3]
    assert torch.equal(O[:, rest], want[:, rest]) and torch.equal(lse[:, rest], want_lse[:, rest])
    assert dsa.device_error() == dsa.DEVERR_NONE


def _scales(r, shape, lo, hi):
    """Any positive fp32 number: none is a power of two."""
    return (2.0 ** r.uniform(lo, hi, shape)).astype(np.float32).astype(np.float64)


@pytest.mark.parametrize("Hq,Hkv,d", [(32, 4, 128), (8, 2, 64), (5, 1, 64)])
@pytest.mark.parametrize("lens", [[1, 37, 300, 64], [20000, 5], [50] * 160])
def test_attention_under_any_scales(Hq, Hkv, d, lens):
    """A cache that another writer filled.  On top of the parity tests' bound:
    log2 of V's scale, here up to 12 in magnitude, is off by two units in the
    last place, 2^-19, and its sum with the score (together below 2^7) by half a
    unit, 2^-18; times ln 2 that is less than 2^-17 of each weight.  K's scale
    enters by the fp32 products that the bound counts."""
    c = Case(lens, 16, Hq, Hkv, d, 41)
    c.scales = [_scales(c.r, s.shape, *e) for s, e in zip(c.scales, ((-13, -7), (-12, -4)))]
    for idx in (None, c.select(48)):
        O, lse = c.run(idx)
        keys = c.keys(idx)
        ref, rl, mag, big, top = KV.attention(c.Q, *c.pools, *c.scales, c.table, c.seq, keys,
                                              c.scale)
        assert big.max() * 1.45 < 2.0 ** 6  # a score in log2 units
        E = 2.0 ** -19 * big
        n = np.array([len(s) for s in keys])[:, None]
        tol = (mag * (np.expm1(2 * E) + 2.0 ** -11 + 2.0 ** -18 + 2.0 ** -17)[..., None] +
               (n * 2.0 ** -31 * top)[..., None])
        tol = tol + (np.abs(ref) + tol) * 2.0 ** -8
        assert np.all(np.abs(O.double().cpu().numpy() - ref) <= tol)
        assert np.all(np.abs(lse.double().cpu().numpy() - rl) <=
                      E + 2.0 ** -18 + np.abs(rl) * 2.0 ** -22)
    assert dsa.device_error() == dsa.DEVERR_NONE


@pytest.mark.parametrize("T", [2, 160, 600])
def test_scales_that_are_aligned_to_four_bytes_only(T):
    """A group's four scales are one vector load where alignment allows."""
    c = Case([70 + t % 5 for t in range(T)], 16, 32, 4, 128, 42)
    cache = list(c.cache())
    idx = dev(c.select(24, holes=False))

    def run(cache):
        lse = torch.empty((T, 32), device="cuda")
        return [dsa.attn_kv8(c.Qt, *cache, c.scale, lse=lse),
                dsa.sparse_attn_kv8(c.Qt, *cache, idx, c.scale), lse]

    want = run(cache)
    for i in (2, 3):
        odd = torch.empty(cache[i].numel() + 1, device="cuda")[1:].view_as(cache[i])
        odd.copy_(cache[i])
        assert odd.data_ptr() % 16 == 4
        cache[i] = odd
        assert all(torch.equal(a, b) for a, b in zip(want, run(cache)))


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("one", [False, True])
def test_append_to_pages_under_any_scale(page, one):
    """Scales that another writer left.  Small new rows keep them: codes are
    x / scale in fp32, rounded to e4m3 (both correctly), as numpy's fp32 says.
    Larger rows outgrow them: the new scale is a power of two, and the older
    codes are rounded again from value * (old / new), two fp32 roundings: the
    code of a number within 2^-22 of the exact one."""
    r = np.random.default_rng(page + one)
    Hkv, d, B = 2, 64, 12
    lens = [int(n) for n in r.integers(1, page - 3, B)]
    new = [1] * B if one else [int(n) for n in r.integers(1, 4, B)]
    off = np.concatenate([[0], np.cumsum(new)])
    c = Cache(B, page, Hkv, d, np.arange(B)[:, None])
    c.scales = [_scales(r, s.shape, -3, 3) for s in c.scales]
    c.ds = [dev(s.astype(np.float32)) for s in c.scales]
    big = 2.0 ** np.where(np.arange(B) % 2, 9, 2)  # every second sequence outgrows its scale
    xs = [bf16(np.clip(r.normal(size=(off[-1], Hkv, d)), -3, 3) * np.repeat(big, new)[:, None, None])
          for _ in "kv"]
    dsa.kv8_append(xs[0][1], xs[1][1], *c.dc, *c.ds, c.dt, dev(np.asarray(lens, np.int32)),
                   None if one else dev(off.astype(np.int32)))
    assert dsa.device_error() == dsa.DEVERR_NONE
    kept = grown = 0
    for i in range(2):
        codes, scales = c.dc[i].cpu().numpy(), c.ds[i].double().cpu().numpy()
        for b in range(B):
            n, m = lens[b], new[b]
            for h in range(Hkv):
                rows = xs[i][0][off[b]:off[b + 1], h]
                was = c.scales[i][b, h]
                now = max(was, KV.need(rows))
                assert scales[b, h] == now
                want = KV.encode(rows.astype(np.float32) / np.float32(now))
                assert np.array_equal(codes[b, n:n + m, h], want)
                old = c.codes[i][b, :n, h]
                if now == was:
                    kept += 1
                    assert np.array_equal(codes[b, :n, h], old)
                else:
                    grown += 1
                    exact = KV.decode(old) * was / now
                    a, z = KV.encode(exact * (1 - 2.0 ** -22)), KV.encode(exact * (1 + 2.0 ** -22))
                    got = codes[b, :n, h]
                    assert np.all((got == a) | (got == z))
                assert np.array_equal(codes[b, n + m:, h], c.codes[i][b, n + m:, h])
    assert kept > 4 and grown > 4
