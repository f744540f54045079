"""GPU parity of the rotary positions against the float64 oracle
(oracle/rope.py).

Tolerance.  cos and sin times rot_scale are off by one rounding (2^-24) and what
their series leave (below 2^-24 again): 2^-23 of rot_scale; the two products and
the sum add 3 * 2^-24.  Together below 2^-21 rot_scale (|a| + |b|) for a pair (a,
b), times out_scale with another 2^-24; then one rounding to the output's type."""
import numpy as np
import pytest
import torch

import oracle.rope as OR
import sparse_long_context_02_b200 as dsa

pytestmark = pytest.mark.gpu

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _bound(x, ref, w, m, off, inter, scale, dt):
    x = np.abs(x)
    half = len(w)
    a, b = ((off + 2 * np.arange(half), off + 2 * np.arange(half) + 1) if inter else
            (off + np.arange(half), off + half + np.arange(half)))
    tol = x * 2.0 ** -23
    tol[..., a] = tol[..., b] = (x[..., a] + x[..., b]) * m * 2.0 ** -21
    tol *= abs(scale) * (1 + 2.0 ** -23)
    fin = torch.finfo(dt)
    step = {BF: 2.0 ** -134, F32: 2.0 ** -150, E4: 2.0 ** -10}[dt]
    return tol + np.maximum((np.abs(ref) + tol) * fin.eps / 2, step)


def _check(got, x, pos, f, m, off, inter, scale=1.0, inverse=False):
    w = OR.turns_to_frequencies(f.cpu().numpy())
    x64 = x.double().cpu().numpy()
    ref = OR.rope(x64, pos.cpu().numpy(), w, m, off, inter, inverse, scale)
    err = np.abs(got.float().double().cpu().numpy() - ref)
    tol = _bound(x64, ref, w, m, off, inter, scale, got.dtype)
    assert np.all(err <= tol), (np.max(err / tol), np.argmax(err / tol))


def _x(L, H, d, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((L, H, d), generator=g, device="cuda").to(dt)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("L,Hq,Hk,d,off,rot", [
    (1, 32, 4, 128, 0, 128), (5, 8, 2, 64, 0, 64), (700, 32, 4, 128, 64, 64),
    (301, 3, 0, 128, 16, 32), (2, 1, 1, 2, 0, 2), (33, 5, 7, 70, 6, 38), (9, 64, 1, 128, 0, 64),
    (4, 1, 2, 1024, 0, 1024), (3, 1000, 24, 8, 0, 8), (1037, 7, 1, 96, 32, 64),
    (150, 4, 2, 72, 8, 64), (297, 2, 2, 80, 0, 16)])
@pytest.mark.parametrize("tin,tout", [(BF, BF), (F32, F32), (BF, E4), (F32, BF), (BF, F32),
                                      (F32, E4)])
def test_rope(L, Hq, Hk, d, off, rot, inter, tin, tout):
    f, m = dsa.rope_freqs(rot, 1e4)
    q = _x(L, Hq, d, tin, 1)
    k = _x(L, Hk, d, tin, 2) if Hk else None
    pos = torch.randint(0, 1 << 18, (L,), generator=torch.Generator().manual_seed(3)).cuda()
    scale = 0.75 if tout == E4 else 1.0
    qo, ko = dsa.rope(q, k, pos, f, m, scale, off, inter, tout)
    _check(qo, q, pos, f, m, off, inter, scale)
    if Hk:
        _check(ko, k, pos, f, m, off, inter, scale)
    else:
        assert ko is None


@pytest.mark.parametrize("scaling,kw", [("linear", {}), ("ntk", {}),
                                        ("yarn", dict(orig_len=4096.0))])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("tin,tout", [(F32, F32), (F32, BF), (BF, F32), (BF, BF)])
def test_backward(scaling, kw, inter, tin, tout):
    f, m = dsa.rope_freqs(64, 1e6, scaling, 8.0, **kw)
    pos = torch.arange(1000, 1517, device="cuda")
    dq, dk = _x(517, 8, 128, tin, 4), _x(517, 2, 128, tin, 5)
    gq, gk = dsa.rope_backward(dq, dk, pos, f, m, 32, inter, tout)
    _check(gq, dq, pos, f, m, 32, inter, inverse=True)
    _check(gk, dk, pos, f, m, 32, inter, inverse=True)


def test_gradient_against_differences():
    """sum(dy * rope(x)) along one coordinate at a time: the map is linear, so
    a step of 2 loses nothing but fp32 rounding (64 terms below 8 each)."""
    f, m = dsa.rope_freqs(16, 100.0, "yarn", 4.0, orig_len=50.0)
    pos = torch.tensor([3, 1000], device="cuda")
    x, dy = _x(2, 2, 16, F32, 6), _x(2, 2, 16, F32, 7)
    g, _ = dsa.rope_backward(dy, None, pos, f, m)
    for i in np.ndindex(2, 2, 16):
        e = torch.zeros_like(x)
        e[i] = 1.0
        up, _ = dsa.rope(x + e, None, pos, f, m)
        dn, _ = dsa.rope(x - e, None, pos, f, m)
        num = ((up.double() - dn.double()) * dy.double()).sum() / 2
        assert abs(num.item() - g[i].item()) <= 64 * 8 * 2.0 ** -21


def test_far_and_negative_positions():
    """The angle is reduced exactly at any 64-bit position."""
    f, m = dsa.rope_freqs(64, 1e4)
    pos = [0, -1, -262144, (1 << 40) + 12345, (1 << 62) + 7, -(1 << 63), (1 << 63) - 1]
    x = _x(len(pos), 2, 64, F32, 8)
    y, _ = dsa.rope(x, None, torch.tensor(pos, device="cuda"), f, m)
    turns = [[((p * int(v)) % (1 << 64)) / 2.0 ** 64 for v in f.tolist()] for p in pos]
    z = np.exp(2j * np.pi * np.array(turns))[:, None]
    a, b = (t.double().cpu().numpy() for t in x.chunk(2, -1))
    v = (a + 1j * b) * z
    ref = np.concatenate([v.real, v.imag], -1)
    tol = np.concatenate([abs(a) + abs(b)] * 2, -1) * 2.0 ** -21
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot,off", [(128, 128, 0), (64, 32, 16), (66, 34, 2)])
def test_parts_of_one_projection_and_in_place(inter, d, rot, off):
    f, m = dsa.rope_freqs(rot, 1e4)
    L, Hq, Hk = 403, 8, 2
    x = _x(L, 1, (Hq + 2 * Hk) * d + 3, BF, 9)[:, 0]
    whole = x.clone()
    q = x[:, 1:1 + Hq * d].unflatten(1, (Hq, d))      # neither pointer nor stride is 16-byte
    k = x[:, 1 + Hq * d:1 + (Hq + Hk) * d].unflatten(1, (Hk, d))
    pos = torch.arange(L, device="cuda")
    qo, ko = dsa.rope(q, k, pos, f, m, 1.0, off, inter)
    _check(qo, q, pos, f, m, off, inter)
    _check(ko, k, pos, f, m, off, inter)
    assert torch.equal(x, whole)
    dsa.rope(q, k, pos, f, m, 1.0, off, inter, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(x[:, :1], whole[:, :1])
    assert torch.equal(x[:, 1 + (Hq + Hk) * d:], whole[:, 1 + (Hq + Hk) * d:])


def test_repeated_row_and_empty():
    """A token stride of zero heads apart is refused, an expanded row too; no
    tokens give empty arrays."""
    f, m = dsa.rope_freqs(64)
    q = _x(1, 4, 64, BF, 10).expand(8, 4, 64)
    pos = torch.arange(8, device="cuda")
    with pytest.raises(dsa.DSAError):
        dsa.rope(q, None, pos, f)
    with pytest.raises(ValueError, match="dense"):
        dsa.rope(_x(8, 64, 4, BF, 10).transpose(1, 2), None, pos, f)
    qo, ko = dsa.rope(q[:0].contiguous(), q[:0].contiguous(), pos[:0], f)
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 4, 64)


def test_special_values():
    """Infinities and NaN stay where their pair is; e4m3 saturates finite
    values and turns infinities into NaN."""
    f, m = dsa.rope_freqs(64)
    x = _x(1, 1, 128, F32, 11)
    x[0, 0, 3], x[0, 0, 100], x[0, 0, 101], x[0, 0, 102] = float("nan"), float("inf"), 1e6, -1e6
    pos = torch.tensor([5], device="cuda")
    y, _ = dsa.rope(x, None, pos, f, out_dtype=E4)
    y = y.float()[0, 0]
    bad = torch.isnan(y).nonzero().flatten().tolist()
    assert bad == [3, 35, 100]
    assert y[101].item() == 448 and y[102].item() == -448


def test_another_stream_and_a_captured_graph():
    f, m = dsa.rope_freqs(128)
    q, k = _x(64, 32, 128, BF, 12), _x(64, 4, 128, BF, 13)
    pos = torch.arange(64, device="cuda")
    want = dsa.rope(q, k, pos, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dsa.rope(q, k, pos, f, stream=s)
    also = dsa.rope(q, k, pos, f, stream=s.cuda_stream)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want + want, got + also))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = dsa.rope(q, k, pos, f)
    q.copy_(_x(64, 32, 128, BF, 14))
    pos += 1000
    g.replay()
    again = dsa.rope(q, k, pos, f)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, again))


def test_cos_and_sin_round_once():
    """Pairs (1, 0) and (0, 1) read off rot_scale cos and sin: within 0.51 units
    in the last place of rot_scale, borders of the quarter turns among the
    angles."""
    f = torch.tensor([1, 1 << 40, (1 << 61) - 1, 1 << 61, (1 << 61) + 1, 1 << 62, 3 << 61],
                     dtype=torch.int64, device="cuda")
    half = f.numel()
    pos = torch.cat([torch.arange(-20, 4000), torch.randint(-1 << 62, 1 << 62, (20000,))]).cuda()
    for m in (1.0, 1.2079441541679836):
        m32 = float(np.float32(m))
        for first, fn in ((1, np.cos), (0, np.sin)):
            x = torch.zeros((len(pos), 1, 2 * half), device="cuda")
            x[..., :half], x[..., half:] = first, 1 - first
            y, _ = dsa.rope(x, None, pos, f, m)
            turns = (pos[:, None] * f).cpu().numpy().astype(np.longdouble) / 2.0 ** 64
            # cos of (1, 0)'s first half; sin of (0, 1)'s, negated
            ref = m32 * fn(2 * np.longdouble(np.pi) * turns +
                           turns * np.longdouble(2.4492935982947064e-16))
            got = y[:, 0, :half].cpu().numpy() * (1 if first else -1)
            assert np.abs(got - ref).max() <= 0.51 * 2.0 ** -23 * (2 if m > 1 else 1)


def test_after_the_attention_backward():
    """Rotary queries and keys through the sparse attention, forward and
    backward, as a training step uses them: the gradients of the unrotated
    inputs against the oracle's."""
    import oracle.attn_bwd as AB
    L, Hq, Hkv, d, kk = 65, 8, 2, 64, 16
    f, m = dsa.rope_freqs(d, 1e4)
    w = OR.turns_to_frequencies(f.cpu().numpy())
    pos = torch.arange(L, device="cuda")
    q, k, V, dO = (_x(L, h, d, BF, 20 + i) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    Q, K = dsa.rope(q, k, pos, f, m)
    rng = np.random.default_rng(5)
    idx = np.full((L, kk), -1, np.int32)
    for t in range(L):
        n = min(kk, t + 1)
        idx[t, :n] = np.sort(rng.choice(t + 1, n, replace=False))
    di = torch.from_numpy(idx).cuda()
    lse = torch.empty((L, Hq), device="cuda")
    O = dsa.sparse_attn_prefill(Q, K, V, di, d ** -0.5, lse=lse)
    dQ, dK, _ = dsa.sparse_attn_backward(Q, K, V, di, O, lse, dO, d ** -0.5)
    dq, dk = dsa.rope_backward(dQ, dK, pos, f, m)
    assert dsa.device_error() == dsa.DEVERR_NONE
    n64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    ref = AB.backward(n64(Q), n64(K), n64(V), idx, n64(dO), d ** -0.5)
    for got, r in ((dq, ref["dQ"]), (dk, ref["dK"])):
        want = OR.rope(r, pos.cpu().numpy(), w, m, inverse=True)
        # the attention's own bound (1 % in the Frobenius norm), kept by a rotation
        assert np.linalg.norm(n64(got) - want) <= 1e-2 * np.linalg.norm(want)
