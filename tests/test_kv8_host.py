"""The paged 8-bit cache without a GPU: the oracle's pins and the calls'
refusals."""
import numpy as np
import pytest
import torch

import gen
import oracle.kv8 as KV
import oracle.kl as KL
import sparse_long_context_02_b200 as dsa
from sparse_long_context_02_b200 import build as dsa_build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 0x10000  # aligned, never dereferenced: every call below fails validation


@pytest.fixture(scope="module")
def L():
    dsa_build.build()
    return dsa.lib()


def test_oracle_codes():
    """Every code's value, and the rounding, against the generator's encoder
    and torch's conversion."""
    assert np.array_equal(KV.VALUES, KL.decode_e4m3(np.arange(256)), equal_nan=True)
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-14, 8, 4000),
                        (KV.VALUES[:126] + KV.VALUES[1:127]) / 2, KV.VALUES[:127],
                        -KV.VALUES[:127], [447.9, 448.0, 2.0 ** -10, 2.0 ** -11]])
    got = KV.encode(x)
    assert np.array_equal(KV.VALUES[got], KL.decode_e4m3(gen.encode_e4m3(x)))
    t = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)
    assert np.array_equal(KV.encode(x.astype(np.float32)), t.numpy())
    assert KV.encode(1e9) == 126 and KV.encode(np.inf) == 127 and KV.encode(np.nan) == 127


def test_oracle_scale():
    assert KV.need([448.0]) == 1.0 and KV.need([-449.0, 3.0]) == 2.0
    assert KV.need([448.0 * 2 ** -30]) == 2.0 ** -30
    assert KV.need([]) == KV.need([0.0]) == 2.0 ** -120
    assert KV.need([np.inf, np.nan, 1.0]) == 2.0 ** -8
    assert KV.need([3.3e38]) == 2.0 ** 120


def test_oracle_append_by_hand():
    codes = np.full((3, 2, 1, 2), 9, np.uint8)
    scales = np.full((3, 1), 7.0)
    table = np.array([[2, 0], [1, -1]])
    x = np.array([[1.0, 448.0], [900.0, -2.0], [0.0, 1.0], [5.0, 5.0]]).reshape(4, 1, 2)
    KV.append(x[:1], codes, scales, table, [0, -1], [0, 1, 1])
    assert scales[:, 0].tolist() == [7, 7, 1] and codes[2, 1, 0].tolist() == [9, 9]
    assert KV.decode(codes[2, 0, 0]).tolist() == [1, 448]
    # two more: the first joins page 2 and raises its scale to 4, the second opens page 0
    KV.append(x[1:3], codes, scales, table, [1, -1], [0, 2, 2])
    assert scales[:, 0].tolist() == [2.0 ** -8, 7, 4]
    assert KV.decode(codes[2, 0, 0]).tolist() == [0.25, 112]
    assert KV.decode(codes[2, 1, 0]).tolist() == [224, -0.5]  # 900 / 4 = 225, steps of 16
    assert KV.decode(codes[0, 0, 0]).tolist() == [0, 256]
    # a table entry outside the pool, a position past the table: nothing moves
    before = codes.copy(), scales.copy()
    KV.append(x[3:], codes, scales, table, [4, 2], [0, 0, 1])
    KV.append(x[3:], codes, scales, table, [4, 4], [0, 1, 1])
    assert np.array_equal(before[0], codes) and np.array_equal(before[1], scales)


# K, V, T, k_stride, v_stride, K8, V8, k_scale, v_scale, num_pages, page, block_table, max_pages,
# seq_lens, new_off, B, Hkv, d, err, stream
APPEND = [FAKE, FAKE, 8, 256, 256, FAKE, FAKE, FAKE, FAKE, 10, 64, FAKE, 4, FAKE, FAKE, 3, 2, 128,
          None, None]


@pytest.mark.parametrize("at,value,status", [
    (0, None, INVALID), (0, FAKE + 8, INVALID), (1, FAKE + 2, INVALID), (2, -1, INVALID),
    (2, 1 << 31, INVALID), (3, 248, INVALID), (3, 260, INVALID), (4, 128, INVALID),
    (5, None, INVALID), (5, FAKE + 8, INVALID), (6, None, INVALID), (7, None, INVALID),
    (8, FAKE + 2, INVALID), (9, 0, INVALID), (9, 1 << 25, INVALID), (10, 48, UNSUPPORTED),
    (10, 0, UNSUPPORTED), (10, 256, UNSUPPORTED), (11, None, INVALID), (12, 0, INVALID),
    (12, 1 << 25, INVALID), (13, None, INVALID), (14, None, INVALID), (14, FAKE + 2, INVALID),
    (15, 0, INVALID), (15, -1, INVALID), (15, 1 << 25, INVALID), (16, 0, INVALID),
    (16, 65, UNSUPPORTED), (17, 96, UNSUPPORTED), (18, FAKE + 1, INVALID)])
def test_append_refusals(L, at, value, status):
    a = list(APPEND)
    a[at] = value
    assert L.dsa_kv8_append(*a) == status
    assert b"dsa_kv8_append" in L.dsa_last_error()


def test_append_of_nothing(L):
    a = list(APPEND)
    a[2] = 0
    assert L.dsa_kv8_append(*a) == OK


def _cache(P=4, page=16, Hkv=2, d=64, B=2, M=3):
    return dict(k8=torch.zeros((P, page, Hkv, d), dtype=torch.uint8),
                v8=torch.zeros((P, page, Hkv, d), dtype=torch.uint8),
                k_scale=torch.zeros((P, Hkv)), v_scale=torch.zeros((P, Hkv)),
                block_table=torch.zeros((B, M), dtype=torch.int32),
                seq_lens=torch.zeros(B, dtype=torch.int32))


@pytest.mark.parametrize("change,match", [
    (dict(k8=torch.zeros((4, 16, 2, 64))), "float8"),
    (dict(v8=torch.zeros((4, 16, 2, 128), dtype=torch.uint8)), "one shape"),
    (dict(k_scale=torch.zeros((4, 3))), "k_scale"),
    (dict(v_scale=torch.zeros((4, 2), dtype=torch.float64)), "v_scale"),
    (dict(block_table=torch.zeros((2, 3), dtype=torch.int64)), "block_table"),
    (dict(seq_lens=torch.zeros(3, dtype=torch.int32)), "seq_lens"), ({}, "CUDA")])
def test_binding_checks_of_the_cache(change, match):
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=match):
        dsa.kv8_append(x, x, **{**_cache(), **change})


# Q, K8, V8, k_scale, v_scale, num_pages, page, block_table, max_pages, seq_lens, row_off, B, T
CACHE = [FAKE, FAKE, FAKE, FAKE, FAKE, 10, 64, FAKE, 4, FAKE, FAKE, 3, 8]
# Hq, Hkv, d, scale, O, lse, workspace, bytes, err, stream
REST = [32, 4, 128, 0.1, FAKE, FAKE, FAKE, 1 << 30, None, None]
SPARSE, DENSE = CACHE + [FAKE, 64] + REST, CACHE + REST


@pytest.mark.parametrize("at,value,status", [
    (0, None, INVALID), (0, FAKE + 8, INVALID), (1, None, INVALID), (2, FAKE + 4, INVALID),
    (3, None, INVALID), (4, FAKE + 1, INVALID), (5, 0, INVALID), (5, 1 << 25, INVALID),
    (6, 8, UNSUPPORTED), (6, 65, UNSUPPORTED), (7, None, INVALID), (8, 0, INVALID),
    (8, 1 << 25, INVALID), (9, None, INVALID), (10, None, INVALID), (10, FAKE + 2, INVALID),
    (11, 0, INVALID), (11, -3, INVALID), (11, 1 << 25, INVALID), (12, -1, INVALID),
    (12, 1 << 30, UNSUPPORTED), (13, None, INVALID), (13, FAKE + 3, INVALID), (14, 0, INVALID),
    (14, 65537, INVALID), (15, 30, INVALID), (15, 64, UNSUPPORTED), (15, 0, INVALID),
    (16, 0, INVALID), (16, 128, INVALID), (17, 96, UNSUPPORTED), (18, 0.0, INVALID),
    (18, -1.0, INVALID), (18, float("nan"), INVALID), (18, float("inf"), INVALID),
    (19, None, INVALID), (20, FAKE + 2, INVALID), (21, None, INVALID), (21, FAKE + 8, INVALID),
    (22, 15, WORKSPACE), (23, FAKE + 1, INVALID)])
def test_attention_refusals(L, at, value, status):
    a = list(SPARSE)
    a[8], a[14] = 4096, 65536  # sizes that need a workspace
    assert L.dsa_attn_kv8_workspace_size(8, 65536, 32, 4, 128) > 15
    a[at] = value
    assert L.dsa_sparse_attn_kv8(*a) == status
    assert b"dsa_sparse_attn_kv8" in L.dsa_last_error()
    if at not in (13, 14):
        assert L.dsa_attn_kv8(*a[:13], *a[15:]) == status
        assert b"dsa_attn_kv8" in L.dsa_last_error()


def test_attention_of_nothing(L):
    a = list(SPARSE)
    a[12] = 0
    assert L.dsa_sparse_attn_kv8(*a) == OK
    a = list(DENSE)
    a[12] = 0
    assert L.dsa_attn_kv8(*a) == OK


def test_attention_workspace_sizes(L):
    f = L.dsa_attn_kv8_workspace_size
    assert f(0, 100, 32, 4, 128) == 0 and f(4, 0, 32, 4, 128) == 0
    assert f(4, 100, 32, 0, 128) == 0 and f(-1, 100, 32, 4, 128) == 0
    assert 0 < f(1, 1 << 20, 32, 4, 128) < 1 << 28
    assert f(64, 2048, 32, 4, 128) < 1 << 28 and f(1 << 20, 2048, 32, 4, 128) < 1 << 30


def test_binding_checks_of_the_attention():
    c = _cache()
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    args = (c["k8"], c["v8"], c["k_scale"], c["v_scale"], c["block_table"], c["seq_lens"])
    with pytest.raises(ValueError, match="CUDA"):
        dsa.attn_kv8(q, *args, 0.1)
    with pytest.raises(ValueError, match="seq_lens"):
        dsa.attn_kv8(q, *args[:5], torch.zeros(1, dtype=torch.int32), 0.1)
