"""More than 512 rows over every key of the paged 8-bit cache, which are dealt
out whole: no workspace, and rows of very different lengths."""
import numpy as np
import pytest
import torch

import oracle.kv8 as KV
import sparse_long_context_02_b200 as dsa
from test_gpu_kv8_attn import Case

pytestmark = pytest.mark.gpu


def test_no_workspace_is_asked_for():
    c = Case([20] * 600, 16, 32, 4, 128, 1)
    cache = c.cache()
    O = torch.empty_like(c.Qt)
    want = dsa.attn_kv8(c.Qt, *cache, c.scale)
    dsa.attn_kv8(c.Qt, *cache, c.scale, O=O, workspace=torch.empty(0, device="cuda"))
    assert torch.equal(O, want)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    dsa.attn_kv8(c.Qt, *cache, c.scale, O=O)
    assert torch.cuda.max_memory_allocated() == before
    # 512 rows are cut into ranges, which need one
    half = [t[:512].contiguous() for t in cache[4:]]
    with pytest.raises(dsa.DSAError, match="workspace"):
        dsa.attn_kv8(c.Qt[:512], *cache[:4], *half, c.scale, O=O[:512],
                     workspace=torch.empty(0, device="cuda"))


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 4, 64), (4, 1, 128)])
def test_one_long_row_among_short_ones(Hq, Hkv, d):
    """One CTA walks the whole of a row.  A warp then adds its share of the
    units (each NSUB-th, NSUB = 8 / heads per CTA) in one chain: two products
    of 16 keys and four weights per lane and unit.  Each addition of a product
    may truncate (2^-23 of the running sum, at most sum p |v|), each of a weight
    rounds (2^-24): with n keys 2 n / (32 NSUB) 2^-23 + 4 n / (32 NSUB) 2^-24 on
    top of the other rows' bound."""
    n, T, page = 120001, 520, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    lens = torch.randint(1, 40, (T,), generator=g, device="cuda", dtype=torch.int32)
    at = 261
    lens[at] = n
    need = -(-n // page)
    P = need + T
    pools = [torch.randint(0, 256, (P, page, Hkv, d), generator=g, device="cuda",
                           dtype=torch.uint8) for _ in "kv"]
    for x in pools:
        x[(x & 127) == 127] = 0x38
    ks = torch.full((P, Hkv), 2.0 ** -9, device="cuda")
    vs = 2.0 ** torch.randint(-8, -3, (P, Hkv), generator=g, device="cuda").float()
    table = torch.full((T, need), -1, dtype=torch.int32, device="cuda")
    table[:, 0] = torch.arange(T, device="cuda")
    table[at] = torch.cat([torch.tensor([at], device="cuda"), T + torch.arange(need - 1, device="cuda")])
    Q = torch.randn((T, Hq, d), generator=g, device="cuda").bfloat16()
    lse = torch.empty((T, Hq), device="cuda")
    scale = d ** -0.5
    O = dsa.attn_kv8(Q, *pools, ks, vs, table, lens, scale, lse=lse)
    assert dsa.device_error() == dsa.DEVERR_NONE
    values = torch.from_numpy(KV.VALUES).cuda()
    share = n / (32 * (8 // min(Hkv, 4)))
    for t in (0, at - 1, at, at + 1, T - 1):
        m = int(lens[t])
        where = torch.arange(m, device="cuda")
        p = table[t, where // page].long()
        K, V = (values[x[p, where % page].int()] * s[p].double()[..., None]
                for x, s in zip(pools, (ks, vs)))
        for h in range(Hq):
            q = Q[t, h].double()
            x = K[:, h * Hkv // Hq] @ q * scale
            big = (K[:, h * Hkv // Hq].abs() @ q.abs()).max().item() * scale
            w = torch.softmax(x, 0)
            v = V[:, h * Hkv // Hq]
            ref, mag = w @ v, w @ v.abs()
            top = (w * vs[p, h * Hkv // Hq]).max().item()
            E = 2.0 ** -19 * big
            chain = share * (2 * 2.0 ** -23 + 4 * 2.0 ** -24) if t == at else 0.0
            tol = mag * (np.expm1(2 * E) + 2.0 ** -11 + 2.0 ** -18 + chain) + m * 2.0 ** -31 * top
            tol = tol + (ref.abs() + tol) * 2.0 ** -8
            assert torch.all((O[t, h].double() - ref).abs() <= tol), (t, h)
            rl = torch.logsumexp(x, 0).item()
            assert abs(lse[t, h].item() - rl) <= (E + 2.0 ** -18 + chain + abs(rl) * 2.0 ** -22)
