"""The attention over the paged 8-bit cache on values that its parity tests do
not meet, against the float64 oracle (oracle/kv8.py)."""
import numpy as np
import pytest
import torch

import sparse_long_context_02_b200 as dsa
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
