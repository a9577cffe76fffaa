"""The vectorised float64 attention of the tests against the oracle (CPU)."""
import numpy as np
import pytest
import torch

import oracle
from attend_reference import attend64


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("scaled", [True, False])
def test_the_reference_is_the_oracle(causal, scaled):
    rng = np.random.RandomState(3)
    g = torch.Generator().manual_seed(3)
    page, H, group, D = 8, 2, 3, 16
    length, K = np.array([0, 13, 30, 5]), np.array([2, 4, 0, -1])
    offs = np.array([0, 3, 8, 9])
    table = rng.permutation(24)[:20].reshape(4, 5)
    kc, vc = [torch.randn((24, page, H, D), generator=g).to(torch.bfloat16) for _ in range(2)]
    q = torch.randn((10, H * group, D), generator=g).to(torch.bfloat16)
    ks, vs = [torch.rand(H, generator=g) + 0.5 for _ in range(2)] if scaled else (None, None)
    f64 = lambda x: None if x is None else x.double().numpy()
    out, lse, mean, ds = attend64(q, kc, vc, table, length, K, offs, causal=causal, scale=0.3, k_scale=ks, v_scale=vs)
    how = dict(causal=causal, scale=0.3, k_scale=f64(ks), v_scale=f64(vs))
    want, wl = oracle.attend(f64(q), f64(kc), f64(vc), table, length, K, offs, **how)
    wmean, _ = oracle.attend(f64(q), f64(kc), np.abs(f64(vc)), table, length, K, offs, **how)
    for a, b in ((out, want), (lse, wl), (mean, wmean)):
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.isnan(a[9]).all()
        assert np.allclose(a[:9], b[:9], rtol=1e-12, atol=1e-13)
    assert (ds[:9] > 0).all()
