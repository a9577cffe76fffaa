"""GPU: attention over a 4-bit cache at every head size, tile height (16, 32,
64 rows, several tiles) and page size (below 16, from 16 on) against float64,
NaN blocks in every place that no row sees.  The bound is that of
test_gpu_attend_mxfp4."""
import numpy as np
import pytest
import torch

import semi_ar_draft_amd as dk
from test_gpu_attend_mxfp4 import call, check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = dk.Context(0)
    yield c
    c.close()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 16, 256])
@pytest.mark.parametrize("gamma,group", [(3, 4), (7, 4), (7, 8), (6, 9), (32, 5)])   # 16, 32, 64, 63 rows, 165
@pytest.mark.parametrize("causal", [True, False])
def test_every_tile(ctx, d, page, gamma, group, causal):
    order = "head" if page == 16 else "token"
    print(f"attend mxfp4 d={d} page={page} {order} gamma={gamma} group={group} causal={causal}", flush=True)
    lengths = [0, 1, 31, 32, 7, 250, 2900, 15]
    K = [gamma, 0, gamma // 2, gamma, -1, 1, gamma, gamma]
    s = make(d + page + gamma, lengths, K, 2, group, d, page, order)
    used = torch.zeros((s["kc"].shape[0], page), dtype=torch.bool)
    for b in range(len(K)):
        t = np.arange(lengths[b] + K[b] + 1 if K[b] >= 0 else 0)
        used[s["table"][b][t // page], t % page] = True
    un = ~used.cuda()
    real = {k: s[k].clone() for k in ("kc", "vc", "kp", "vp")}
    for name in ("kp", "vp"):
        s[name].masked_fill_(un[:, None, :, None], 255)
    for name in ("kc", "vc"):
        s[name].masked_fill_(un[:, :, None, None], 0xFF)
    out, lse = call(ctx, s, causal)
    ctx.check()
    check(dict(s, **real), out, lse, causal)
    again, lse2 = call(ctx, s, causal)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 32])
@pytest.mark.parametrize("gamma,group", [(3, 4), (7, 4), (7, 8)])
def test_drafts_that_are_nan_to_later_rows_alone(ctx, d, page, gamma, group):
    """A NaN block of values in the second draft: rows before it are as without it."""
    print(f"attend mxfp4 NaN draft d={d} page={page} gamma={gamma} group={group}", flush=True)
    s = make(9, [40, 333, 0], [gamma, 2, 3], 2, group, d, page)
    out, lse = call(ctx, s)
    check(s, out, lse)
    t = dict(s, vp=s["vp"].clone())
    block = d // 32 - 1
    for b in range(3):
        at = s["length"][b] + 2
        t["vp"][s["table"][b][at // page], 1, at % page, block] = 255
    got, lse2 = call(ctx, t)
    ctx.check()
    hit = torch.zeros_like(out, dtype=torch.bool)
    for b in range(3):
        hit[s["offs"][b] + 2:s["offs"][b + 1], group:, 32 * block:32 * block + 32] = True
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], out[~hit]) and torch.equal(lse, lse2)
