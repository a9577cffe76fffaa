"""GPU: infinite values that a row sees.  They make its results infinite (NaN
where both signs meet) in their columns and nothing else, in any step of a tile
and whatever weight they come with, also one that bf16 holds exactly."""
import numpy as np
import pytest
import torch

import semi_ar_draft_amd as dk
from test_gpu_attend import call, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,group", [(64, 1), (128, 4), (128, 8), (256, 2)])
@pytest.mark.parametrize("equal", [True, False])
@pytest.mark.parametrize("causal", [True, False])
def test_values_that_are_infinite(d, group, equal, causal):
    ctx = dk.Context(0)
    try:
        s = make(d + group, [400, 90, 5], [7, 3, 2], 2, group, d, 16)
        if equal:                                                # every weight is the same power of two
            s["q"].zero_()
        clean, lse = call(ctx, s, causal)
        inf = float("inf")
        for b, (L, K) in enumerate(zip(s["length"], s["K"])):
            for t in {0, 3, L // 2, L - 1, L, L + K}:
                for kind in ((inf,), (-inf,), (inf, -inf)):
                    v = s["vc"].clone()
                    at = [t, t - 1 if t else 1][:len(kind)]
                    for place, value in zip(at, kind):
                        v[s["table"][b][place // 16], place % 16, 1, 5:9] = value
                    out, l2 = call(ctx, dict(s, vc=v), causal)
                    ctx.check()
                    assert torch.equal(l2, lse)
                    want = clean.clone()
                    for i in range(K + 1):
                        see = [x for place, x in zip(at, kind) if place <= (L + i if causal else L + K)]
                        if see:
                            want[s["offs"][b] + i, group:, 5:9] = sum(see)
                    assert torch.equal(torch.isnan(out), torch.isnan(want)), (b, t, kind)
                    assert torch.equal(torch.nan_to_num(out.float()), torch.nan_to_num(want.float())), (b, t, kind)
    finally:
        ctx.close()
