"""GPU: a draft row that allows nothing has an empty sum (lse = -infinity) and
probabilities of 0: no target token is accepted through it, its acceptance
probability is 0, and what follows comes from the target alone."""
import numpy as np
import pytest
import torch

import oracle
import semi_ar_draft_amd as dk
from parity import compare_verify
from test_gpu_masked_rows import context, masked_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,env", [(6, {}), (6, dict(DSPARK_PERSIST="0")), (70, {}), (70, dict(DSPARK_CHAIN="0"))])
@pytest.mark.parametrize("fused", [False, True])
def test_acceptance_of_a_draft_row_that_allows_nothing(B, env, fused):
    wl, inp, d = masked_inputs(B, 50, 9, dk.MASKED)
    args = (d["W1"], d["W2"], d["anchor"])
    ctx = context(**env)
    try:
        def draft(u):
            if fused:
                h = torch.zeros((B, wl.gamma, 8), dtype=torch.bfloat16, device="cuda")
                E = torch.zeros((wl.V, 8), dtype=torch.bfloat16, device="cuda")
                return ctx.draft_markov_conf(u, *args, d["req_ids"], 1.0, 5, wl.gamma, h, E, h[0, 0].repeat(2), 0.0)[:3]
            return ctx.draft_markov(u, *args, d["req_ids"], 1.0, 5, wl.gamma)

        tok, lse, ytok = draft(d["U"])
        good = ctx.accept_prob(d["target"], d["U"], *args, tok, lse, 1.0)
        ctx.check()
        u = d["U"].clone()
        u[2, 3] = dk.MASKED
        u[4, 0] = dk.MASKED
        t2, l2, _ = draft(u)
        with pytest.raises(dk.DSparkError, match="token id out of range"):
            ctx.check()
        assert l2[2, 3] == -float("inf") and l2[4, 0] == -float("inf")
        got = ctx.accept_prob(d["target"], u, *args, t2, l2, 1.0)
        ctx.check()
        assert got[2, 3] == 0 and got[4, 0] == 0
        same = torch.ones_like(good, dtype=torch.bool)
        same[2, 3:] = False                                      # the next rows' bias is that of another token
        same[4] = False
        assert torch.equal(got[same], good[same]) and torch.isfinite(got).all()
    finally:
        ctx.close()


@pytest.mark.parametrize("chain", "01")
def test_verification_draws_from_the_target_there(chain):
    wl, inp, d = masked_inputs(6, 50, 9, dk.MASKED)
    args = (d["W1"], d["W2"], d["anchor"])
    ctx = context(DSPARK_VERIFY_CHAIN=chain)
    try:
        u = d["U"].clone()
        u[4, 0] = dk.MASKED
        tok, lse, ytok = ctx.draft_markov(u, *args, d["req_ids"], 1.0, 5, wl.gamma)
        with pytest.raises(dk.DSparkError):
            ctx.check()
        K = torch.full((6,), 3, dtype=torch.int32, device="cuda")
        acc, out = ctx.verify(d["target"], u, *args, tok, lse, ytok, K, d["req_ids"], 1.0, 5)
        ctx.check()
        assert acc[4] == 0 and d["target"][4, 0, out[4, 0].long()] > -1e29
        f = lambda x: x.cpu().numpy()
        with np.errstate(over="ignore"):
            ov = oracle.verify(inp["target"], f(tok), f(lse).astype(np.float64), f(ytok), u.cpu(), inp["W1"], inp["W2"],
                               inp["anchor"], f(K), inp["req_ids"], 1.0, 5, wl.gamma)
        rep = compare_verify(f(acc), f(out), ov, np.full(6, wl.gamma + 1), f(K))
        assert rep.ok(), rep.summary()
    finally:
        ctx.close()
