"""GPU: drafts and verifications of rows that a grammar has masked (most
entries at DSPARK_MASKED or -infinity) against the oracle, on every draft and
verify path: a masked entry is never chosen and leaves the log-normalisers as
the allowed entries alone make them.  A row that allows nothing is flagged."""
import os

import numpy as np
import pytest
import torch

import oracle
import synth
import semi_ar_draft_amd as dk
from parity import compare_draft, compare_verify

pytestmark = pytest.mark.gpu


def context(**env):
    old = {k: os.environ.get(k) for k in env}
    os.environ.update(env)
    try:
        return dk.Context(0)
    finally:
        for k, v in old.items():
            if v is None:
                del os.environ[k]
            else:
                os.environ[k] = v


def masked_inputs(B, allowed, seed, value, **over):
    """U and target with `allowed` entries left in every row; the target allows what the draft does, and a few more."""
    wl = synth.WORKLOADS["sample"].with_(B=B, V=4096, d_h=8, d_e=8, conf=False, **over)
    inp = synth.make_inputs(wl, seed=seed)
    rng = np.random.RandomState(seed)
    keep = torch.from_numpy(np.argsort(rng.rand(B, wl.V), 1)[:, :allowed + 3])
    for name, n in (("U", allowed), ("target", allowed + 3)):
        x = inp[name]
        y = torch.full_like(x, value)
        at = keep[:, None, :n].expand(-1, x.shape[1], -1)
        inp[name] = y.scatter(2, at, x.gather(2, at))
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in inp.items()}
    return wl, inp, d


PATHS = [(8, {}), (8, dict(DSPARK_PERSIST="0")), (40, dict(DSPARK_PERSIST="0")), (70, {}), (70, dict(DSPARK_CHAIN="0"))]


@pytest.mark.parametrize("T", [1.0, 0.0, 0.3])
@pytest.mark.parametrize("allowed", [1, 5, 400])
@pytest.mark.parametrize("B,env", PATHS)
def test_masked_rows(B, env, allowed, T):
    value = dk.MASKED if allowed != 5 else -float("inf")
    print(f"masked rows B={B} {env} allowed={allowed} T={T} value={value}", flush=True)
    wl, inp, d = masked_inputs(B, allowed, 40 + allowed, value)
    G, seed = wl.gamma, 17
    finite = lambda x: x.clamp(min=-1e30)                        # the oracle's sums of float64 take no infinities
    od = oracle.draft_markov(finite(inp["U"]), inp["W1"], inp["W2"], inp["anchor"], inp["req_ids"], T, seed, G)
    for chain in "01":
        ctx = context(**env, DSPARK_VERIFY_CHAIN=chain)
        try:
            tok, lse, ytok = ctx.draft_markov(d["U"], d["W1"], d["W2"], d["anchor"], d["req_ids"], T, seed, G)
            ctx.check()
            assert torch.isfinite(d["U"].gather(2, tok.long()[..., None])).all()
            assert (d["U"].gather(2, tok.long()[..., None]) > -1e29).all()
            rep, taint = compare_draft(tok.cpu().numpy(), lse.cpu().numpy(), ytok.cpu().numpy(), od)
            acc, out = ctx.verify(d["target"], d["U"], d["W1"], d["W2"], d["anchor"], tok, lse, ytok, None, d["req_ids"], T,
                                  seed)
            ctx.check()
            ov = oracle.verify(finite(inp["target"]), od.tokens, od.lse, od.ytok, finite(inp["U"]), inp["W1"], inp["W2"],
                               inp["anchor"], None, inp["req_ids"], T, seed, G)
            compare_verify(acc.cpu().numpy(), out.cpu().numpy(), ov, taint, None, rep=rep)
            print(rep.summary(), flush=True)
            assert rep.ok(), rep.summary()
        finally:
            ctx.close()


def test_acceptance_of_masked_rows():
    wl, inp, d = masked_inputs(8, 6, 3, dk.MASKED)
    ctx = context()
    try:
        tok, lse, _ = ctx.draft_markov(d["U"], d["W1"], d["W2"], d["anchor"], d["req_ids"], 1.0, 5, wl.gamma)
        a = ctx.accept_prob(d["target"], d["U"], d["W1"], d["W2"], d["anchor"], tok, lse, 1.0)
        ctx.check()
        want = oracle.accept_prob(inp["target"], tok.cpu().numpy(), lse.cpu().numpy(), inp["U"], inp["W1"], inp["W2"],
                                  inp["anchor"], 1.0, wl.gamma)
        assert np.abs(a.cpu().numpy() - want).max() <= 5e-5
    finally:
        ctx.close()


@pytest.mark.parametrize("chain", "01")
def test_a_row_that_allows_nothing_is_flagged(chain):
    wl, inp, d = masked_inputs(6, 50, 9, dk.MASKED)
    ctx = context(DSPARK_VERIFY_CHAIN=chain)
    try:
        args = (d["W1"], d["W2"], d["anchor"])
        tok, lse, ytok = ctx.draft_markov(d["U"], *args, d["req_ids"], 1.0, 5, wl.gamma)
        for K in (0, 2):                                          # a bonus row, a row with a draft to test
            Kd = torch.full((6,), K, dtype=torch.int32, device="cuda")
            good = ctx.verify(d["target"], d["U"], *args, tok, lse, ytok, Kd, d["req_ids"], 1.0, 5)
            ctx.check()
            t = d["target"].clone()
            t[3, 0] = dk.MASKED
            acc, out = ctx.verify(t, d["U"], *args, tok, lse, ytok, Kd, d["req_ids"], 1.0, 5)
            with pytest.raises(dk.DSparkError, match="token id out of range"):
                ctx.check()
            rest = [0, 1, 2, 4, 5]
            assert torch.equal(acc[rest], good[0][rest]) and torch.equal(out[rest], good[1][rest])
            assert acc[3] == 0 and out[3, 0] == 0
        u = d["U"].clone()
        u[2, 1] = dk.MASKED
        got = ctx.draft_markov(u, *args, d["req_ids"], 1.0, 5, wl.gamma)
        with pytest.raises(dk.DSparkError, match="token id out of range"):
            ctx.check()
        rest = [0, 1, 3, 4, 5]
        assert torch.equal(got[0][rest], tok[rest]) and got[0][2, 0] == tok[2, 0] and got[0][2, 1] == 0
    finally:
        ctx.close()
