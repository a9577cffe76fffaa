"""GPU: rows whose logits all lie far below zero in units of the temperature
are rows like any others: the draft and the bonus draw take the entries that
the oracle takes.  (Only logits below -1e29 count as masked.)"""
import numpy as np
import pytest
import torch

import oracle
import synth
from parity import compare_draft, compare_verify
from test_gpu_masked_rows import PATHS, context

pytestmark = pytest.mark.gpu


def low_inputs(B, seed, shift):
    """Rows around -shift, one entry of each 6 above the others' level, so that its lead is beyond float32 rounding."""
    wl = synth.WORKLOADS["sample"].with_(B=B, V=4096, d_h=8, d_e=8, conf=False)
    inp = synth.make_inputs(wl, seed=seed)
    g = torch.Generator().manual_seed(seed)
    for name in ("U", "target"):
        x = inp[name].clamp(-3, 3)
        at = torch.randint(0, wl.V, (*x.shape[:2], 1), generator=g)
        inp[name] = x.scatter_add(2, at, torch.full(at.shape, 30.0)) - shift
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in inp.items()}
    return wl, inp, d


@pytest.mark.parametrize("T,shift", [(1e-6, 500.0), (1e-7, 80.0), (3e-8, 30.0)])
@pytest.mark.parametrize("B,env", PATHS)
def test_rows_far_below_zero(B, env, T, shift):
    print(f"low rows B={B} {env} T={T} shift={shift}", flush=True)
    wl, inp, d = low_inputs(B, 7, shift)
    G, seed = wl.gamma, 19
    od = oracle.draft_markov(inp["U"], inp["W1"], inp["W2"], inp["anchor"], inp["req_ids"], T, seed, G)
    K = torch.zeros(B, dtype=torch.int32)
    for chain in "01":
        ctx = context(**env, DSPARK_VERIFY_CHAIN=chain)
        try:
            tok, lse, ytok = ctx.draft_markov(d["U"], d["W1"], d["W2"], d["anchor"], d["req_ids"], T, seed, G)
            acc, out = ctx.verify(d["target"], d["U"], d["W1"], d["W2"], d["anchor"], tok, lse, ytok, K.cuda(), d["req_ids"],
                                  T, seed)
            ctx.check()
            assert (d["U"].amax(2) / T < -1.86e8).any() or shift < 50
            rep, taint = compare_draft(tok.cpu().numpy(), lse.cpu().numpy(), ytok.cpu().numpy(), od)
            ov = oracle.verify(inp["target"], od.tokens, od.lse, od.ytok, inp["U"], inp["W1"], inp["W2"], inp["anchor"],
                               K.numpy(), inp["req_ids"], T, seed, G)
            compare_verify(acc.cpu().numpy(), out.cpu().numpy(), ov, taint, K.numpy(), rep=rep)
            print(rep.summary(), flush=True)
            assert rep.ok(), rep.summary()
        finally:
            ctx.close()

