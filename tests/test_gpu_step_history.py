"""GPU: the penalties of a serving step count every token before the drafts, the
anchor among them.  The sequences are kept on the host, token by token as they
were emitted, and each step's constrained rows are held against them."""
import numpy as np
import pytest

import semi_ar_draft_amd as dk
from test_gpu_constrain import compare, want_of
from test_gpu_paged_step import Server, host

pytestmark = pytest.mark.gpu


class WithAnchor:
    """The context, its penalties one token further: the anchor behind the cached ones."""

    def __init__(self, ctx):
        self._ctx = ctx

    def __getattr__(self, name):
        return getattr(self._ctx, name)

    def constrain(self, *args, n_hist, **kw):
        return self._ctx.constrain(*args, n_hist=n_hist + 1, **kw)


class Serving(Server):
    def step(self, commit=True):
        self.hist.scatter_(1, self.length[:, None].long(), self.anchor[:, None])
        super().step(commit)


@pytest.mark.parametrize("B,eight", [(9, False), (24, True)])
def test_every_token_before_the_drafts_counts(B, eight):
    ctx = dk.Context(0)
    try:
        s = Serving(WithAnchor(ctx), B, eight, 6)
        s.prefill()
        s.pres.add_(0.25)                                         # every written token loses something
        told = [list(h[:n]) + [a] for h, n, a in zip(host(s.hist), s.prompt, host(s.anchor))]
        for _ in range(4):
            anchor = host(s.anchor)
            s.step()
            ctx.check()
            tokens, K, offs = host(s.draft[0]), host(s.sched[0]), host(s.rows[0])
            rows = [slice(offs[b], offs[b + 1]) for b in range(B)]
            logits = [s.logits[r].double().cpu().numpy() for r in rows]
            longest = max(map(len, told))
            rules = dict(B=B, n_pos=s.G + 1, V=s.V, K=K, n_hist=[len(t) for t in told], n_prompt=s.prompt,
                         hist=np.array([t + [0] * (longest - len(t)) for t in told]), tokens=tokens, rep=host(s.rep),
                         freq=host(s.freq), pres=host(s.pres), bias_n=host(s.bias[2]), bias_id=host(s.bias[0]),
                         bias_val=host(s.bias[1]), allowed=np.repeat(s.allowed[:, None], s.G + 1, 1))
            compare([s.target[r] for r in rows], *want_of(rules, logits))
            for b in range(B):
                if s.allowed[b, anchor[b]] and anchor[b] not in host(s.bias[0])[b]:
                    assert host(s.target[rows[b]])[0, anchor[b]] != np.float32(logits[b][0, anchor[b]])
            acc, emitted = [host(x) for x in s.verified]
            for b in range(B):
                told[b] += [int(t) for t in emitted[b, :acc[b] + 1]]
                assert host(s.length)[b] == len(told[b]) - 1      # cached: all but the new anchor
                assert host(s.hist)[b, :len(told[b]) - 1].tolist() == told[b][:-1]
    finally:
        ctx.close()
