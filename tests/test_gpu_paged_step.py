"""GPU: serving steps over the paged cache as they are used -- draft,
confidence, schedule, pages, cache write, attention, constraints, packed
verification, pages back -- every call against its oracle, the state carried
from step to step, then the same step captured and replayed to the eager
result with eager work between the replays."""
import numpy as np
import pytest
import torch

import oracle
import synth
import semi_ar_draft_amd as dk
from parity import compare_verify
from test_gpu_attend import check as check_attention
from test_gpu_constrain import compare, want_of, words_of

pytestmark = pytest.mark.gpu

PAGE, HEADS, GROUP, D, PROMPT, N_BIAS, HIST = 16, 2, 3, 64, 150, 4, 400


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Server:
    """Device state of a batch and one step over it; every shape is fixed."""

    def __init__(self, ctx, B, eight, seed):
        self.ctx, self.B, self.eight, self.seed = ctx, B, eight, seed
        wl = synth.WORKLOADS["sample"].with_(B=B, V=2048, r=64, d_h=16, d_e=16, sts=True, sched=True)
        self.inp = synth.make_inputs(wl, seed=wl.seed + seed)
        self.d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in self.inp.items()}
        self.G, self.V = wl.gamma, wl.V
        self.d["sps"] = 1.0 / (2.0 * B + torch.arange(1, 16 * B, device="cuda"))    # some drafts are worth their row, some not
        rng = np.random.RandomState(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.Ek, self.Ev = [torch.randn((self.V, HEADS, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
        self.Eq = torch.randn((self.V, HEADS * GROUP, D), generator=g, device="cuda").to(torch.bfloat16)
        self.coef = torch.randn((1, -(-self.V // (HEADS * GROUP * D)), 1), generator=g, device="cuda")
        self.ks, self.vs = [(torch.rand(HEADS, generator=g, device="cuda") + 0.5) / 50 for _ in range(2)] if eight else (None, None)
        self.prompt = rng.randint(1, PROMPT + 1, B)
        self.prompt[:3] = [1, PAGE, PROMPT]
        self.hist = i32(rng.randint(0, self.V, (B, HIST)))
        cols = -(-HIST // PAGE)
        self.n_pages = int(-(-(self.prompt + 8 * (self.G + 1)) // PAGE).sum())
        self.length, self.held, self.n_free = i32(np.zeros(B)), i32(np.zeros(B)), i32([self.n_pages])
        self.table, self.free = i32(np.full((B, cols), -1)), i32(rng.permutation(self.n_pages))
        self.kc = torch.zeros((self.n_pages, PAGE, HEADS, D), dtype=torch.bfloat16, device="cuda")
        if eight:
            self.kc = self.kc.to(torch.float8_e4m3fn)
        self.vc = self.kc.clone()
        self.anchor, self.n_prompt = i32(rng.randint(0, self.V, B)), i32(self.prompt)
        f = lambda x: torch.from_numpy(x.astype(np.float32)).cuda()
        self.rep, self.freq, self.pres = f(0.8 + rng.rand(B)), f(rng.rand(B) * 0.5), f(rng.rand(B) * 0.5)
        self.bias = (i32(np.sort(rng.randint(0, self.V, (B, N_BIAS)), 1)), f(rng.randn(B, N_BIAS)), i32(rng.randint(0, N_BIAS + 1, B)))
        self.allowed = rng.rand(B, self.V) < 0.9                       # a grammar a request
        self.masks = i32(words_of(self.allowed))
        n = B * (self.G + 1)
        e = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device="cuda")
        fl = lambda: e(B, self.G, dtype=torch.float32)
        self.draft = (e(B, self.G), fl(), fl(), fl(), fl())
        self.sched = (e(B), e(1), e(1, dtype=torch.float64))
        self.rows = (e(B + 1), e(n), e(n), e(n))
        self.q, self.k, self.v = [e(n, h, D, dtype=torch.bfloat16) for h in (HEADS * GROUP, HEADS, HEADS)]
        self.out, self.lse = torch.zeros_like(self.q), e(n, HEADS * GROUP, dtype=torch.float32)
        self.logits, self.target = e(n, self.V, dtype=torch.bfloat16), e(n, self.V, dtype=torch.float32)
        self.mask = e(n, self.V // 32)
        self.verified = (e(B), e(B, self.G + 1))
        self.finished = e(B)

    STATE = ("length", "held", "n_free", "table", "free", "kc", "vc", "anchor", "hist")
    RESULT = STATE + ("out", "target")

    def save(self, names):
        return {k: getattr(self, k).clone() for k in names}

    def load(self, state):
        for k, v in state.items():
            getattr(self, k).copy_(v)

    def prefill(self):
        """The prompts' rows through the same calls."""
        K, n = i32(self.prompt - 1), int(self.prompt.sum()) + 5
        offs, req, pos, slot = self.ctx.pages_reserve(K, self.length, self.table, self.held, self.free, self.n_free, PAGE,
                                                      self.n_pages, n_rows=n)
        tok = self.hist[req.clamp(min=0).long(), pos.clamp(min=0).long()].long()
        self.ctx.cache_write(self.Ek[tok], self.Ev[tok], slot, self.kc, self.vc, self.ks, self.vs)
        self.ctx.pages_commit(self.length, K, self.table, self.held, self.free, self.n_free, PAGE, self.n_pages)

    def step(self, commit=True):
        c, d, G = self.ctx, self.d, self.G
        tokens, lse, ytok, _, surv = self.draft
        c.draft_markov_conf(d["U"], d["W1"], d["W2"], self.anchor, d["req_ids"], 1.0, self.seed, G, d["h"], d["E"], d["wc"],
                            d["bc"], d["sts_T"], out=self.draft)
        K = c.schedule(surv, d["sps"], out=self.sched)[0]
        offs, req, pos, slot = c.pages_reserve(K, self.length, self.table, self.held, self.free, self.n_free, PAGE,
                                               self.n_pages, out=self.rows)
        r = req.clamp(min=0).long()
        i = (torch.arange(len(r), device="cuda") - offs[r]).clamp(0, G)
        tok = torch.where(i == 0, self.anchor[r], tokens[r, (i - 1).clamp(min=0)]).long()
        at = (tok + 7 * pos.clamp(min=0)) % self.V
        self.k.copy_(self.Ek[at])
        self.v.copy_(self.Ev[at])
        self.q.copy_(self.Eq[tok])
        c.cache_write(self.k, self.v, slot, self.kc, self.vc, self.ks, self.vs)
        c.attend(self.q, self.kc, self.vc, self.table, self.length, G, K=K, t_offsets=offs, k_scale=self.ks, v_scale=self.vs,
                 out=self.out, lse=self.lse)
        mixed = (self.out.reshape(len(r), 1, -1).float() * self.coef).reshape(len(r), -1)[:, :self.V]
        self.logits.copy_(d["U"][r, i.clamp(max=G - 1)] + mixed)
        self.mask.copy_(self.masks[r])
        c.constrain(self.logits, G + 1, K=K, t_offsets=offs, hist=self.hist, n_hist=self.length, n_prompt=self.n_prompt,
                    tokens=tokens, rep=self.rep, freq=self.freq, pres=self.pres, bias=self.bias, mask=self.mask, out=self.target)
        acc, emitted = c.verify_packed(self.target, offs[:self.B], d["U"], d["W1"], d["W2"], self.anchor, tokens, lse, ytok, K,
                                       d["req_ids"], 1.0, self.seed, out=self.verified)
        if commit:
            self.commit()

    def commit(self):
        """The kept rows' tokens (the anchor and the accepted drafts) join the history, the last emitted one is next."""
        acc, emitted = self.verified
        tokens = torch.cat([self.anchor[:, None], self.draft[0]], 1)
        j = torch.arange(self.G + 1, device="cuda")
        at = (self.length[:, None] + j).clamp(max=HIST - 1).long()
        self.hist.scatter_(1, at, torch.where(j <= acc[:, None], tokens, self.hist.gather(1, at)))
        self.anchor.copy_(emitted.gather(1, acc[:, None].long())[:, 0])
        self.ctx.pages_commit(self.length, acc, self.table, self.held, self.free, self.n_free, PAGE, self.n_pages,
                              finished=self.finished)


@pytest.fixture(scope="module")
def ctx():
    c = dk.Context(0)
    yield c
    c.close()


def host(x):
    return x.cpu().numpy()


@pytest.mark.parametrize("B,eight", [(24, False), (9, True)])
def test_steps_match_the_oracles(ctx, B, eight):
    print(f"paged steps B={B} 8bit={eight}", flush=True)
    s = Server(ctx, B, eight, 3)
    s.prefill()
    ctx.check()
    assert np.array_equal(host(s.length), s.prompt)
    kept = 0
    for n in range(3):
        before = {k: host(v) for k, v in s.save(("length", "held", "n_free", "table", "free", "anchor")).items()}
        s.step(commit=False)
        ctx.check()
        tokens, K = host(s.draft[0]), host(s.sched[0])
        offs, req, pos, slot = [host(x) for x in s.rows]
        want = oracle.pages_reserve(K, before["length"], before["table"], before["held"], before["free"], before["n_free"][0],
                                    PAGE, len(req))
        for w, g in zip(want, (offs, req, pos, slot, host(s.table), host(s.held), host(s.n_free)[0])):
            assert np.array_equal(w, g)
        total, length = offs[-1], before["length"]
        wrote = (torch.from_numpy(slot[:total] // PAGE).long(), torch.from_numpy(slot[:total] % PAGE).long())
        for cache, x, scale in ((s.kc, s.k, s.ks), (s.vc, s.v, s.vs)):
            got = cache.cpu().float()[wrote].double().numpy()
            x = x[:total].cpu().float().double().numpy()
            assert np.array_equal(got, x if scale is None else oracle.to_e4m3(x / host(scale).astype(np.float64)[:, None]))
        check_attention(dict(q=s.q[:total], kc=s.kc, vc=s.vc, table=host(s.table), length=length, K=K, offs=offs, ks=s.ks,
                             vs=s.vs, scale=D ** -0.5), s.out[:total], s.lse[:total])
        rules = dict(B=B, n_pos=s.G + 1, V=s.V, K=K, n_hist=length, n_prompt=s.prompt, hist=host(s.hist), tokens=tokens,
                     rep=host(s.rep), freq=host(s.freq), pres=host(s.pres), bias_n=host(s.bias[2]), bias_id=host(s.bias[0]),
                     bias_val=host(s.bias[1]), allowed=np.repeat(s.allowed[:, None], s.G + 1, 1))
        rows = [slice(offs[b], offs[b + 1]) for b in range(B)]
        compare([s.target[r] for r in rows], *want_of(rules, [s.logits[r].double().cpu().numpy() for r in rows]))
        target = np.zeros((B, s.G + 1, s.V))
        for b, r in enumerate(rows):
            target[b, :K[b] + 1] = host(s.target[r])
        ov = oracle.verify(target, tokens, host(s.draft[1]), host(s.draft[2]), s.inp["U"], s.inp["W1"], s.inp["W2"],
                           before["anchor"], K, s.inp["req_ids"], 1.0, s.seed, s.G)
        rep = compare_verify(host(s.verified[0]), host(s.verified[1]), ov, np.full(B, s.G + 1), K)
        assert rep.ok(), rep.summary()
        for b in range(B):                                        # nothing that the grammar forbids is emitted
            for t in host(s.verified[1])[b]:
                assert t < 0 or s.allowed[b, t]
        acc = host(s.verified[0])
        kept += int(acc.sum())
        s.finished.copy_(i32(np.arange(B) == n))                   # a request ends with every step
        wl, wh, wf, wt = oracle.pages_commit(length, acc, want[4], want[5], before["free"], want[6], PAGE, host(s.finished))
        s.commit()
        ctx.check()
        for w, g in ((wl, s.length), (wh, s.held), ([wt], s.n_free), (wf, s.free)):
            assert np.array_equal(w, host(g))
    print("accepted drafts:", kept)
    owned = np.concatenate([host(s.table)[b, :host(s.held)[b]] for b in range(B)] + [host(s.free)[:s.n_free.item()]])
    assert np.array_equal(np.sort(owned), np.arange(s.n_pages))    # every page once, in the pool or with one request


def test_the_step_captured_and_replayed(ctx):
    s = Server(ctx, 16, False, 4)
    s.prefill()
    start = s.save(s.STATE)
    want = []
    for n in range(3):
        s.step()
        torch.cuda.synchronize()
        want.append(s.save(s.RESULT))
    ctx.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step()
    side.synchronize()
    print("capturing the step", flush=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.step()
    for turn in range(2):
        s.load(start)
        s.out.zero_()
        s.target.zero_()
        for n in range(3):
            graph.replay()
            torch.cuda.synchronize()
            got = s.save(s.RESULT)
            for k in s.RESULT:
                a, b = got[k], want[n][k]
                if k in ("out", "target"):                         # rows of no request hold what earlier steps left
                    t = int(s.rows[0][-1])
                    a, b = a[:t], b[:t]
                assert torch.equal(a.float() if a.dtype == torch.float8_e4m3fn else a,
                                   b.float() if b.dtype == torch.float8_e4m3fn else b), (turn, n, k)
            if turn == 1:                                          # other eager work between the replays
                s.step()
                torch.cuda.synchronize()
                s.load(got)
    ctx.check()
