"""Timed cases of the operators around a packed verify batch.

The scheduler gives every request a verify length K[b]; the target then runs
over the K[b] + 1 rows of every request laid end to end, and the verification
reads the logits it returns.  Between the two stand the operators timed here:

  reserve    pages of the key-value cache for the rows of a step, and the row
             offsets, positions and cache slots of the packed batch
  commit     lengths advanced by what was accepted, surplus pages given back
  write      the rows' keys and values into their cache slots
  attend     attention of the packed rows over the paged cache
  constrain  penalties, biases and grammar masks on the rows' logits

``run`` computes them in elementary torch operations (``own`` false) or calls
the library (``own`` true).  Lengths and verify lengths are a fixed multiset
of the case, dealt to the requests by the seed, so that the work of a case is
known without its inputs.
"""
import math

import numpy as np
import torch

own = False

MASKED = -1.0e30
_CONTEXT = []


def _context():
    """The library's context, made once and kept as a serving program keeps it."""
    if not _CONTEXT:
        import semi_ar_draft_amd
        _CONTEXT.append(semi_ar_draft_amd.Context(0))
    return _CONTEXT[0]


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one request in flight: the bookkeeping of a step is pure latency
        dict(name="reserve_one", op="reserve", B=1, gamma=7, page=16, lo=1, hi=1200, spare=64),
        # the scheduled workload's batch, long contexts among short ones
        dict(name="reserve_sched", op="reserve", B=512, gamma=7, page=16, lo=1, hi=32768, spare=64),
        # a small batch after its verification
        dict(name="commit_few", op="commit", B=9, gamma=7, page=16, lo=30, hi=2500, ends=0),
        # every sixteenth request ends and gives all its pages back
        dict(name="commit_sched", op="commit", B=512, gamma=16, page=16, lo=1, hi=32768, ends=16),
        # a step's new keys and values of one layer
        dict(name="write_step", op="write", B=128, gamma=7, heads=8, d=128, page=16, kv="bf16", order="token"),
        # a long prompt's rows into an 8-bit cache that keeps a head's tokens together
        dict(name="write_prompt_8bit", op="write", B=1, gamma=16380, heads=8, d=128, page=64, kv="e4m3",
             order="head"),
        # one request, one token: the latency of decoding without a draft
        dict(name="attend_one_token", op="attend", B=1, gamma=0, heads_q=32, heads=8, d=128, page=16, lo=1, hi=1201,
             kv="bf16", order="token", causal=True, lse=False),
        # the verify rows of the sample workload's batch, contexts of very different lengths
        dict(name="attend_verify", op="attend", B=128, gamma=7, heads_q=32, heads=8, d=128, page=16, lo=64, hi=8192,
             kv="bf16", order="token", causal=True, lse=False),
        # few requests with long documents, 8-bit cache, log-sum-exps kept for a later join
        dict(name="attend_long_8bit", op="attend", B=6, gamma=7, heads_q=32, heads=4, d=128, page=64, lo=60000,
             hi=131000, kv="e4m3", order="head", causal=True, lse=True),
        # a draft block whose positions see each other, over the draft's own small cache
        dict(name="attend_block", op="attend", B=48, gamma=6, heads_q=16, heads=16, d=64, page=32, lo=0, hi=2047,
             kv="bf16", order="token", causal=False, lse=False),
        # the target's packed logits of the sample workload, a grammar on every other request
        dict(name="constrain_verify", op="constrain", B=128, gamma=7, vocab=151936, logits="bf16", packed=True,
             hist=8192, bias=32, mask=True),
        # the draft's own logits of a small batch, penalised by the history alone
        dict(name="constrain_draft", op="constrain", B=4, gamma=6, vocab=129280, logits="f32", packed=False,
             hist=1500, bias=0, mask=False),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    most = max(work(c)["bytes"] for c in listed())
    op = rng.choice(["reserve", "commit", "write", "attend", "attend", "attend", "constrain", "constrain"])
    c = None
    while c is None or work(c)["bytes"] > most or _plain_values(c) > 6.0e8:
        gamma = rng.choice([0, 1, 3, 5, 7, 7, 16, rng.randint(0, 32)])
        if op in ("reserve", "commit"):
            c = dict(op=op, B=log(1, 1500), gamma=gamma, page=rng.choice([8, 16, 32, 64, 128]), lo=rng.choice([0, 1, 17]),
                     hi=log(20, 32768))
            if op == "reserve":
                c["spare"] = log(1, 2000)
            else:
                c["ends"] = rng.choice([0, 1, 5, 16])
        elif op == "write":
            c = dict(op=op, B=log(1, 512), gamma=rng.choice([gamma, log(1, 16000)]), heads=log(1, 16),
                     d=rng.choice([64, 128, 256]), page=rng.choice([8, 16, 32, 64, 128]), kv=rng.choice(["bf16", "e4m3"]),
                     order=rng.choice(["token", "head"]))
        elif op == "attend":
            heads = log(1, 16)
            hi = log(1, 131072)
            c = dict(op=op, B=log(1, 256), gamma=gamma, heads_q=heads * rng.choice([1, 2, 3, 4, 5, 8, 16]), heads=heads,
                     d=rng.choice([64, 128, 128, 256]), page=rng.choice([8, 16, 32, 64, 128]), lo=rng.randint(0, hi),
                     hi=hi, kv=rng.choice(["bf16", "e4m3"]), order=rng.choice(["token", "head"]),
                     causal=rng.random() < 0.75, lse=rng.random() < 0.5)
        else:
            c = dict(op=op, B=log(1, 256), gamma=gamma, vocab=log(1000, 160000), logits=rng.choice(["bf16", "f32"]),
                     packed=rng.random() < 0.6, hist=log(1, 32768), bias=rng.choice([0, 0, 1, 37, 300]),
                     mask=rng.random() < 0.6)
    return c


def _plain_values(c):
    """Values of the largest array that the plain form needs."""
    if c["op"] == "attend":
        keys = c["B"] * (c["hi"] + c["gamma"] + 1)
        return keys * max(c["heads"] * c["d"], c["heads_q"] * (c["gamma"] + 1))
    if c["op"] == "constrain":
        return c["B"] * (c["gamma"] + 1) * c["vocab"]
    if c["op"] in ("reserve", "commit"):
        return c["B"] * c["hi"] / c["page"] * 4
    return c["B"] * (c["gamma"] + 1) * c["heads"] * c["d"]


def _lengths(c, n):
    """n cache lengths from c["lo"] to c["hi"], even over the logarithm."""
    lo, hi = c["lo"], c["hi"]
    if n == 1:
        return [hi]
    return [lo + int(round((hi - lo + 1) ** (i / (n - 1)))) - 1 for i in range(n)]


def _drafts(c):
    """Verify lengths of the requests: half of them the whole draft."""
    g = c["gamma"]
    return [g if c["B"] == 1 or i % 2 == 0 else (7 * i) % (g + 1) for i in range(c["B"])]


def work(c):
    K = _drafts(c)
    rows = sum(K) + c["B"]
    size = 1 if c.get("kv") == "e4m3" else 2
    if c["op"] == "reserve":
        # K, len, held in; offsets, held out; three numbers and a page id for each row
        return {"bytes": 4.0 * (5 * c["B"] + 4 * rows), "flops": 0.0}
    if c["op"] == "commit":
        # len, accepted, ended, held in; len, held out; page ids moved
        L = _lengths(c, c["B"])
        given = sum(-(-(L[i] + K[i] + 1) // c["page"]) for i in range(c["B"]) if _ends(c, i))
        return {"bytes": 4.0 * (6 * c["B"] + 2 * given), "flops": 0.0}
    if c["op"] == "write":
        return {"bytes": rows * (2.0 * c["heads"] * c["d"] * (2 + size) + 4), "flops": 0.0}
    if c["op"] == "attend":
        L = _lengths(c, c["B"])
        keys = sum(a + b + 1 for a, b in zip(L, K))
        seen = sum((b + 1) * (a + b + 1) - (b * (b + 1) // 2 if c["causal"] else 0) for a, b in zip(L, K))
        n = 2.0 * keys * c["heads"] * c["d"] * size + 4.0 * rows * c["heads_q"] * c["d"]
        n += 4.0 * sum(-(-(a + b + 1) // c["page"]) for a, b in zip(L, K)) + (4.0 * rows * c["heads_q"] if c["lse"] else 0)
        return {"bytes": n, "flops": 4.0 * seen * c["heads_q"] * c["d"]}
    n = rows if c["packed"] else c["B"] * (c["gamma"] + 1)
    b = n * c["vocab"] * (4.0 + (2 if c["logits"] == "bf16" else 4)) + (n * c["vocab"] / 8.0 if c["mask"] else 0)
    return {"bytes": b + 4.0 * sum(_lengths(dict(lo=0, hi=c["hist"]), c["B"])) + 8.0 * c["B"] * c["bias"],
            "flops": 0.0}


def _ends(c, i):
    return bool(c["ends"]) and i % c["ends"] == c["ends"] // 2


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _dealt(c, seed):
    """The case's lengths and verify lengths in the order of the seed."""
    order = np.random.RandomState(seed % (1 << 32)).permutation(c["B"])
    L = np.array(_lengths(c, c["B"]) if "lo" in c else [0] * c["B"], dtype=np.int64)
    return L[order], np.array(_drafts(c), dtype=np.int64)[order], order


def _tables(held, page_ids, cols):
    """Block tables [B][cols] of the first held[b] ids each, -1 behind, and how many ids they take."""
    table = np.full((len(held), cols), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = page_ids[at:at + n]
        at += n
    return table, at


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    r = np.random.RandomState(seed % (1 << 32))
    L, K, order = _dealt(c, seed)
    B, G = c["B"], c["gamma"] + 1
    s = dict(c, G=G)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if c["op"] in ("reserve", "commit"):
        page = c["page"]
        rows = L + K + 1 if c["op"] == "commit" else L
        held = -(-rows // page)
        new = int((-(-(L + K + 1) // page) - held).clip(0).sum())
        n_pages = int(held.sum()) + new + c.get("spare", 8)
        ids = r.permutation(n_pages).astype(np.int32)
        cols = int((-(-(L + K + 1) // page)).max()) + G // page + 2
        table, used = _tables(held, ids, cols)
        free = np.full(n_pages + 1, -1, dtype=np.int32)
        free[:n_pages - used] = ids[used:]
        s.update(n_pages=n_pages, cols=cols, table=_ints(table), held=_ints(held), free=_ints(free),
                 n_free=_ints([n_pages - used]), len=_ints(L), K=_ints(K), rows=int(K.sum()) + B,
                 grow=G // page + 2, held_out=_ints(np.zeros(B)), n_free_out=_ints([0]), len_out=_ints(np.zeros(B)),
                 longest=int(held.max()))
        if c["op"] == "commit":
            s["accepted"] = _ints([r.randint(0, k + 1) for k in K])
            s["ended"] = _ints([_ends(c, i) for i in order])
        else:
            s["out"] = (_ints(np.zeros(B + 1)),) + tuple(_ints(np.zeros(s["rows"])) for _ in range(3))
        return s

    if c["op"] in ("write", "attend"):
        H, d, page = c["heads"], c["d"], c["page"]
        offs = np.concatenate([[0], np.cumsum(K + 1)])
        rows = int(offs[-1])
        held = -(-(L + K + 1) // page)
        n_pages = int(held.sum()) + 3
        ids = r.permutation(n_pages).astype(np.int32)
        shape = (n_pages, page, H, d) if c["order"] == "token" else (n_pages, H, page, d)
        k_scale = v_scale = None
        if c["kv"] == "e4m3":
            # what a calibration leaves: the largest values stand near the type's
            k_scale, v_scale = [(1.0 + 0.25 * torch.rand(H, generator=g, device="cuda")) / 64 for _ in range(2)]

        def cache():
            x = normal(*shape)
            x = x.to(torch.bfloat16) if c["kv"] == "bf16" else (x * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
            return x if c["order"] == "token" else x.permute(0, 2, 1, 3)

        kc, vc = cache(), cache()
        row_req = np.repeat(np.arange(B), K + 1)
        row_i = np.arange(rows) - offs[row_req]
        table, _ = _tables(held, ids, int(held.max()))
        s.update(kc=kc, vc=vc, k_scale=k_scale, v_scale=v_scale, n_rows=rows)
        heads_q = c.get("heads_q", H)
        # query, key and value of a row lie side by side, as the projection leaves them
        qkv = (normal(rows, (heads_q + 2 * H) * d) * 1.5).to(torch.bfloat16)
        s["q"] = qkv[:, :heads_q * d].view(rows, heads_q, d)
        if c["op"] == "write":
            pos = L[row_req] + row_i
            s["slot"] = _ints(table[row_req, pos // page].astype(np.int64) * page + pos % page)
            s["k"], s["v"] = [qkv[:, (heads_q + i * H) * d:(heads_q + (i + 1) * H) * d].view(rows, H, d) for i in (0, 1)]
            return s
        s.update(table=_ints(table), len=_ints(L), K=_ints(K), offs=_ints(offs), row_req=_ints(row_req).long(),
                 row_i=_ints(row_i).long(), scale=d ** -0.5, longest=int((L + K + 1).max()),
                 out=torch.zeros((rows, heads_q, d), dtype=torch.bfloat16, device="cuda"),
                 out_lse=torch.zeros((rows, heads_q), device="cuda") if c["lse"] else None)
        return s

    V = c["vocab"]
    offs = np.concatenate([[0], np.cumsum(K + 1)])
    if not c["packed"]:
        K = np.full(B, G - 1)
        offs = np.arange(B + 1) * G
    rows = int(offs[-1])
    wide = -(-V // 8) * 8                                  # rows start on 16-byte borders
    x = normal(rows, wide) * 3
    x = (x.to(torch.bfloat16) if c["logits"] == "bf16" else x)[:, :V]
    n_hist = np.array(_lengths(dict(lo=0, hi=c["hist"]), B))[order]
    # token ids fall off steeply, so histories repeat themselves
    hist = torch.rand((B, c["hist"]), generator=g, device="cuda").pow_(3).mul_(V).int().clamp_(max=V - 1)
    s.update(x=x, V=V, K=_ints(K) if c["packed"] else None, offs=_ints(offs[:-1]), hist=hist,
             n_hist=_ints(n_hist), n_prompt=_ints(n_hist * r.randint(20, 90) // 100),
             row_req=torch.from_numpy(np.repeat(np.arange(B), K + 1)).cuda(),
             row_i=torch.from_numpy(np.arange(rows) - offs[np.repeat(np.arange(B), K + 1)]).cuda(),
             tokens=None, mask=None, bias=None,
             rep=1 + 0.3 * torch.rand(B, generator=g, device="cuda"),
             freq=0.5 * torch.rand(B, generator=g, device="cuda"), pres=0.5 * torch.rand(B, generator=g, device="cuda"),
             out=torch.empty((rows, wide), device="cuda")[:, :V])
    if c["packed"] and G > 1:
        s["tokens"] = torch.rand((B, G - 1), generator=g, device="cuda").pow_(3).mul_(V).int().clamp_(max=V - 1)
    if c["bias"]:
        ids = torch.rand((B, c["bias"]), generator=g, device="cuda").mul_(V).int().clamp_(max=V - 1).sort(1).values
        s["bias"] = (ids, normal(B, c["bias"]) * 4, _ints(r.randint(0, c["bias"] + 1, B)))
    if c["mask"]:
        # a grammar leaves about one entry in sixteen; the other requests have none
        words = torch.randint(-2 ** 31, 2 ** 31, (4, rows, -(-V // 32)), generator=g, device="cuda")
        words = words[0] & words[1] & words[2] & words[3]
        s["mask"] = torch.where((s["row_req"] % 2 == 0)[:, None], words, torch.full_like(words, -1)).int()
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _RUN_OWN[s["op"]](_context(), s)
    return _RUN_PLAIN[s["op"]](s)


def _own_reserve(ctx, s):
    offs, req, pos, slot = ctx.pages_reserve(s["K"], s["len"], s["table"], s["held"], s["free"][:-1], s["n_free"],
                                             s["page"], s["n_pages"], held_out=s["held_out"],
                                             n_free_out=s["n_free_out"], out=s["out"])
    return {"offs": offs, "req": req, "pos": pos, "slot": slot, "table": s["table"], "held": s["held_out"],
            "n_free": s["n_free_out"]}


def _own_commit(ctx, s):
    ctx.pages_commit(s["len"], s["accepted"], s["table"], s["held"], s["free"][:-1], s["n_free"], s["page"],
                     s["n_pages"], finished=s["ended"], len_out=s["len_out"], held_out=s["held_out"],
                     n_free_out=s["n_free_out"])
    return {"len": s["len_out"], "held": s["held_out"], "n_free": s["n_free_out"], "free": s["free"][:-1]}


def _own_write(ctx, s):
    ctx.cache_write(s["k"], s["v"], s["slot"], s["kc"], s["vc"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"k": s["kc"], "v": s["vc"]}


def _own_attend(ctx, s):
    ctx.attend(s["q"], s["kc"], s["vc"], s["table"], s["len"], s["G"] - 1, K=s["K"], t_offsets=s["offs"],
               causal=s["causal"], scale=s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"],
               lse=s["out_lse"])
    return {"out": s["out"], "lse": s["out_lse"]}


def _own_constrain(ctx, s):
    G, V = s["G"], s["V"]
    how = dict(hist=s["hist"], n_hist=s["n_hist"], n_prompt=s["n_prompt"], rep=s["rep"], freq=s["freq"],
               pres=s["pres"], bias=s["bias"])
    if s["packed"]:
        ctx.constrain(s["x"], G, K=s["K"], t_offsets=s["offs"], tokens=s["tokens"], mask=s["mask"], out=s["out"], **how)
    else:
        mask = None if s["mask"] is None else s["mask"].view(s["B"], G, -1)
        ctx.constrain(s["x"].unflatten(0, (s["B"], G)), G, tokens=s["tokens"], mask=mask,
                      out=s["out"].unflatten(0, (s["B"], G)), **how)
    return {"out": s["out"]}


def _plain_reserve(s):
    page, rows = s["page"], s["rows"]
    K, L, held = s["K"].long(), s["len"].long(), s["held"].long()
    ends = torch.cumsum(K + 1, 0)
    offs = torch.cat([torch.zeros_like(ends[:1]), ends])
    need = torch.maximum(held, (L + K + page) // page)
    extra = need - held
    before = torch.cumsum(extra, 0) - extra
    j = torch.arange(s["grow"], device="cuda")[None]
    ids = s["free"].long()[(s["n_free"].long() - 1 - before[:, None] - j).clamp(min=0)]
    at = held[:, None] + j
    s["table"].scatter_(1, at, torch.where(j < extra[:, None], ids, s["table"].long().gather(1, at)).int())
    row = torch.arange(rows, device="cuda")
    req = torch.searchsorted(ends, row, right=True)
    pos = L[req] + row - offs[req]
    slot = s["table"].long()[req, pos // page] * page + pos % page
    return {"offs": offs.int(), "req": req.int(), "pos": pos.int(), "slot": slot.int(), "table": s["table"],
            "held": need.int(), "n_free": s["n_free"] - extra.sum().int()}


def _plain_commit(s):
    page, held = s["page"], s["held"].long()
    ended = s["ended"] != 0
    L = torch.where(ended, 0, s["len"].long() + s["accepted"].long() + 1)
    keep = (L + page - 1) // page
    given = held - keep
    before = torch.cumsum(given, 0) - given
    j = torch.arange(s["longest"], device="cuda")[None]
    ids = s["table"].long().gather(1, (keep[:, None] + j).clamp(max=s["cols"] - 1))
    # what is not given back goes to the slack entry behind the list
    to = torch.where(j < given[:, None], s["n_free"].long() + before[:, None] + j, s["n_pages"])
    s["free"].scatter_(0, to.reshape(-1), ids.int().reshape(-1))
    return {"len": L.int(), "held": keep.int(), "n_free": s["n_free"] + given.sum().int(), "free": s["free"][:-1]}


def _to_8bit(x, scale):
    """x / scale at the nearest e4m3 value (ties to even, the largest value kept), in 64 bits: a quotient rounded to 32
    bits first could come to stand on a border."""
    q = (x.double() / scale.double()[:, None]).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(q / step) * step).float().to(torch.float8_e4m3fn)


def _plain_write(s):
    slot = s["slot"].long()
    k, v = s["k"], s["v"]
    kc, vc = s["kc"], s["vc"]
    if s["kv"] == "e4m3":
        k, v = _to_8bit(k, s["k_scale"]).view(torch.uint8), _to_8bit(v, s["v_scale"]).view(torch.uint8)
        kc, vc = kc.view(torch.uint8), vc.view(torch.uint8)
    at = (slot // s["page"], slot % s["page"])
    kc.index_put_(at, k)
    vc.index_put_(at, v)
    return {"k": s["kc"], "v": s["vc"]}


def _plain_attend(s):
    B, G, H, d, page, n = s["B"], s["G"], s["heads"], s["d"], s["page"], s["longest"]
    group = s["heads_q"] // H
    L, K = s["len"].long(), s["K"].long()
    t = torch.arange(n, device="cuda")
    ids = s["table"].long()[:, t // page].clamp(min=0)
    i = torch.arange(G, device="cuda")
    rows = (s["offs"].long()[:-1, None] + i).clamp(max=s["n_rows"] - 1)
    q = s["q"][rows].float().view(B, G, H, group, d).permute(0, 2, 1, 3, 4).reshape(B * H, G * group, d)
    k = s["kc"][ids, t % page].float().permute(0, 2, 3, 1).reshape(B * H, d, n)
    scores = torch.matmul(q, k).mul_(s["scale"]).view(B, H, G, group, n)
    del k
    if s["k_scale"] is not None:
        scores *= s["k_scale"][:, None, None, None]
    last = L[:, None] + (i if s["causal"] else K[:, None].expand(B, G))
    scores.masked_fill_(t > last[:, None, :, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(top).exp_()
    total = p.sum(-1)
    v = s["vc"][ids, t % page].float().permute(0, 2, 1, 3).reshape(B * H, n, d)
    o = torch.matmul(p.view(B * H, G * group, n), v).view(B, H, G, group, d) / total[..., None]
    if s["v_scale"] is not None:
        o *= s["v_scale"][:, None, None, None]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, G, s["heads_q"], d)[s["row_req"], s["row_i"]]
    lse = None
    if s["lse"]:
        lse = (top[..., 0] + total.log()).permute(0, 2, 1, 3).reshape(B, G, s["heads_q"])[s["row_req"], s["row_i"]]
    return {"out": o.to(torch.bfloat16), "lse": lse}


def _plain_constrain(s):
    B, V, req, i = s["B"], s["V"], s["row_req"], s["row_i"]
    at = torch.arange(s["hist"].shape[1], device="cuda")[None]
    hist = s["hist"].long()
    told = at < s["n_hist"][:, None]
    wrote = told & (at >= s["n_prompt"][:, None])
    count = torch.zeros((B, V), device="cuda").scatter_add_(1, hist, wrote.float())
    seen = torch.zeros((B, V), device="cuda").scatter_add_(1, hist, told.float())
    count, seen = count[req], seen[req]
    if s["tokens"] is not None:
        drafted = s["tokens"].long()[req]
        one = (torch.arange(drafted.shape[1], device="cuda")[None] < i[:, None]).float()
        count.scatter_add_(1, drafted, one)
        seen.scatter_add_(1, drafted, one)
    x = s["x"].float()
    rep = s["rep"][req, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["freq"][req, None] * count - s["pres"][req, None] * (count > 0).float()
    if s["bias"] is not None:
        ids, values, n = s["bias"]
        in_use = torch.arange(ids.shape[1], device="cuda")[None] < n[:, None]
        x += torch.zeros((B, V), device="cuda").scatter_add_(1, ids.long(), torch.where(in_use, values, 0.0))[req]
    x = x.clamp(min=MASKED)
    if s["mask"] is not None:
        v = torch.arange(V, device="cuda")
        x = torch.where((s["mask"][:, v // 32] >> (v % 32).int()) & 1 != 0, x, MASKED)
    return {"out": x}


_RUN_OWN = {"reserve": _own_reserve, "commit": _own_commit, "write": _own_write, "attend": _own_attend,
            "constrain": _own_constrain}
_RUN_PLAIN = {"reserve": _plain_reserve, "commit": _plain_commit, "write": _plain_write, "attend": _plain_attend,
              "constrain": _plain_constrain}


# ---------------------------------------------------------------------------
# The definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "reserve":
        return _exact_reserve(s)
    if c["op"] == "commit":
        return _exact_commit(s)
    if c["op"] == "write":
        return _exact_write(s)
    if c["op"] == "attend":
        return _exact_attend(s)
    return _exact_constrain(s)


def _exact_reserve(s):
    K, L, held, free = [s[k].cpu().numpy().copy() for k in ("K", "len", "held", "free")]
    table, top = s["table"].cpu().numpy().copy(), int(s["n_free"])
    offs, req, pos, slot = [0], [], [], []
    for b in range(s["B"]):
        while held[b] * s["page"] < L[b] + K[b] + 1:
            top -= 1
            table[b, held[b]] = free[top]
            held[b] += 1
        for p in range(L[b], L[b] + K[b] + 1):
            req.append(b)
            pos.append(p)
            slot.append(int(table[b, p // s["page"]]) * s["page"] + p % s["page"])
        offs.append(len(req))
    return {k: torch.from_numpy(np.array(v, dtype=np.int32)) for k, v in
            dict(offs=offs, req=req, pos=pos, slot=slot, table=table, held=held, n_free=[top]).items()}


def _exact_commit(s):
    L, acc, ended, held, free = [s[k].cpu().numpy().copy() for k in ("len", "accepted", "ended", "held", "free")]
    table, top = s["table"].cpu().numpy(), int(s["n_free"])
    for b in range(s["B"]):
        L[b] = 0 if ended[b] else L[b] + acc[b] + 1
        keep = math.ceil(L[b] / s["page"])
        for p in range(keep, held[b]):
            free[top] = table[b, p]
            top += 1
        held[b] = keep
    return {k: torch.from_numpy(np.array(v, dtype=np.int32)) for k, v in
            dict(len=L, held=held, n_free=[top], free=free[:-1]).items()}


def _exact_write(s):
    slot = s["slot"].long()
    levels = None
    if s["kv"] == "e4m3":
        codes = torch.arange(127, dtype=torch.uint8, device="cuda")      # 0 .. 448, increasing
        levels = codes.view(torch.float8_e4m3fn).double()
    got = {}
    for name, rows, cache, scale in (("k", s["k"], s["kc"], s["k_scale"]), ("v", s["v"], s["vc"], s["v_scale"])):
        x = rows.double()
        if levels is not None:
            x = x / scale.double()[None, :, None]
            a = x.abs()
            above = torch.searchsorted(levels, a.contiguous()).clamp(max=126)
            below = (above - 1).clamp(min=0)
            up, down = levels[above] - a, a - levels[below]
            # on a border the code with an even last bit
            pick = torch.where((up < down) | ((up == down) & (above % 2 == 0)), above, below)
            x = torch.where(a > 448, torch.full_like(a, 448.0), levels[pick]) * torch.sign(x)
        full = cache.double().contiguous()
        full[slot // s["page"], slot % s["page"]] = x
        got[name] = full
    return got


def _exact_attend(s):
    page, H, d = s["page"], s["heads"], s["d"]
    group = s["heads_q"] // H
    L, K, offs, table = [s[k].cpu().numpy() for k in ("len", "K", "offs", "table")]
    out = torch.zeros((s["n_rows"], s["heads_q"], d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["n_rows"], s["heads_q"]), dtype=torch.float64, device="cuda")
    for b in range(s["B"]):
        n, m = int(L[b] + K[b] + 1), int(K[b]) + 1
        pages = torch.from_numpy(table[b, :-(-n // page)].astype(np.int64)).cuda()

        def keys(cache, scale):
            x = cache[pages].reshape(-1, H, d)[:n].double()
            return x if scale is None else x * scale.double()[None, :, None]

        k, v = keys(s["kc"], s["k_scale"]), keys(s["vc"], s["v_scale"])
        for h in range(H):
            q = s["q"][offs[b]:offs[b] + m, h * group:(h + 1) * group].double().reshape(m * group, d)
            e = (q @ k[:, h].t().contiguous()) * s["scale"]
            if s["causal"]:
                own_row = torch.arange(m * group, device="cuda") // group
                e[torch.arange(n, device="cuda")[None] > int(L[b]) + own_row[:, None]] = -math.inf
            z = torch.logsumexp(e, 1)
            o = torch.exp(e - z[:, None]) @ v[:, h].contiguous()
            out[offs[b]:offs[b] + m, h * group:(h + 1) * group] = o.view(m, group, d)
            lse[offs[b]:offs[b] + m, h * group:(h + 1) * group] = z.view(m, group)
    return {"out": out, "lse": lse if s["lse"] else None}


def _exact_constrain(s):
    V, row = s["V"], 0
    req = s["row_req"].cpu().numpy()
    n_hist, n_prompt = s["n_hist"].cpu().numpy(), s["n_prompt"].cpu().numpy()
    out = torch.empty((len(req), V), dtype=torch.float64, device="cuda")
    for b in range(s["B"]):
        h = s["hist"][b].long()
        count = torch.bincount(h[n_prompt[b]:n_hist[b]], minlength=V).double()
        prompt = torch.bincount(h[:min(n_prompt[b], n_hist[b])], minlength=V) > 0
        bias = torch.zeros(V, dtype=torch.float64, device="cuda")
        if s["bias"] is not None:
            n = int(s["bias"][2][b])
            bias.index_add_(0, s["bias"][0][b, :n].long(), s["bias"][1][b, :n].double())
        rep, freq, pres = [s[k][b].double() for k in ("rep", "freq", "pres")]
        i = 0
        while row < len(req) and req[row] == b:
            if i > 0 and s["tokens"] is not None:
                count[s["tokens"][b, i - 1].long()] += 1
            x = s["x"][row].double()
            hit = prompt | (count > 0)
            x = torch.where(hit & (x > 0), x / rep, torch.where(hit, x * rep, x))
            x = x - freq * count - pres * (count > 0) + bias
            x = torch.clamp(x, min=MASKED)
            if s["mask"] is not None:
                bits = s["mask"][row].view(torch.uint8)[:, None] >> torch.arange(8, dtype=torch.uint8, device="cuda")
                x[(bits.reshape(-1)[:V] & 1) == 0] = MASKED
            out[row] = x
            row += 1
            i += 1
    return {"out": out}
