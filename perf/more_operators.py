"""Timed cases of the operators around a 4-bit cache and of rotary positions.

A step's packed rows come out of the projection as query, key and value; before
they attend, queries and keys are rotated by their positions, and keys and
values go into the paged cache.  Timed here:

  rope    queries and keys rotated (both layouts, whole heads or part of them,
          plain and stretched frequencies)
  store   the same with keys and values going into their cache slots: bf16,
          e4m3, or MXFP4 (e2m1 values, a power of two for each 32 of them);
          rot = 0: keys that are rotated already.  A 4-bit cache's rows are
          read back, as a prompt's next piece reads them
  read    rows of a cache back as bf16
  attend  attention of packed rows over an MXFP4 cache

``run`` computes them in elementary torch operations (``own`` false) or calls
the library (``own`` true).  Lengths and verify lengths are a fixed multiset of
the case, dealt to the requests by the seed, so that the work of a case is
known without its inputs.
"""
import math

import numpy as np
import torch

own = False

SIZE = {"bf16": 2.0, "e4m3": 1.0, "mxfp4": 17.0 / 32}
THETA = 500000.0
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
        # one request, one token: the latency of decoding without a draft
        dict(name="rope_one", op="rope", rows=1, run=1, heads_q=32, heads=8, d=128, rot=128, layout="half",
             scaling="none", by=1, far=8192),
        # the verify rows of a batch, a quarter of each wide head rotated, neighbouring values paired
        dict(name="rope_part", op="rope", rows=1021, run=8, heads_q=16, heads=4, d=256, rot=64, layout="interleaved",
             scaling="ntk", by=4, far=32768),
        # a long prompt far behind the trained context
        dict(name="rope_prompt", op="rope", rows=16381, run=16381, heads_q=32, heads=8, d=128, rot=128, layout="half",
             scaling="yarn", by=16, far=131072),
        # a step's rows of the sample workload's batch into a bf16 cache
        dict(name="store_step", op="store", rows=821, run=8, heads_q=32, heads=8, d=128, rot=128, layout="half",
             scaling="none", by=1, far=8192, page=16, kv="bf16", order="token"),
        # a piece of a prompt into a 4-bit cache that keeps a head's tokens together, and read back
        dict(name="store_prompt_4bit", op="store", rows=8190, run=8190, heads_q=32, heads=8, d=128, rot=128,
             layout="half", scaling="linear", by=4, far=65536, page=64, kv="mxfp4", order="head"),
        # keys that were rotated before: a small batch's rows into a 4-bit cache, and read back
        dict(name="store_few_4bit", op="store", rows=63, run=7, heads_q=16, heads=16, d=64, rot=0, layout="half",
             scaling="none", by=1, far=2048, page=32, kv="mxfp4", order="token"),
        # a shared prefix of a 4-bit cache, for a prompt's next piece
        dict(name="read_prefix_4bit", op="read", rows=32749, heads=8, d=128, page=16, kv="mxfp4", order="token"),
        # a short context out of an 8-bit cache
        dict(name="read_short_8bit", op="read", rows=197, heads=4, d=256, page=64, kv="e4m3", order="head"),
        # one request, one token over the 4-bit cache
        dict(name="attend_one_token", op="attend", B=1, gamma=0, heads_q=32, heads=8, d=128, page=16, lo=1, hi=1201,
             order="token", causal=True, lse=False),
        # the verify rows of the sample workload's batch, contexts of very different lengths
        dict(name="attend_verify", op="attend", B=128, gamma=7, heads_q=32, heads=8, d=128, page=16, lo=64, hi=8192,
             order="token", causal=True, lse=False),
        # few requests with long documents, log-sum-exps kept for a later join
        dict(name="attend_long", op="attend", B=6, gamma=7, heads_q=32, heads=4, d=128, page=64, lo=60000,
             hi=131000, order="head", causal=True, lse=True),
        # a draft block whose positions see each other, over the draft's own small cache
        dict(name="attend_block", op="attend", B=48, gamma=6, heads_q=16, heads=16, d=64, page=32, lo=0, hi=2047,
             order="token", causal=False, lse=False),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    most = max(work(c)["bytes"] for c in listed())
    op = rng.choice(["rope", "rope", "store", "store", "store", "read", "attend", "attend", "attend"])
    c = None
    while c is None or work(c)["bytes"] > most or _plain_values(c) > 6.0e8:
        heads = log(1, 16)
        d = rng.choice([64, 128, 128, 256])
        page, order = rng.choice([8, 16, 32, 64, 128]), rng.choice(["token", "head"])
        if op == "attend":
            hi = log(1, 131072)
            c = dict(op=op, B=log(1, 256), gamma=rng.choice([0, 1, 3, 5, 7, 7, 16, rng.randint(0, 32)]),
                     heads_q=heads * rng.choice([1, 2, 3, 4, 5, 8, 16]), heads=heads, d=d, page=page,
                     lo=rng.randint(0, hi), hi=hi, order=order, causal=rng.random() < 0.75, lse=rng.random() < 0.5)
            continue
        rows = log(1, 40000)
        if op == "read":
            c = dict(op=op, rows=rows, heads=heads, d=d, page=page, kv=rng.choice(["bf16", "e4m3", "mxfp4", "mxfp4"]),
                     order=order)
            continue
        if op == "rope":
            d = rng.choice([64, 80, 96, 128, 128, 192, 256])
        by = rng.choice([2, 4, 8, 16])
        c = dict(op=op, rows=rows, run=rng.choice([1, 2, 8, 8, 33, rows]), heads_q=heads * rng.choice([1, 2, 4, 5, 8]),
                 heads=heads, d=d, rot=rng.choice([d, d, d, 32, 48, 64]), layout=rng.choice(["half", "interleaved"]),
                 scaling=rng.choice(["none", "linear", "ntk", "yarn"]), by=by, far=log(40000, 1000000))
        if c["scaling"] == "none":
            c["by"] = 1
        if op == "store":
            c.update(page=page, kv=rng.choice(["bf16", "e4m3", "mxfp4", "mxfp4"]), order=order)
            if c["kv"] == "mxfp4" and rng.random() < 0.3:
                c["rot"] = 0
    return c


def _plain_values(c):
    """Values of the largest array that the plain form needs."""
    if c["op"] == "attend":
        keys = c["B"] * (c["hi"] + c["gamma"] + 1)
        return keys * max(c["heads"] * c["d"], c["heads_q"] * (c["gamma"] + 1))
    return 2.0 * c["rows"] * c.get("heads_q", c["heads"]) * c["d"]


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
    if c["op"] == "attend":
        K, L = _drafts(c), _lengths(c, c["B"])
        rows = sum(K) + c["B"]
        keys = sum(a + b + 1 for a, b in zip(L, K))
        seen = sum((b + 1) * (a + b + 1) - (b * (b + 1) // 2 if c["causal"] else 0) for a, b in zip(L, K))
        n = 2.0 * keys * c["heads"] * c["d"] * SIZE["mxfp4"] + 4.0 * rows * c["heads_q"] * c["d"]
        n += 4.0 * sum(-(-(a + b + 1) // c["page"]) for a, b in zip(L, K)) + (4.0 * rows * c["heads_q"] if c["lse"] else 0)
        return {"bytes": n, "flops": 4.0 * seen * c["heads_q"] * c["d"]}
    rows, kv = c["rows"], c["heads"] * c["d"]
    read = rows * (2.0 * kv * (SIZE[c.get("kv", "bf16")] + 2) + 4)
    if c["op"] == "read":
        return {"bytes": read, "flops": 0.0}
    q = c["heads_q"] * c["d"]
    turned = 3.0 * rows * (c["heads_q"] + c["heads"]) * c["rot"]
    if c["op"] == "rope":
        return {"bytes": rows * (4.0 * (q + kv) + 4) + 4.0 * c["rot"], "flops": turned}
    n = rows * (2.0 * kv * (2 + SIZE[c["kv"]]) + 4) + (rows * (4.0 * q + 4) + 4.0 * c["rot"] if c["rot"] else 0.0)
    return {"bytes": n + (read if c["kv"] == "mxfp4" else 0.0), "flops": turned}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _frequencies(c):
    """Radians a position, for every pair, and the factor of sines and cosines: what a program works out once."""
    rot, by = c["rot"], float(c["by"])
    i = torch.arange(rot // 2, dtype=torch.float64)
    theta = THETA * by ** (rot / (rot - 2.0)) if c["scaling"] == "ntk" else THETA
    f = torch.exp(-2.0 * i / rot * math.log(theta))
    if c["scaling"] == "linear":
        return f / by, 1.0
    if c["scaling"] != "yarn":
        return f, 1.0
    # pairs that turn often within the trained context stay, those that turn less than once are stretched
    trained = c["far"] / by
    at = [rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(THETA)) for turns in (32.0, 1.0)]
    lo, hi = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f / by * ramp + f * (1 - ramp), 0.1 * math.log(by) + 1.0


def _places(r, rows, run, page, far, spare):
    """Positions of runs of neighbouring tokens, their slots in pages of any order, and how many pages there are."""
    n = -(-rows // run)
    first = r.randint(0, max(1, far - run), n).astype(np.int64)
    lead = first % page
    length = np.minimum(run, rows - run * np.arange(n))
    pages = (lead + length + page - 1) // page
    begin = np.concatenate([[0], np.cumsum(pages)])
    n_pages = int(((length + 2 * page - 2) // page).sum()) + spare      # enough wherever the runs begin
    ids = r.permutation(n_pages)
    which = np.repeat(np.arange(n), length)
    i = np.arange(rows) - run * which
    at = lead[which] + i
    return first[which] + i, ids[begin[which] + at // page] * page + at % page, n_pages


def _quantise(x):
    """MXFP4 codes and scale bytes of x [..., d] (float32 or float64): codes [..., d], bytes [..., d / 32]."""
    blocks = x.unflatten(-1, (-1, 32))
    m, e = torch.frexp(blocks.abs().amax(-1))
    # the least power whose 7 holds the largest: its own rounding is then no more than half a step either
    e = torch.where(m == 0, -120, (e - 3 + (m > 0.875).to(e.dtype)).clamp(-120, 125))
    q = blocks * torch.exp2(-e[..., None].to(x.dtype))
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(x.dtype)
    a = (torch.round(a / step) * step).clamp(max=6)
    code = torch.where(a <= 2, 2 * a, torch.where(a <= 4, a + 2, 7.0)).to(torch.uint8) | (torch.signbit(blocks).to(torch.uint8) << 3)
    return code.flatten(-2), (e + 127).to(torch.uint8)


def _packed(code):
    """Two codes a byte, the first in the low half."""
    return code[..., 0::2] | (code[..., 1::2] << 4)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    r = np.random.RandomState(seed % (1 << 32))
    H, d = c["heads"], c["d"]
    s = dict(c)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def caches(n_pages, kv):
        """Keys and values of a cache in use, and their scales."""
        page, got, scales = c["page"], [], []
        for _ in range(2):
            shape = (n_pages, page, H) if c["order"] == "token" else (n_pages, H, page)
            x = normal(*shape, d)
            # heads of different strength
            x *= (0.5 + torch.rand(H, generator=g, device="cuda") * 2).view((H, 1) if c["order"] == "token" else (H, 1, 1))
            scale = None
            if kv == "bf16":
                x = x.to(torch.bfloat16)
            elif kv == "e4m3":
                # what a calibration leaves: the largest values stand near the type's
                scale = (1.0 + 0.25 * torch.rand(H, generator=g, device="cuda")) / 32
                x = (x * 30).clamp(-448, 448).to(torch.float8_e4m3fn)
            else:
                code, scale = _quantise(x)
                x = _packed(code)
                # the scales of a head's tokens lie together, whatever the order of the cache
                scale = scale if c["order"] == "head" else scale.permute(0, 2, 1, 3).contiguous()
            got.append(x if c["order"] == "token" else x.permute(0, 2, 1, 3))
            scales.append(scale)
        s.update(kc=got[0], vc=got[1], k_scale=scales[0], v_scale=scales[1])

    if c["op"] == "attend":
        order = r.permutation(c["B"])
        L, K = np.array(_lengths(c, c["B"]), dtype=np.int64)[order], np.array(_drafts(c), dtype=np.int64)[order]
        offs = np.concatenate([[0], np.cumsum(K + 1)])
        rows, page = int(offs[-1]), c["page"]
        held = -(-(L + K + 1) // page)
        n_pages = int(held.sum()) + 3
        ids = r.permutation(n_pages)
        table = np.full((c["B"], int(held.max())), -1, dtype=np.int32)
        table[np.arange(table.shape[1])[None] < held[:, None]] = ids[:int(held.sum())]
        caches(n_pages, "mxfp4")
        row_req = np.repeat(np.arange(c["B"]), K + 1)
        qkv = (normal(rows, (c["heads_q"] + 2 * H) * d) * 1.5).to(torch.bfloat16)
        s.update(q=qkv[:, :c["heads_q"] * d].view(rows, c["heads_q"], d), n_rows=rows, G=c["gamma"] + 1, table=_ints(table),
                 len=_ints(L), K=_ints(K), offs=_ints(offs), row_req=_ints(row_req).long(),
                 row_i=_ints(np.arange(rows) - offs[row_req]).long(), scale=d ** -0.5, longest=int((L + K + 1).max()),
                 out=torch.zeros((rows, c["heads_q"], d), dtype=torch.bfloat16, device="cuda"),
                 out_lse=torch.zeros((rows, c["heads_q"]), device="cuda") if c["lse"] else None)
        return s

    rows = c["rows"]
    pos, slot, n_pages = _places(r, rows, c.get("run", rows), c.get("page", 16), c.get("far", 1), 3)
    if c["op"] != "rope":
        caches(n_pages, c["kv"])
        s["slot"] = _ints(slot)
        s["back"] = [torch.zeros((rows, H, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    if c["op"] == "read":
        return s
    # query, key and value of a row lie side by side, as the projection leaves them
    hq = c["heads_q"]
    qkv = (normal(rows, (hq + 2 * H) * d) * 1.5).to(torch.bfloat16)
    s["q"], s["k"], s["v"] = [x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, H * d, H * d], 1)]
    s["pos"] = _ints(pos)
    if c["rot"]:
        f, factor = _frequencies(c)
        s.update(freq=f.cuda(), factor=factor, q_out=torch.zeros((rows, hq, d), dtype=torch.bfloat16, device="cuda"))
    if c["op"] == "rope":
        s["k_out"] = torch.zeros((rows, H, d), dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _RUN_OWN[s["op"]](_context(), s)
    return _RUN_PLAIN[s["op"]](s)


def _own_rope(ctx, s):
    ctx.rope(s["q"], s["k"], s["pos"], s["freq"], interleaved=s["layout"] == "interleaved", factor=s["factor"],
             q_out=s["q_out"], k_out=s["k_out"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_store(ctx, s):
    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if s["rot"]:
        ctx.rope_write(s["q"], s["k"], s["v"], s["pos"], s["slot"], s["freq"], s["kc"], s["vc"],
                       interleaved=s["layout"] == "interleaved", factor=s["factor"], q_out=s["q_out"], **scales)
    else:
        ctx.cache_write(s["k"], s["v"], s["slot"], s["kc"], s["vc"], **scales)
    q = s["q_out"] if s["rot"] else None
    if s["kv"] != "mxfp4":
        return {"q": q, "k": s["kc"], "v": s["vc"]}
    ctx.cache_read(s["kc"], s["vc"], s["slot"], out=s["back"], **scales)
    return {"q": q, "k": s["back"][0], "v": s["back"][1]}


def _own_read(ctx, s):
    ctx.cache_read(s["kc"], s["vc"], s["slot"], k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["back"])
    return {"k": s["back"][0], "v": s["back"][1]}


def _own_attend(ctx, s):
    ctx.attend(s["q"], s["kc"], s["vc"], s["table"], s["len"], s["G"] - 1, K=s["K"], t_offsets=s["offs"],
               causal=s["causal"], scale=s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"],
               lse=s["out_lse"])
    return {"out": s["out"], "lse": s["out_lse"]}


def _turn(s, x):
    """x rotated by the rows' positions, in 64 bits: a far position's angle needs them, and so does a value that a
    cache of few bits rounds."""
    rot = s["rot"]
    a = s["pos"].double()[:, None] * s["freq"]
    cos, sin = (a.cos() * s["factor"])[:, None], (a.sin() * s["factor"])[:, None]
    y = x.double()
    if s["layout"] == "half":
        x0, x1 = y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone()
        y[..., :rot // 2] = x0 * cos - x1 * sin
        y[..., rot // 2:rot] = x1 * cos + x0 * sin
    else:
        x0, x1 = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
        y[..., 0:rot:2] = x0 * cos - x1 * sin
        y[..., 1:rot:2] = x1 * cos + x0 * sin
    return y


def _plain_rope(s):
    return {"q": _turn(s, s["q"]).to(torch.bfloat16), "k": _turn(s, s["k"]).to(torch.bfloat16)}


def _to_8bit(x, scale):
    """x / scale at the nearest e4m3 value (ties to even, the largest value kept), in 64 bits: a quotient rounded to 32
    bits first could come to stand on a border."""
    q = (x.double() / scale.double()[:, None]).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(q / step) * step).float().to(torch.float8_e4m3fn)


def _plain_store(s):
    slot = s["slot"].long()
    at = (slot // s["page"], slot % s["page"])
    q, k, v = None, s["k"], s["v"]
    if s["rot"]:
        q, k = _turn(s, s["q"]).to(torch.bfloat16), _turn(s, k)
    if s["kv"] == "bf16":
        s["kc"].index_put_(at, k.to(torch.bfloat16))
        s["vc"].index_put_(at, v)
        return {"q": q, "k": s["kc"], "v": s["vc"]}
    if s["kv"] == "e4m3":
        s["kc"].view(torch.uint8).index_put_(at, _to_8bit(k, s["k_scale"]).view(torch.uint8))
        s["vc"].view(torch.uint8).index_put_(at, _to_8bit(v, s["v_scale"]).view(torch.uint8))
        return {"q": q, "k": s["kc"], "v": s["vc"]}
    for x, cache, scale in ((k, s["kc"], s["k_scale"]), (v, s["vc"], s["v_scale"])):
        code, byte = _quantise(x.double())
        cache.index_put_(at, _packed(code))
        scale[at[0], :, at[1]] = byte
    return {"q": q, **_plain_read(s)}


def _decoded(cache, scale, page, place):
    """Values in 32 bits of an MXFP4 cache's tokens at (page, place), which may be tables: [..., heads, d]."""
    byte = cache[page, place]
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).int()
    mag = code & 7
    x = torch.where(mag < 5, mag * 0.5, torch.where(mag < 7, mag - 2.0, 6.0))
    x = torch.where(code > 7, -x, x)
    power = torch.exp2(scale[page.unsqueeze(-1), torch.arange(scale.shape[1], device="cuda"), place.unsqueeze(-1)].float() - 127)
    return (x.unflatten(-1, (-1, 32)) * power[..., None]).flatten(-2)


def _plain_read(s):
    slot = s["slot"].long()
    at = (slot // s["page"], slot % s["page"])
    got = {}
    for name, cache, scale in (("k", s["kc"], s["k_scale"]), ("v", s["vc"], s["v_scale"])):
        if s["kv"] == "mxfp4":
            got[name] = _decoded(cache, scale, *at).to(torch.bfloat16)
        elif s["kv"] == "e4m3":
            got[name] = (cache.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scale[:, None]).to(torch.bfloat16)
        else:
            got[name] = cache[at]
    return got


def _plain_attend(s):
    B, G, H, d, page, n = s["B"], s["G"], s["heads"], s["d"], s["page"], s["longest"]
    group = s["heads_q"] // H
    L, K = s["len"].long(), s["K"].long()
    t = torch.arange(n, device="cuda")
    ids = s["table"].long()[:, t // page].clamp(min=0)
    place = (t % page)[None].expand(B, n)
    i = torch.arange(G, device="cuda")
    rows = (s["offs"].long()[:-1, None] + i).clamp(max=s["n_rows"] - 1)
    q = s["q"][rows].float().view(B, G, H, group, d).permute(0, 2, 1, 3, 4).reshape(B * H, G * group, d)
    k = _decoded(s["kc"], s["k_scale"], ids, place).permute(0, 2, 3, 1).reshape(B * H, d, n)
    scores = torch.matmul(q, k).mul_(s["scale"]).view(B, H, G, group, n)
    del k
    last = L[:, None] + (i if s["causal"] else K[:, None].expand(B, G))
    scores.masked_fill_(t > last[:, None, :, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(top).exp_()
    total = p.sum(-1)
    v = _decoded(s["vc"], s["v_scale"], ids, place).permute(0, 2, 1, 3).reshape(B * H, n, d)
    o = torch.matmul(p.view(B * H, G * group, n), v).view(B, H, G, group, d) / total[..., None]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, G, s["heads_q"], d)[s["row_req"], s["row_i"]]
    lse = None
    if s["lse"]:
        lse = (top[..., 0] + total.log()).permute(0, 2, 1, 3).reshape(B, G, s["heads_q"])[s["row_req"], s["row_i"]]
    return {"out": o.to(torch.bfloat16), "lse": lse}


_RUN_OWN = {"rope": _own_rope, "store": _own_store, "read": _own_read, "attend": _own_attend}
_RUN_PLAIN = {"rope": _plain_rope, "store": _plain_store, "read": _plain_read, "attend": _plain_attend}


# ---------------------------------------------------------------------------
# The definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        return {"q": _exact_turn(c, s, s["q"]), "k": _exact_turn(c, s, s["k"])}
    if c["op"] == "store":
        return _exact_store(c, s)
    if c["op"] == "read":
        return {"k": _exact_rows(c, s["kc"], s["k_scale"], s["slot"]), "v": _exact_rows(c, s["vc"], s["v_scale"], s["slot"])}
    return _exact_attend(s)


def _exact_turn(c, s, x):
    """Pairs as complex numbers, times c e^(i pos f)."""
    rot, by, f, factor = c["rot"], float(c["by"]), [], 1.0
    for j in range(rot // 2):
        plain = THETA ** (-2.0 * j / rot)
        if c["scaling"] == "linear":
            plain /= by
        elif c["scaling"] == "ntk":
            plain = (THETA * by ** (rot / (rot - 2))) ** (-2.0 * j / rot)
        elif c["scaling"] == "yarn":
            def pair_of(turns):
                return rot * math.log(c["far"] / by / (turns * 2 * math.pi)) / (2 * math.log(THETA))
            lo, hi = max(math.floor(pair_of(32)), 0), min(math.ceil(pair_of(1)), rot - 1)
            w = min(1.0, max(0.0, (j - lo) / max(hi - lo, 0.001)))
            plain = plain * (1 - w) + plain * w / by
            factor = 1.0 + math.log(by) / 10
        f.append(plain)
    angle = torch.outer(s["pos"].double(), torch.tensor(f, dtype=torch.float64, device="cuda"))
    y = x.double().clone()
    part = y[..., :rot]
    pairs = part.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if c["layout"] == "half" else part.unflatten(-1, (rot // 2, 2))
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(angle, factor), angle)[:, None]
    z = torch.view_as_real(z)
    y[..., :rot] = (z.transpose(-1, -2) if c["layout"] == "half" else z).flatten(-2)
    return y


def _nearest(levels, a):
    """The level nearest each a >= 0, on a border the one with an even number, the last one kept."""
    up = torch.searchsorted(levels, a.contiguous()).clamp(max=len(levels) - 1)
    down = (up - 1).clamp(min=0)
    over, under = levels[up] - a, a - levels[down]
    return levels[torch.where((over < under) | ((over == under) & (up % 2 == 0)), up, down)]


def _exact_store(c, s):
    q, k, v = None, s["k"].double(), s["v"].double()
    if c["rot"]:
        q, k = _exact_turn(c, s, s["q"]), _exact_turn(c, s, k)
    got = {"q": q}
    slot = s["slot"].long()
    for name, x, cache, scale in (("k", k, s["kc"], s["k_scale"]), ("v", v, s["vc"], s["v_scale"])):
        if c["kv"] == "mxfp4":
            levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
            top = x.reshape(*x.shape[:-1], -1, 32).abs().amax(-1).repeat_interleave(32, -1)
            e = torch.ceil(torch.log2((top / 7).clamp(min=2.0 ** -200))).clamp(-120, 125)
            e += (top > 7 * torch.exp2(e)).double() - (top <= 7 * torch.exp2(e - 1)).double() * (e > -120)
            unit = torch.exp2(e)
            got[name] = _nearest(levels, x.abs() / unit) * torch.sign(x) * unit
            continue
        if c["kv"] == "e4m3":
            levels = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
            x = x / scale.double()[None, :, None]
            x = _nearest(levels, x.abs()) * torch.sign(x)
        full = cache.double().contiguous()
        full[slot // c["page"], slot % c["page"]] = x
        got[name] = full
    return got


def _exact_rows(c, cache, scale, slot):
    page, place = slot.long() // c["page"], slot.long() % c["page"]
    if c["kv"] == "bf16":
        return cache.double()[page, place]
    if c["kv"] == "e4m3":
        return cache.double()[page, place] * scale.double()[:, None]
    levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    byte = cache[page, place].int()
    x = torch.empty((*byte.shape[:-1], c["d"]), dtype=torch.float64, device="cuda")
    x[..., 0::2], x[..., 1::2] = levels[byte % 16], levels[byte // 16]
    return x * torch.exp2(scale.permute(0, 2, 1, 3)[page, place].double() - 127).repeat_interleave(32, -1)


def _exact_attend(s):
    page, H, d = s["page"], s["heads"], s["d"]
    group = s["heads_q"] // H
    c = dict(page=page, kv="mxfp4", d=d)
    L, K, offs, table = [s[k].cpu().numpy() for k in ("len", "K", "offs", "table")]
    out = torch.zeros((s["n_rows"], s["heads_q"], d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["n_rows"], s["heads_q"]), dtype=torch.float64, device="cuda")
    for b in range(s["B"]):
        n, m = int(L[b] + K[b] + 1), int(K[b]) + 1
        t = np.arange(n)
        slot = torch.from_numpy(table[b][t // page].astype(np.int64) * page + t % page).cuda()
        k, v = _exact_rows(c, s["kc"], s["k_scale"], slot), _exact_rows(c, s["vc"], s["v_scale"], slot)
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
