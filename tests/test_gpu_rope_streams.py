"""GPU: the calls of rotary positions and of the 4-bit cache from two contexts on
two streams at once, and over inputs that another stream has just written."""
import numpy as np
import pytest
import torch

import semi_ar_draft_amd as dk
from test_gpu_attend import dev
from test_gpu_attend_mxfp4 import make
from test_gpu_rope import i32

pytestmark = pytest.mark.gpu


def test_two_contexts_on_two_streams():
    n, freq = 700, dk.rope_frequencies(128, device="cuda")[0]
    g = torch.Generator(device="cuda").manual_seed(2)
    sets = []
    for seed in (1, 2):
        s = make(seed, [500, 30, 2000, 90], [3, 1, 5, 0], 2, 4, 128, 16)
        s.update({k: dev(s[k]) for k in ("table", "length", "K", "offs")})
        s["x"] = [torch.randn((n, h, 128), generator=g, device="cuda").to(torch.bfloat16) for h in (8, 2, 2)]
        s["pos"], s["slot"] = i32(np.arange(n) * seed), i32(np.random.RandomState(seed).permutation(n))
        pages = -(-n // 16)
        s["cache"] = [torch.zeros((pages, 16, 2, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
        s["cache"] += [torch.zeros((pages, 2, 16, 4), dtype=torch.uint8, device="cuda") for _ in range(2)]
        sets.append(s)

    def work(ctx, s, stream):
        kc, vc, kp, vp = s["cache"]
        q = ctx.rope_write(*s["x"], s["pos"], s["slot"], freq, kc, vc, kp, vp, stream=stream)
        k, v = ctx.cache_read(kc, vc, s["slot"], kp, vp, stream=stream)
        turned = ctx.rope(s["x"][0], s["x"][1], s["pos"], freq, interleaved=True, stream=stream)
        out = ctx.attend(s["q"], s["kc"], s["vc"], s["table"], s["length"], 5, K=s["K"], t_offsets=s["offs"], k_scale=s["kp"],
                         v_scale=s["vp"], stream=stream)
        return [q, k, v, *turned, out]

    with dk.Context(0) as a, dk.Context(0) as b:
        alone = [[t.clone() for t in work(c, s, None)] for c, s in zip((a, b), sets)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(5):
            got = [None, None]
            for i, (c, s, st) in enumerate(zip((a, b), sets, streams)):
                got[i] = work(c, s, st)
            torch.cuda.synchronize()
            for x, y in zip(alone, got):
                assert all([torch.equal(u, w) for u, w in zip(x, y)])
        # inputs that the call's own stream has just made
        st = streams[0]
        s = sets[0]
        with torch.cuda.stream(st):
            for _ in range(20):
                s["x"][0].mul_(1)
            s["x"][0].neg_()
        q = a.rope_write(*s["x"], s["pos"], s["slot"], freq, *s["cache"], stream=st)
        st.synchronize()
        assert torch.equal(q, -alone[0][0])
        a.check(st)
        b.check()
