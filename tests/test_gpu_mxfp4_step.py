"""GPU: serving steps over a 4-bit cache as they are used -- pages, rotary
positions and cache write in one launch, attention, rows read back, pages
back -- against the oracles, the state carried from step to step; then a step
captured and replayed to the eager result with eager work between."""
import numpy as np
import pytest
import torch

import oracle
import semi_ar_draft_amd as dk
from attend_reference import worst_error
from test_gpu_rope import codes_of, f64, i32, values

pytestmark = pytest.mark.gpu

PAGE, HEADS, GROUP, D, GAMMA = 16, 2, 4, 128, 5


class Server:
    """Device state of a batch over a 4-bit cache; every shape is fixed."""

    def __init__(self, ctx, seed, rot, inter):
        self.ctx, self.inter = ctx, inter
        rng = np.random.RandomState(seed)
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.prompt = np.array([1, PAGE, 150, 33, 7])
        self.B = B = len(self.prompt)
        cols = 16
        self.n_pages = B * cols
        z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device="cuda")
        self.length, self.held, self.n_free = z(B), z(B), i32([self.n_pages])
        self.table, self.free = i32(np.full((B, cols), -1)), i32(rng.permutation(self.n_pages))
        # a new cache holds zeros; its powers too
        self.kc, self.vc = [z(self.n_pages, PAGE, HEADS, D // 2, dtype=torch.uint8) for _ in range(2)]
        self.kp, self.vp = [z(self.n_pages, HEADS, PAGE, D // 32, dtype=torch.uint8) for _ in range(2)]
        self.freq, self.factor = dk.rope_frequencies(rot, 10000.0, "yarn", 4.0, trained=64, device="cuda")
        self.n = B * (GAMMA + 1)
        self.rows = (z(B + 1), z(self.n), z(self.n), z(self.n))
        self.qkv = z(self.n, (HEADS * GROUP + 2 * HEADS) * D, dtype=torch.bfloat16)
        self.out, self.lse = z(self.n, HEADS * GROUP, D, dtype=torch.bfloat16), z(self.n, HEADS * GROUP, dtype=torch.float32)
        self.q_out = torch.zeros_like(self.out)
        self.back = [z(self.n, HEADS, D, dtype=torch.bfloat16) for _ in range(2)]
        self.K, self.acc = z(B), z(B)
        self.all_k, self.all_v = [], []                  # what was written: (request, position) -> exact rows

    STATE = ("length", "held", "n_free", "table", "free", "kc", "vc", "kp", "vp", "out", "lse", "q_out")

    def split(self, qkv):
        hq = HEADS * GROUP * D
        return [x.unflatten(1, (-1, D)) for x in qkv.split([hq, HEADS * D, HEADS * D], 1)]

    def fill(self, n):
        return (torch.randn((n, (HEADS * GROUP + 2 * HEADS) * D), generator=self.g, device="cuda") * 1.5).to(torch.bfloat16)

    def write(self, qkv, pos, slot, q_out):
        q, k, v = self.split(qkv)
        return self.ctx.rope_write(q, k, v, pos, slot, self.freq, self.kc, self.vc, self.kp, self.vp, interleaved=self.inter,
                                   factor=self.factor, q_out=q_out)

    def prefill(self):
        n = int(self.prompt.sum()) + 3
        offs, req, pos, slot = self.ctx.pages_reserve(i32(self.prompt - 1), self.length, self.table, self.held, self.free,
                                                      self.n_free, PAGE, self.n_pages, n_rows=n)
        qkv = self.fill(n)
        self.write(qkv, pos, slot, None)
        self.ctx.pages_commit(self.length, i32(self.prompt - 1), self.table, self.held, self.free, self.n_free, PAGE,
                              self.n_pages)
        return qkv, req, pos, slot

    def step(self):
        c = self.ctx
        offs, req, pos, slot = c.pages_reserve(self.K, self.length, self.table, self.held, self.free, self.n_free, PAGE,
                                               self.n_pages, out=self.rows)
        self.write(self.qkv, pos, slot, self.q_out)
        c.attend(self.q_out, self.kc, self.vc, self.table, self.length, GAMMA, K=self.K, t_offsets=offs, k_scale=self.kp,
                 v_scale=self.vp, out=self.out, lse=self.lse)
        c.cache_read(self.kc, self.vc, slot, self.kp, self.vp, out=self.back)

    def commit(self):
        self.ctx.pages_commit(self.length, self.acc, self.table, self.held, self.free, self.n_free, PAGE, self.n_pages)


def check_rows(s, qkv, pos, slot):
    """The cache holds the rows' turned keys and values, rounded once."""
    _, k, v = s.split(qkv)
    pos, slot = pos.cpu().numpy(), slot.cpu().numpy()
    live = slot >= 0
    at = (slot[live] // PAGE, slot[live] % PAGE)
    turned = oracle.rope(f64(k), pos, s.freq.cpu().numpy(), s.inter, s.factor)[live]
    for x, cache, power in ((turned, s.kc, s.kp), (f64(v)[live], s.vc, s.vp)):
        code, byte = oracle.to_mxfp4(x)
        assert np.array_equal(power.cpu().numpy().transpose(0, 2, 1, 3)[at], byte)
        got = oracle.from_mxfp4(codes_of(cache)[at], byte)
        near = np.abs(oracle.from_mxfp4(code, byte) - x)
        assert (np.abs(got - x) <= near * (1 + 1e-12) + 2.0 ** -40 * np.abs(x).max()).all()


def check_attention(s):
    t = dict(q=s.q_out, kc=torch.from_numpy(values(s.kc, s.kp)).float(), vc=torch.from_numpy(values(s.vc, s.vp)).float(),
             table=s.table.cpu().numpy(), length=s.length.cpu().numpy(), K=s.K.cpu().numpy(), offs=s.rows[0].cpu().numpy(),
             scale=D ** -0.5, ks=None, vs=None)
    assert worst_error(t, s.out, s.lse, True, 2.0 ** -15, 2.0 ** -60) <= 1.0


@pytest.mark.parametrize("rot,inter", [(128, False), (64, True)])
def test_steps_over_a_4bit_cache(rot, inter):
    with dk.Context(0) as ctx:
        s = Server(ctx, 3 + rot, rot, inter)
        check_rows(s, *(lambda qkv, req, pos, slot: (qkv, pos, slot))(*s.prefill()))
        rng = np.random.RandomState(7)
        for step in range(5):
            K = rng.randint(-1, GAMMA + 1, s.B)
            K[step % s.B] = GAMMA
            s.K.copy_(i32(K))
            s.acc.copy_(i32([rng.randint(0, k + 1) if k >= 0 else -1 for k in K]))
            s.qkv.copy_(s.fill(s.n))
            s.out.fill_(7)
            s.step()
            ctx.check()
            check_rows(s, s.qkv, s.rows[2], s.rows[3])
            check_attention(s)
            rows = int((K + 1).sum())
            assert (s.out[rows:] == 7).all()             # rows behind the last are left
            slot = s.rows[3].cpu().numpy()[:rows]
            for y, cache, power in zip(s.back, (s.kc, s.vc), (s.kp, s.vp)):
                assert np.array_equal(f64(y)[:rows], values(cache, power)[slot // PAGE, slot % PAGE])
            s.commit()
            ctx.check()


def test_a_captured_step_replays_to_the_eager_result():
    with dk.Context(0) as ctx:
        s = Server(ctx, 11, 128, False)
        s.prefill()
        s.K.copy_(i32([GAMMA, 0, 2, -1, 4]))
        s.acc.copy_(i32([1, 0, 2, -1, 0]))
        s.qkv.copy_(s.fill(s.n))
        start = {k: getattr(s, k).clone() for k in s.STATE}

        def whole():
            s.step()
            s.commit()

        def load():
            for k, v in start.items():
                getattr(s, k).copy_(v)

        whole()                                          # the workspace grows
        load()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            whole()
        for turn in range(4):
            s.qkv.copy_(s.fill(s.n))
            s.K.copy_(i32([GAMMA, 0, turn, -1, 4 - turn]))
            s.acc.copy_(i32([turn, 0, 0, -1, 4 - turn]))
            load()
            whole()
            eager = {k: getattr(s, k).clone() for k in s.STATE}
            load()
            graph.replay()
            torch.cuda.synchronize()
            assert all([torch.equal(eager[k], getattr(s, k)) for k in s.STATE])
        ctx.check()


def test_caches_past_four_gigabytes():
    """Slots, powers and pages whose offsets pass 32 bits."""
    with dk.Context(0) as ctx:
        heads, page, n_pages = 16, 64, 90000             # 5.9 GB a cache
        kc, vc = [torch.empty((n_pages, page, heads, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
        kp, vp = [torch.empty((n_pages, heads, page, 4), dtype=torch.uint8, device="cuda") for _ in range(2)]
        g = torch.Generator(device="cuda").manual_seed(1)
        n = 100
        x = [torch.randn((n, heads, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
        table = np.array([[n_pages - 1, 70000]])
        t = np.arange(n)
        slot = table[0][t // page] * page + t % page
        freq, _ = dk.rope_frequencies(128, device="cuda")
        q = ctx.rope_write(x[0], x[1], x[2], i32(t), i32(slot), freq, kc, vc, kp, vp)
        k, v = ctx.cache_read(kc, vc, i32(slot), kp, vp)
        out = ctx.attend(q, kc, vc, i32(table), i32([n - 1]), 0, K=i32([0]), t_offsets=i32([n - 1]), k_scale=kp, v_scale=vp)
        ctx.check()
        code, byte = oracle.to_mxfp4(f64(x[2]))
        assert np.array_equal(f64(v), oracle.from_mxfp4(code, byte))
        kd, vd = k.double(), v.double()
        e = torch.einsum("hd,thd->ht", q[n - 1].double(), kd) * 128 ** -0.5
        want = torch.einsum("ht,thd->hd", torch.softmax(e, 1), vd)
        assert (out[n - 1].double() - want).abs().max() <= 2.0 ** -7 * want.abs().max()
