"""GPU: blocks of a 4-bit cache whose power is 2^126 or 2^127 (bytes 253 and 254:
another program's, the writes stop at 252).  What bf16 holds of their values is
taken as it is, what passes it is infinite, wherever in its step a token stands.

Keys are zeros, so every weight is 1: a row that sees n tokens gets v / n of a
single value v, exactly but for the quotient (2^-22 of it allowed) and the
rounding of the result (2^-8)."""
import numpy as np
import pytest
import torch

import oracle
import semi_ar_draft_amd as dk
from test_gpu_attend_mxfp4 import call, make
from test_gpu_rope import caches, f64, i32

pytestmark = pytest.mark.gpu

LEVELS = np.array(oracle.E2M1 + tuple(-v for v in oracle.E2M1))
CODES = torch.arange(16, dtype=torch.uint8)
LARGEST = (2 - 2.0 ** -7) * 2.0 ** 127                   # of bf16


@pytest.fixture(scope="module")
def ctx():
    c = dk.Context(0)
    yield c
    c.close()


def block_values(byte):
    """Codes 0 .. 15 twice, as bf16 has them."""
    v = np.tile(LEVELS, 2) * 2.0 ** (byte - 127)
    return np.where(np.abs(v) > LARGEST, np.copysign(np.inf, v), v)


def zero_cache(s):
    for c, p in (("kc", "kp"), ("vc", "vp")):
        s[c].zero_()
        s[p].fill_(127)


@pytest.mark.parametrize("byte", [252, 253, 254])
@pytest.mark.parametrize("d,page,order", [(64, 8, "token"), (128, 16, "token"), (128, 64, "head"), (256, 32, "token")])
@pytest.mark.parametrize("gamma,group", [(3, 2), (7, 16)])
def test_values_of_the_largest_powers(ctx, byte, d, page, order, gamma, group):
    """In a step that every row sees whole, in one that some do not, and among the drafts."""
    length = 40
    v = block_values(byte)
    for token in (5, 33, length + 2):
        print(f"byte={byte} d={d} page={page} {order} gamma={gamma} group={group} token={token}", flush=True)
        s = make(1, [length, 9], [gamma, 0], 2, group, d, page, order)
        zero_cache(s)
        block = d // 32 - 1
        at = (int(s["table"][0][token // page]), token % page)
        s["vc"][at[0], at[1], 1, 16 * block:16 * block + 16] = (CODES[0::2] | CODES[1::2] << 4).repeat(2).cuda()
        s["vp"][at[0], 1, at[1], block] = byte
        out, lse = call(ctx, s)
        ctx.check()
        out = f64(out)
        for i in range(gamma + 1):
            n = length + i + 1
            want = np.zeros((2 * group, d))
            if token < n:
                want[group:, 32 * block:32 * block + 32] = v / n
            odd = ~np.isfinite(want)
            assert not np.isfinite(out[i][odd]).any()
            assert (np.abs(out[i][~odd] - want[~odd]) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want[~odd])).all()
        assert (out[gamma + 1:] == 0).all()              # the other request


def test_a_long_request_with_such_a_block(ctx):
    """Joined from many workgroups' pieces."""
    s = make(2, [6000], [2], 1, 4, 128, 16)
    zero_cache(s)
    for token, byte in ((100, 253), (6001, 254)):
        at = (int(s["table"][0][token // 16]), token % 16)
        s["vc"][at[0], at[1], 0, :16] = (CODES[0::2] | CODES[1::2] << 4).repeat(2).cuda()
        s["vp"][at[0], 0, at[1], 0] = byte
    out, _ = call(ctx, s)
    ctx.check()
    out = f64(out)
    for i in range(3):
        with np.errstate(invalid="ignore"):
            want = block_values(253) + (block_values(254) if i else 0)
        odd = ~np.isfinite(want) | (np.abs(want) > LARGEST)
        assert not np.isfinite(out[i][:, :32][:, ~np.isfinite(want)]).any()
        want = want[~odd] / (6001 + i)
        assert (np.abs(out[i][:, :32][:, ~odd] - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want)).all()
        assert (out[i][:, 32:] == 0).all()


def test_rows_of_such_blocks_come_back(ctx):
    kc, vc, kp, vp = caches("mxfp4", 1, 8, 1, 64, "token")
    kc[:, :, 0] = (CODES[0::2] | CODES[1::2] << 4).repeat(4).cuda()
    vc.copy_(kc)
    kp[0, 0] = torch.tensor([253, 254], dtype=torch.uint8, device="cuda")
    vp[0, 0] = torch.tensor([255, 252], dtype=torch.uint8, device="cuda")
    k, v = ctx.cache_read(kc, vc, i32(np.arange(8)), kp, vp)
    ctx.check()
    want = np.concatenate([block_values(253), block_values(254)])
    assert np.array_equal(f64(k), np.broadcast_to(want, (8, 1, 64)))
    assert np.isnan(f64(v)[..., :32]).all() and np.array_equal(f64(v)[..., 32:], np.broadcast_to(block_values(252), (8, 1, 32)))


def test_the_least_power_comes_back(ctx):
    """Byte 0, 2^-127: what bf16 holds as it is (its subnormals: to within half a step of 2^-133)."""
    kc, vc, kp, vp = caches("mxfp4", 1, 8, 1, 64, "token")
    kc[:, :, 0] = (CODES[0::2] | CODES[1::2] << 4).repeat(4).cuda()
    vc.copy_(kc)
    kp.zero_()
    vp.fill_(1)
    k, v = ctx.cache_read(kc, vc, i32(np.arange(8)), kp, vp)
    ctx.check()
    assert (np.abs(f64(k) - np.tile(LEVELS, 4) * 2.0 ** -127) <= 2.0 ** -134).all()
    assert (np.abs(f64(v) - np.tile(LEVELS, 4) * 2.0 ** -126) <= 2.0 ** -134).all()
