"""GPU: attention whose waves walk many steps of a tile, against the float64
reference.  The work is an even line of steps (32 tokens of a tile each, and
one for a tile) over four waves a compute unit, so only batches with much more
work than waves reach the loop's later steps: loads into buffers that have been
used, page ids several steps ahead, maxima that rise late.  The cases say from
the formula how many steps a wave takes."""
import numpy as np
import pytest
import torch

import semi_ar_draft_amd as dk
from attend_reference import worst_error
from test_gpu_attend import call, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = dk.Context(0)
    yield c
    c.close()


def plan(s, gamma):
    """(rows of a tile, units of a wave's stretch, workgroups that share the longest tile)."""
    Hq, heads, d = s["q"].shape[1], s["kc"].shape[2], s["q"].shape[2]
    group = Hq // heads
    most = group * (gamma + 1)
    rows = 16 if most <= 16 else 32 if most <= 32 or d == 256 else 64
    n = s["K"] + 1
    steps = np.where(n > 0, -(-(s["length"] + n) // 32), 0)
    total = int((heads * -(-(group * n) // rows) * (steps + 1)).sum())
    waves = 4 * torch.cuda.get_device_properties(0).multi_processor_count
    stretch = max(2, -(-total // waves))
    return rows, stretch, int(steps.max()) // (4 * stretch)


def bounds(eight):
    return dict(weight=2.0 ** -11, floor=2.0 ** -32) if eight else dict(weight=2.0 ** -15)


def rising(s):
    """Keys that grow along the sequence: a row's maximum rises by hundreds of units over it, step after step."""
    page = s["kc"].shape[1]
    size = torch.ones(s["kc"].shape[:2], device="cuda")
    for b, L in enumerate(s["length"] + s["K"] + 1):
        for p in range(-(-int(L) // page)):
            t = torch.arange(p * page, (p + 1) * page, device="cuda")
            size[int(s["table"][b][p])] = 0.1 + 6.0 * t / int(L)
    k = s["kc"].float() * size[:, :, None, None]
    s["kc"].copy_((k.clamp(-448, 448) if s["ks"] is not None else k).to(s["kc"].dtype))


# group and gamma for 16, 32 and 64 rows a tile, and 100 (two tiles of 64, four of 32)
ROWS = {16: (4, 3), 32: (4, 7), 64: (8, 7), 100: (25, 3)}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("rows", [16, 32, 64, 100])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_steps_a_wave(ctx, d, rows, eight, causal):
    group, gamma = ROWS[rows]
    page, order = [(8, "token"), (16, "head"), (64, "token"), (16, "token")][(rows // 16 + eight + 2 * causal) % 4]
    heads = 16 if rows < 100 else 8
    length = [4100, 2933, 5007, 3331, 0, 64]                      # steps of every remainder, odd and even counts
    s = make(rows + d, length, [gamma, gamma - 1, gamma, 0, gamma, -1], heads, group, d, page, order, eight)
    if rows != 32:
        rising(s)
    tile, stretch, _ = plan(s, gamma)
    ahead = 1 if d * tile // 16 >= 512 and not eight else 2
    print(f"stretches d={d} rows={rows} tile={tile} 8bit={eight} causal={causal} page={page} {order}: {stretch} units", flush=True)
    assert stretch - 1 >= ahead + 3
    out, lse = call(ctx, s, causal)
    ctx.check()
    worst = worst_error(s, out, lse, causal, **bounds(eight))
    print("worst error over its bound: %.3f" % worst, flush=True)
    assert worst <= 1.0
    again, lse2 = call(ctx, s, causal)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("d,group", [(64, 8), (128, 8), (256, 4), (128, 4)])
def test_tiles_joined_from_many_workgroups(ctx, d, group, eight):
    """One tile of 32 or 64 rows over more than twenty workgroups: the join's later rounds."""
    s = make(d, [9000], [7], 1, group, d, 16, "token", eight)
    rising(s)
    tile, stretch, shared = plan(s, 7)
    print(f"joined d={d} tile={tile} 8bit={eight}: {shared} workgroups", flush=True)
    assert tile > 16 and shared > 20
    out, lse = call(ctx, s)
    ctx.check()
    worst = worst_error(s, out, lse, True, **bounds(eight))
    print("worst error over its bound: %.3f" % worst, flush=True)
    assert worst <= 1.0
