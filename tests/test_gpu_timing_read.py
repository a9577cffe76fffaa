"""GPU: dspark_timing_read writes the 15 entries that its callers' arrays have;
dspark_timing_read_classes as many as it is told."""
import ctypes

import pytest
import torch

import semi_ar_draft_amd as dk
from test_gpu_attend import call, make

pytestmark = pytest.mark.gpu

N = len(dk.KERNEL_CLASSES)


def arrays():
    return (ctypes.c_double * (N + 2))(*[7.0] * (N + 2)), (ctypes.c_int * (N + 2))(*[7] * (N + 2))


def test_as_many_entries_as_the_caller_has():
    ctx = dk.Context(0)
    try:
        s = make(1, [20, 9], [1, 0], 1, 2, 64, 8)
        x = torch.zeros(64, device="cuda")
        ctx.timing(True)

        def work():
            ctx.read_timing()
            call(ctx, s)
            ctx.stream_read(x)

        attend, diag = dk.KERNEL_CLASSES.index("attend"), dk.KERNEL_CLASSES.index("diag")
        work()
        ms, n = arrays()
        assert ctx.lib.dspark_timing_read(ctx._h, ms, n) == dk.DSPARK_OK
        assert list(ms[15:]) == [7.0] * (N + 2 - 15) and list(n[15:]) == [7] * (N + 2 - 15)
        assert n[diag] > 0 and ms[diag] > 0 and n[0] == 0
        for k in (N, attend + 1, attend, 1):
            work()
            ms, n = arrays()
            assert ctx.lib.dspark_timing_read_classes(ctx._h, k, ms, n) == dk.DSPARK_OK
            assert list(ms[k:]) == [7.0] * (N + 2 - k) and list(n[k:]) == [7] * (N + 2 - k)
            if k > attend:
                assert n[attend] == 2 and ms[attend] > 0
            assert ctx.read_timing()["attend"] == (0.0, 0)        # every class's events are forgotten
        for k in (0, -1, N + 1):
            assert ctx.lib.dspark_timing_read_classes(ctx._h, k, ms, n) == dk.DSPARK_EINVAL
        work()
        assert ctx.read_timing()["attend"][1] == 2
    finally:
        ctx.close()
