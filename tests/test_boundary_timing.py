"""C-ABI boundary of the timing calls, without a GPU."""
import ctypes

import semi_ar_draft_amd as dk


def test_null_arguments_are_refused():
    lib = dk.load_library()
    ms, n = (ctypes.c_double * 19)(), (ctypes.c_int * 19)()
    assert lib.dspark_timing_read(None, ms, n) == dk.DSPARK_EINVAL
    assert lib.dspark_timing_read_classes(None, 19, ms, n) == dk.DSPARK_EINVAL
