"""C-ABI boundary of the calls of rotary positions and of the 4-bit cache, without
a GPU: null contexts, and the compiled binding's checks of its tensors."""
import importlib

import pytest
import torch

import semi_ar_draft_amd as dk

CALLS = ("dspark_rope", "dspark_rope_write", "dspark_cache_read", "dspark_cache_write_mxfp4", "dspark_attend_mxfp4")


@pytest.mark.parametrize("name", CALLS)
def test_a_null_context_is_refused(name):
    f = getattr(dk.load_library(), name)
    args = [0.0 if getattr(t, "__name__", "") in ("c_float", "c_double") else None if "p" in getattr(t, "_type_", "") else 0
            for t in f.argtypes]
    assert f(*args) == dk.DSPARK_EINVAL


@pytest.fixture(scope="module")
def native():
    dk.load_library()
    return importlib.import_module("semi_ar_draft_amd._native")


def i32(*n):
    return torch.zeros(n, dtype=torch.int32)


def bf(*n):
    return torch.zeros(n, dtype=torch.bfloat16)


def four():
    u = lambda *n: torch.zeros(n, dtype=torch.uint8)
    return [u(8, 16, 2, 32), u(8, 16, 2, 32), u(8, 2, 16, 2), u(8, 2, 16, 2)]


FREQ = lambda: torch.zeros(32, dtype=torch.float64)
GOOD = {
    "cache_read": lambda: [*four(), i32(4), bf(4, 2, 64), bf(4, 2, 64)],
    "rope": lambda: [FREQ(), False, 1.0, i32(4), bf(4, 2, 64), bf(4, 2, 64), bf(4, 6, 64), bf(4, 6, 64)],
    "rope_write": lambda: [*four(), FREQ(), False, 1.0, i32(4), i32(4), bf(4, 2, 64), bf(4, 2, 64), bf(4, 6, 64),
                           bf(4, 6, 64)],
    "cache_write": lambda: [*four(), bf(4, 2, 64), bf(4, 2, 64), i32(4)],
}


@pytest.mark.parametrize("name", GOOD)
def test_tensors_off_the_device_are_refused(native, name):
    with pytest.raises((TypeError, ValueError), match="device|cuda|GPU"):
        getattr(native, name)(0, 0, 0, *GOOD[name]())


@pytest.mark.parametrize("name", GOOD)
def test_wrong_arguments_are_refused(native, name):
    f, good = getattr(native, name), GOOD[name]()
    with pytest.raises(TypeError):
        f(0, 0, 0, *good[:-1])
    with pytest.raises(TypeError):
        f(0, 0, 0, *good, None)
    for i, x in enumerate(good):
        for bad in ("x", object()):
            with pytest.raises((TypeError, ValueError)):
                f(0, 0, 0, *good[:i], bad, *good[i + 1:])
        if isinstance(x, torch.Tensor):
            for bad in (x.double(), x[None]):
                with pytest.raises((TypeError, ValueError)):
                    f(0, 0, 0, *good[:i], bad, *good[i + 1:])
