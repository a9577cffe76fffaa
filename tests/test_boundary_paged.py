"""C-ABI boundary of the calls over a paged cache and of the logit constraints,
without a GPU: null contexts, and the compiled binding's checks of its tensors
(a tensor that is not on the device never reaches the library)."""
import importlib

import pytest
import torch

import semi_ar_draft_amd as dk

CALLS = ("dspark_pages_reserve", "dspark_pages_commit", "dspark_cache_write", "dspark_attend", "dspark_constrain")


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


GOOD = {
    "pages_reserve": lambda: [16, 8, 4, i32(2), i32(2), i32(2, 3), i32(2), i32(2), i32(8), i32(1), i32(1), i32(3), i32(4),
                              i32(4), i32(4)],
    "pages_commit": lambda: [16, 8, i32(2), i32(2), i32(2), None, i32(2, 3), i32(2), i32(2), i32(8), i32(1), i32(1)],
    "cache_write": lambda: [bf(8, 16, 2, 64), bf(8, 16, 2, 64), None, None, bf(4, 2, 64), bf(4, 2, 64), i32(4)],
    "attend": lambda: [bf(8, 16, 2, 64), bf(8, 16, 2, 64), None, None, bf(2, 4, 64), i32(2), i32(2, 3), 0, None, None, True,
                       0.125, bf(2, 4, 64), None],
    "constrain": lambda: [bf(2, 1, 64), torch.zeros(2, 1, 64), 1] + [None] * 13,
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
