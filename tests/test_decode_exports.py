"""Every function that the library exports is declared in its header, and a slots form does what its call does."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import q4_weight_quantized_gb300 as q4k

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from q4_weight_quantized_gb300.build import build_library
    build_library()
    return q4k.load()


@pytest.mark.skipif(shutil.which("nm") is None, reason="needs nm")
def test_exports_are_declared(lib):
    out = subprocess.run(["nm", "-D", "--defined-only", q4k.LIB_PATH], capture_output=True, text=True, check=True).stdout
    names = {line.split()[-1] for line in out.splitlines() if line.split()[-1].startswith("q4k_")}
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "q4k.h")).read(), flags=re.S)
    assert names and names == set(re.findall(r"\b(q4k_[a-z0-9_]+)\s*\(", src))


@pytest.mark.parametrize("name", sorted(q4k._SLOTS))
def test_a_slots_form_checks_what_its_call_checks(lib, name):
    """Every pointer NULL and every number 1: both refuse alike, and so do they where one number is out of range."""
    types = getattr(lib, name).argtypes
    f32 = ctypes.c_float

    def both(change=None, value=0):
        one = [(1.0 if t is f32 else 1) if t in (f32, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_size_t) else None for t in types]
        if change is not None:
            one[change] = value
        return getattr(lib, name)(*one), getattr(lib, name + "_slots")(q4k._SLOTS[name](*[0 if a is None else a for a in one]))

    assert getattr(lib, name + "_slots")(None) == q4k.Q4K_ERR_NULL
    a, b = both()
    assert a == b == q4k.Q4K_ERR_NULL
    for i, t in enumerate(types):
        if t is ctypes.c_int64:
            a, b = both(i, -5)
            assert a == b != q4k.Q4K_OK
