"""The package's packed calls pass every argument to the place that the C function has it in."""
import ctypes
import struct

import pytest

import q4_weight_quantized_gb300 as q4k


@pytest.mark.parametrize("name", sorted(q4k._SLOTS))
def test_slots_match_the_signature(name):
    args = getattr(q4k.load(), name).argtypes
    form = "=" + "".join("d" if a is ctypes.c_float else "q" for a in args)
    values = [1.5 if c == "d" else i for i, c in enumerate(form[1:])]
    assert q4k._SLOTS[name](*values) == struct.pack(form, *values)


def test_wrappers_fill_the_slots_in_order(monkeypatch):
    """Each wrapper called with a different value in every argument: the slots hold them in the C function's order."""
    cache = q4k.KvCache()
    calls = {
        "q4k_kv_append": ([cache] + list(range(1001, 1021)), 22),
        "q4k_attn_decode": ([cache] + list(range(1001, 1006)) + [0.25, 0.5] + list(range(1008, 1013)) + [0.75, 1014, 1015], 17),
        "q4k_kv_evict": ([cache] + list(range(1001, 1013)), 14),
        "q4k_norm_residual": (list(range(1000, 1007)) + [0.25, 1008, 1009, 0.5] + list(range(1011, 1018)) + [0.75, 1019, 1020], 22),
        "q4k_sample": (list(range(1000, 1011)), 12),
    }
    seen = {}

    class Lib:
        def __getattr__(self, name):
            return lambda slots: seen.setdefault(name, slots) and 0 or 0
    monkeypatch.setattr(q4k, "load", lambda: Lib())
    for name, (args, n) in calls.items():
        getattr(q4k, name)(*args, stream=77)
        want = [ctypes.addressof(a) if a is cache else a for a in args] + [77]
        assert len(want) == n and seen[name + "_slots"] == q4k._SLOTS[name](*want), name
