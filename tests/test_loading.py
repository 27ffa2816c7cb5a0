"""A library loaded from a path has its signatures each time: without them ctypes
would pass 64-bit addresses as ints."""
import ctypes

import pytest


@pytest.mark.parametrize("name,function", [("gdr", "gdr_forward"), ("blocknorm", "blocknorm_add_forward"), ("rwkv8", "rwkv8_forward")])
def test_each_loaded_library_has_its_signatures(name, function):
    import importlib

    from linear_rnn_state_gb300 import _build

    _build.build()
    module = importlib.import_module(f"linear_rnn_state_gb300.{name}")
    for _ in range(20):  # each one given up before the next is loaded, which may get its place in memory
        lib = module.load(_build.DEBUG_LIB)
        assert getattr(lib, function).argtypes[0] is ctypes.c_void_p
        del lib
