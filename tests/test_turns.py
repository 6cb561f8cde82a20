"""Calls of several host threads on one workspace take turns (no GPU: the calls end without a launch)."""
import ctypes
import threading

import pytest


@pytest.fixture(scope="module")
def rg():
    from exact_modular_int8_gb300 import build as b

    b.build()
    import exact_modular_int8_gb300 as m

    return m


@pytest.fixture(scope="module")
def mem():
    buf = (ctypes.c_uint8 * 65536)()
    return (ctypes.addressof(buf) + 255) // 256 * 256, buf


def empty_calls(lib, ws, other):
    """Calls without entries: they enqueue nothing but the clearing of the workspace's first words."""
    big = 1 << 14
    return {
        "res_gemm_i64": lambda: lib.res_gemm_i64(None, None, None, 0, 4, 4, 0, 0, ws, big, None),
        "enclose_gemm_f64": lambda: lib.enclose_gemm_f64(None, None, None, None, 0, 4, 4, 0, None, ws, big, None),
        "scaled_gemm_f8": lambda: lib.scaled_gemm_f8(None, 16, None, None, 16, None, None, 0, 4, 0, 4, 16, 4, ws, big,
                                                     None),
        "linear_f8": lambda: lib.linear_f8(None, 0, 0, None, 0, 0, None, 0, 0, 0, other, big, 0, ws, big, None),
        "linear_f8_backward": lambda: lib.linear_f8_backward(None, 0, 0, other, big, None, None, 0, 0, 0, 0, 0, ws, big,
                                                             None),
        "moe_layer_f8": lambda: lib.moe_layer_f8(None, 2, None, None, None, None, None, None, 0, 32, 16, 4, 2, 1, 0, ws,
                                                 big, None),
    }


@pytest.mark.parametrize("name", list(empty_calls(None, 0, 0)))
def test_a_call_waits_for_the_turn_on_its_workspace(rg, mem, name):
    lib, ws, other = rg.library(), mem[0], mem[0] + 32768
    done = threading.Event()
    t = threading.Thread(target=lambda: (empty_calls(lib, ws, other)[name](), done.set()))
    assert lib.rg_hold_workspace(ws, 1) == rg.RG_OK
    try:
        t.start()
        assert not done.wait(0.3)
        empty_calls(lib, other, ws)[name]()  # another workspace: no waiting
    finally:
        assert lib.rg_hold_workspace(ws, 0) == rg.RG_OK
    assert done.wait(30)
    t.join()


def test_turns_are_given_back(rg, mem):
    lib, ws = rg.library(), mem[0]
    assert lib.rg_hold_workspace(None, 1) == rg.RG_ERR_ARG
    assert lib.rg_hold_workspace(ws, 0) == rg.RG_ERR_ARG  # nobody has it
    for f in empty_calls(lib, ws, ws + 32768).values():
        f()
    assert lib.rg_hold_workspace(ws, 1) == rg.RG_OK
    assert lib.rg_hold_workspace(ws, 0) == rg.RG_OK
