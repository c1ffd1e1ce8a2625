"""Results of the 8-bit operators that share a buffer are refused, whichever two: values, scales, rows'
statistics and parameters' gradients.  Pointers are made-up addresses that no kernel ever sees: every call
here has such a pair, and no other fault."""

import os
from itertools import combinations

import pytest

EINVAL = -1
ROW, COL, TILE = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from matrix_optimizer_owner_gb300 import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from matrix_optimizer_owner_gb300 import build
        build.build()
    return _lib.load()


def _at(name, same):
    """An address of its own for every name, and one for the two that share."""
    names = ("x", "r", "dy", "gate", "up", "h_in", "w", "ws", "out", "out_s", "also", "also_s", "src", "src_s", "h",
             "y", "y8", "y8_s", "h8", "h8_s", "mean", "rstd", "dx", "dw", "db", "g8", "g8_s", "u8", "u8_s", "dg",
             "du", "dgr", "dgr_s", "dgc", "dgc_s", "dur", "dur_s", "duc", "duc_s")
    return (1 << 20) * (1 + names.index(same[0] if name in same else name))


def _m(name, groups, same):
    from matrix_optimizer_owner_gb300._lib import Fp8Struct
    return Fp8Struct(_at(name, same), 256, _at(name + "_s", same), 256, 0, groups)


def _quantize(lib, same):
    return lib.mfsdp_quantize_fp8(200, 200, 0, _at("x", same), 200, _m("out", ROW, same),
                                  _m("also", COL, same), None)


def _regroup(lib, same):
    return lib.mfsdp_regroup_fp8(200, 200, _m("src", TILE, same), _m("out", ROW, same), _m("also", COL, same),
                                 None)


def _norm_forward(lib, same):
    a = lambda n: _at(n, same)  # noqa: E731
    return lib.mfsdp_norm_residual_forward(0, 200, 200, 0, 0, a("x"), 200, a("r"), 200, None, None, 1e-5, a("h"),
                                           200, a("y"), 200, _m("y8", ROW, same), _m("h8", ROW, same),
                                           a("mean"), a("rstd"), None)


def _norm_backward(lib, same):
    a = lambda n: _at(n, same)  # noqa: E731
    return lib.mfsdp_norm_residual_backward(0, 200, 200, 0, 0, a("dy"), 200, a("r"), 200, a("h_in"), 200, None,
                                            a("w"), a("mean"), a("rstd"), a("dx"), 200, a("dw"), a("db"),
                                            a("ws"), 1 << 24, None)


def _act_forward(lib, same):
    a = lambda n: _at(n, same)  # noqa: E731
    return lib.mfsdp_activation_forward(0, 200, 200, 0, a("gate"), 200, a("up"), 200, a("y"), 200,
                                        _m("y8", ROW, same), _m("g8", ROW, same), _m("u8", ROW, same), None)


def _act_backward(lib, same):
    a = lambda n: _at(n, same)  # noqa: E731
    return lib.mfsdp_activation_backward(0, 200, 200, 0, a("dy"), 200, None, 0, _m("g8", ROW, same), None, 0,
                                         _m("u8", ROW, same), a("dg"), 200, a("du"), 200, _m("dgr", ROW, same),
                                         _m("dgc", COL, same), _m("dur", ROW, same), _m("duc", COL, same), None)


def _pairs(results, inputs=()):
    return [*combinations(results, 2), *((i, r) for i in inputs for r in results)]


@pytest.mark.parametrize("call,same", [
    *((_quantize, p) for p in _pairs(("out", "out_s", "also", "also_s"), ("x",))),
    *((_regroup, p) for p in _pairs(("out", "out_s", "also", "also_s"), ("src", "src_s"))),
    *((_norm_forward, p) for p in _pairs(("h", "y", "y8", "y8_s", "h8", "h8_s", "mean", "rstd"))),
    *((_norm_backward, p) for p in _pairs(("dx", "dw", "db"))),
    *((_act_forward, p) for p in _pairs(("y", "y8", "y8_s", "g8", "g8_s", "u8", "u8_s"))),
    *((_act_backward, p) for p in _pairs(("dg", "du", "dgr", "dgr_s", "dgc", "dgc_s", "dur", "dur_s", "duc",
                                          "duc_s"), ("g8", "g8_s", "u8", "u8_s")))],
    ids=lambda v: v.__name__[1:] if callable(v) else "-".join(v))
def test_shared_results_are_refused(lib, call, same):
    assert call(lib, same) == EINVAL


def test_no_gradient_of_no_rows_shares_a_buffer(lib):
    """With no rows the parameters' gradients are still written."""
    a = lambda n: _at(n, ("dw", "db"))  # noqa: E731
    assert lib.mfsdp_norm_residual_backward(0, 0, 200, 0, 0, None, 200, None, 200, None, 200, None, None, None,
                                            None, None, 200, a("dw"), a("db"), a("ws"), 1 << 24, None) == EINVAL
