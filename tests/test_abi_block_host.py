"""Host-side refusals of the block operators' C entry points (no GPU needed:
every call below fails validation before any CUDA call)."""
import ctypes

import pytest

from sparse_linear_layers_bitnet_b200 import _abi
from sparse_linear_layers_bitnet_b200 import build as nvbuild

INVALID, UNSUPPORTED, WORKSPACE = _abi.BITNET_ERR_INVALID_ARG, _abi.BITNET_ERR_UNSUPPORTED, _abi.BITNET_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    nvbuild.build()
    return _abi.load()


def at(megabyte, off=0):
    return (megabyte << 20) + off   # fake device addresses, never read


def call(f, base, **changed):
    args = dict(base, **changed)
    assert list(args) == list(base)
    return f(*args.values())


def test_add_rmsnorm_quant_refusals(lib):
    f = lib.bitnet_add_rmsnorm_quant
    ok = dict(X=at(1), R=at(2), w=at(3), T=4, K=512, eps_norm=1e-6, eps_act=1e-5, H=at(4), Xq=at(5), absmax=at(6),
              rinv=at(7), stream=None)
    for name in ("X", "R", "H", "Xq", "absmax"):
        assert call(f, ok, **{name: None}) == INVALID, name
    for name in ("X", "R", "H", "Xq"):
        assert call(f, ok, **{name: ok[name] + 8}) == INVALID, name
    assert call(f, ok, w=at(3, 2)) == INVALID
    for K in (0, 4, 65544):
        assert call(f, ok, K=K) == INVALID
    assert call(f, ok, T=-1) == INVALID
    assert call(f, ok, T=1 << 31) == UNSUPPORTED
    for eps in ("eps_norm", "eps_act"):
        assert call(f, ok, **{eps: 0.0}) == INVALID
        assert call(f, ok, **{eps: float("nan")}) == INVALID
    # H over part of an input, codes over an input or over H
    assert call(f, ok, H=at(1, 1024)) == INVALID
    assert call(f, ok, Xq=at(2, 1024)) == INVALID
    assert call(f, ok, Xq=at(4)) == INVALID
    assert b"overlap" in lib.bitnet_last_error()
    assert call(f, ok, T=0, X=None, R=None, H=None, Xq=None, absmax=None) == _abi.BITNET_OK


def test_rmsnorm_grad_refusals(lib):
    f = lib.bitnet_rmsnorm_grad
    ok = dict(dY=at(1), dy_dtype=1, H=at(2), w=at(3), rinv=at(4), dR=at(5), g_dtype=1, T=4, K=512, dH=at(6), dw=at(7),
              accumulate=0, ws=at(8), ws_bytes=1 << 30, stream=None)
    for name in ("dY", "H", "rinv", "dH"):
        assert call(f, ok, **{name: None}) == INVALID, name
    for name in ("dY", "H", "w", "dR", "dH", "ws"):
        assert call(f, ok, **{name: ok[name] + 8}) == INVALID, name
    for name in ("dy_dtype", "g_dtype"):
        assert call(f, ok, **{name: 2}) == INVALID
    for K in (0, 12, 65544):
        assert call(f, ok, K=K) == INVALID
    assert call(f, ok, T=-1) == INVALID
    assert call(f, ok, T=1 << 31) == UNSUPPORTED
    assert call(f, ok, ws=None) == WORKSPACE
    assert call(f, ok, ws_bytes=lib.bitnet_rmsnorm_grad_workspace_size(4, 512) - 1) == WORKSPACE
    assert call(f, ok, dH=at(1)) == INVALID       # over dY
    assert call(f, ok, dH=at(2, 16)) == INVALID   # over H
    assert call(f, ok, dH=at(5, 16)) == INVALID   # over a part of dR
    assert b"overlap" in lib.bitnet_last_error()
    assert call(f, ok, T=0, dw=None) == _abi.BITNET_OK
    assert lib.bitnet_rmsnorm_grad_workspace_size(1, 512) >= 512 * 4
