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
    for name in ("w", "absmax", "rinv"):
        assert call(f, ok, **{name: ok[name] + 2}) == INVALID, name
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
    for name in ("rinv", "dw"):
        assert call(f, ok, **{name: ok[name] + 2}) == INVALID, name
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


def test_rope_refusals(lib):
    f = lib.bitnet_rope
    ok = dict(X=at(1), dtype=1, ldx=512, pos=at(2), table=at(3), n_pos=64, T=4, n_heads=4, head_dim=128, rot_dim=128,
              layout=0, inverse=0, Y=at(4), ldy=512, ws=at(5), ws_bytes=256, stream=None)
    for name in ("X", "Y", "pos", "table"):
        assert call(f, ok, **{name: None}) == INVALID, name
    for name, off in (("X", 1), ("Y", 1), ("pos", 2), ("table", 4), ("ws", 8)):
        assert call(f, ok, **{name: ok[name] + off}) == INVALID, name
    for name, bad in (("dtype", 3), ("ldx", 511), ("ldy", 511), ("n_pos", 0), ("T", -1), ("n_heads", 0), ("head_dim", 0),
                      ("rot_dim", 130), ("rot_dim", 63), ("rot_dim", -2), ("layout", 2)):
        assert call(f, ok, **{name: bad}) == INVALID, name
    assert call(f, ok, head_dim=257, ldx=4096, ldy=4096) == UNSUPPORTED
    assert call(f, ok, T=1 << 31) == UNSUPPORTED
    assert call(f, ok, ws=None) == WORKSPACE and call(f, ok, ws_bytes=255) == WORKSPACE
    assert call(f, ok, Y=at(1), ldy=1024) == INVALID and call(f, ok, Y=at(1, 256)) == INVALID
    assert call(f, ok, T=0, X=None, Y=None, pos=None) == _abi.BITNET_OK


def cache(**changed):
    c = _abi.BitnetKvCache(at(10), at(11), 32, 16 * 5 * 128, 16 * 128, 128, 16, 5, 128)
    for k, v in changed.items():
        setattr(c, k, v)
    return ctypes.byref(c)


BAD_CACHES = [("k", None, INVALID), ("v", None, INVALID), ("k", at(10, 8), INVALID), ("n_pages", 0, INVALID),
              ("n_pages", 1 << 31, UNSUPPORTED), ("page_size", 24, UNSUPPORTED), ("page_size", 4, UNSUPPORTED),
              ("page_size", 1 << 17, UNSUPPORTED), ("page_size", 0, INVALID), ("n_kv_heads", 0, INVALID),
              ("n_kv_heads", 65536, UNSUPPORTED), ("head_dim", 257, UNSUPPORTED), ("head_dim", 0, INVALID),
              ("row_stride", 124, INVALID), ("row_stride", 120, INVALID), ("head_stride", 2044, INVALID),
              ("page_stride", 8, INVALID)]


def test_rope_append_refusals(lib):
    f = lib.bitnet_rope_append
    ok = dict(QKV=at(1), dtype=1, ld=3840, pos=at(2), seq=at(3), table=at(4), n_pos=64, T=4, n_heads=20, rot_dim=128,
              layout=1, cache=cache(), pages=at(5), n_seqs=2, max_pages=8, Q=at(6), ws=at(7), ws_bytes=256, stream=None)
    for name in ("QKV", "pos", "table", "pages", "Q", "cache"):
        assert call(f, ok, **{name: None}) == INVALID, name
    for field, value, status in BAD_CACHES:
        assert call(f, ok, cache=cache(**{field: value})) == status, field
    for name, bad in (("dtype", 3), ("ld", 3839), ("n_pos", 0), ("T", -1), ("n_heads", 0), ("n_seqs", -1), ("max_pages", 0),
                      ("rot_dim", 130), ("rot_dim", 63), ("layout", 2)):
        assert call(f, ok, **{name: bad}) == INVALID, name
    assert call(f, ok, cache=cache(v=at(10))) == INVALID        # keys and values in one place
    assert call(f, ok, seq=None) == INVALID                     # four rows, two sequences
    assert call(f, ok, Q=at(1, 4096)) == INVALID
    assert call(f, ok, T=1 << 31) == UNSUPPORTED
    assert call(f, ok, ws=None) == WORKSPACE and call(f, ok, ws_bytes=0) == WORKSPACE
    assert call(f, ok, T=0, QKV=None, pos=None, Q=None) == _abi.BITNET_OK
    assert call(f, ok, T=0, rot_dim=0, table=None, n_pos=0) == _abi.BITNET_OK


def test_paged_attn_refusals(lib):
    f = lib.bitnet_paged_attn
    need = lib.bitnet_paged_attn_workspace_size(4, 20, 5, 128)
    ok = dict(Q=at(1), ldq=2560, n_seqs=4, n_heads=20, cache=cache(), pages=at(2), max_pages=8, lens=at(3), scale=0.1,
              O=at(4), o_dtype=1, ldo=2560, lse=at(5), ws=at(6), ws_bytes=need, stream=None)
    for name in ("Q", "pages", "lens", "O", "cache"):
        assert call(f, ok, **{name: None}) == INVALID, name
    for field, value, status in BAD_CACHES:
        assert call(f, ok, cache=cache(**{field: value})) == status, field
    for name, bad in (("ldq", 2559), ("ldo", 2559), ("n_seqs", -1), ("n_heads", 0), ("n_heads", 18), ("max_pages", 0),
                      ("o_dtype", 2), ("scale", float("nan")), ("scale", float("inf")), ("O", at(1, 512)), ("Q", at(1, 1)),
                      ("lens", at(3, 2)), ("ws", at(6, 8))):
        assert call(f, ok, **{name: bad}) == INVALID, name
    assert call(f, ok, max_pages=(1 << 26) + 1) == UNSUPPORTED       # 2^30 keys of pages of 16
    assert call(f, ok, n_seqs=(1 << 20) + 1) == UNSUPPORTED
    assert call(f, ok, ws=None) == WORKSPACE and call(f, ok, ws_bytes=need - 1) == WORKSPACE
    assert call(f, ok, n_seqs=0, Q=None, O=None, pages=None, lens=None) == _abi.BITNET_OK
