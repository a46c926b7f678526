"""GPU gradient of RMSNorm with a residual branch against the formula in 64
bits and against differences of the forward.

Bounds, with u = 2^-24 and the formula's own terms (e = dY w, h, r given):
  dH: the dot product of K terms is a sum of fp32 products (three roundings in a
      term: e, u = h r, the product) added in some order: |err| <= (K + 4) u
      sum |e u|; the result has five more roundings of terms no larger than
      |r e|, |r u m| and |dR|, and one to its type.
  dw: T terms with three roundings each, added in some order: (T + 4) u sum |dY u|.
"""
import numpy as np
import pytest

from sparse_linear_layers_bitnet_b200 import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
U = 2.0 ** -24


@pytest.fixture(scope="module")
def bn(cuda_device):
    import sparse_linear_layers_bitnet_b200 as m
    m.load()
    return m


def bf16(x):
    return synth.bf16_bits_to_f32(synth.to_bf16_bits(x))


def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dtype)


def formula(dY, H, r, w, dR):
    g, h, r = dY.astype(np.float64), H.astype(np.float64), r.astype(np.float64)[:, None]
    K = h.shape[1]
    e = g * (1.0 if w is None else w.astype(np.float64))
    u = h * r
    m = (e * u).sum(1, keepdims=True) / K
    am = np.abs(e * u).sum(1, keepdims=True) / K
    dH = r * (e - u * m) + (0.0 if dR is None else dR.astype(np.float64))
    bound = np.abs(r * u) * ((K + 4) * U * am) + 6 * U * (np.abs(r * e) + np.abs(r * u * m) + np.abs(dH))
    dw = (g * u).sum(0)
    return dH, bound, dw, (H.shape[0] + 4) * U * np.abs(g * u).sum(0)


def inputs(T, K, dy, g, weighted, residual, seed):
    r = np.random.default_rng(seed)
    H = bf16((r.normal(size=(T, K)) * np.where(r.random(K) < 0.02, 20.0, 1.0)).astype(np.float32))
    if T > 1:
        H[1] = 0.0                                   # r = eps^-1/2, the largest factor
    dY = (0.01 * r.normal(size=(T, K))).astype(np.float32)
    dR = (0.01 * r.normal(size=(T, K))).astype(np.float32) if residual else None
    if dy == torch.bfloat16:
        dY = bf16(dY)
    if residual and g == torch.bfloat16:
        dR = bf16(dR)
    rinv = (1.0 / np.sqrt((H.astype(np.float64) ** 2).mean(1) + 1e-6)).astype(np.float32)
    w = (1 + 0.1 * r.normal(size=K)).astype(np.float32) if weighted else None
    return dY, H, rinv, w, dR


def check(got, ref, bound, dtype):
    got = got.float().cpu().numpy().astype(np.float64)
    if dtype == torch.bfloat16:                      # one rounding to bf16, of a value within bound of ref
        bound = bound + 2.0 ** -8 * (np.abs(ref) + bound) + 2.0 ** -134
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - ref) <= bound + 1e-37)


# K: one chunk, every register width (1, 2 and 3 chunks a thread), ragged warps, and rows beyond them
@pytest.mark.parametrize("T,K", [(1, 8), (1, 2560), (3, 264), (700, 520), (33, 3200), (300, 4104), (13, 8192), (9, 8640), (7, 9240), (5, 16384),
                                 (301, 16392), (3, 65536)])
@pytest.mark.parametrize("dy,g,weighted,residual", [(torch.bfloat16, torch.bfloat16, True, True),
                                                    (torch.float32, torch.bfloat16, True, False),
                                                    (torch.float32, torch.float32, False, True),
                                                    (torch.bfloat16, torch.float32, True, False)])
def test_against_the_formula(bn, T, K, dy, g, weighted, residual):
    dY, H, rinv, w, dR = inputs(T, K, dy, g, weighted, residual, T + K)
    ref, bound, dw_ref, dw_bound = formula(dY, H, rinv, w, dR)
    out = torch.full((T, K), float("nan"), dtype=g, device="cuda")
    dH, dw = bn.bitnet_rmsnorm_grad(dev(dY, dy), dev(H, torch.bfloat16), dev(rinv, torch.float32),
                                    w=None if w is None else dev(w, torch.float32),
                                    dR=None if dR is None else dev(dR, g), dH=out)
    assert dH is out
    check(dH, ref, bound, g)
    check(dw, dw_ref, dw_bound, torch.float32)


def test_against_differences(bn):
    """L(h) = sum dY y(h) + sum dR h along random directions, in 64 bits: the central difference at
    step 2^-10 has an error of its third derivative's order, 1e-6 of |L'| here; the bound takes 1e-4."""
    r = np.random.default_rng(7)
    T, K = 4, 512
    dY, H, rinv, w, dR = inputs(T, K, torch.float32, torch.float32, True, True, 7)
    H = bf16(r.normal(size=(T, K)).astype(np.float32))
    rinv = (1.0 / np.sqrt((H.astype(np.float64) ** 2).mean(1) + 1e-6)).astype(np.float32)
    dH, dw = bn.bitnet_rmsnorm_grad(dev(dY, torch.float32), dev(H, torch.bfloat16), dev(rinv, torch.float32),
                                    w=dev(w, torch.float32), dR=dev(dR, torch.float32),
                                    dH=torch.empty((T, K), device="cuda"))
    dH, dw = dH.cpu().numpy().astype(np.float64), dw.cpu().numpy().astype(np.float64)

    def loss(h, ww):
        y = h / np.sqrt((h ** 2).mean(1, keepdims=True) + 1e-6) * ww
        return (dY.astype(np.float64) * y).sum() + (dR.astype(np.float64) * h).sum()
    h0, w0, s = H.astype(np.float64), w.astype(np.float64), 2.0 ** -10
    for _ in range(8):
        v, z = r.normal(size=(T, K)), r.normal(size=K)
        d = (loss(h0 + s * v, w0) - loss(h0 - s * v, w0)) / (2 * s)
        assert abs(d - (dH * v).sum()) <= 1e-4 * np.sqrt((dH ** 2).sum() * (v ** 2).sum())
        d = (loss(h0, w0 + s * z) - loss(h0, w0 - s * z)) / (2 * s)
        assert abs(d - (dw * z).sum()) <= 1e-4 * np.sqrt((dw ** 2).sum() * (z ** 2).sum())


@pytest.mark.parametrize("T,K", [(40, 3200), (5, 16392)])
def test_in_place_accumulation_and_repeats(bn, T, K):
    dY, H, rinv, w, dR = inputs(T, K, torch.bfloat16, torch.bfloat16, True, True, 3)
    a = (dev(dY, torch.bfloat16), dev(H, torch.bfloat16), dev(rinv, torch.float32))
    wd = dev(w, torch.float32)
    dH, dw = bn.bitnet_rmsnorm_grad(*a, w=wd, dR=dev(dR, torch.bfloat16))
    d2 = dev(dR, torch.bfloat16)
    dw2 = torch.ones(K, device="cuda")
    bn.bitnet_rmsnorm_grad(*a, w=wd, dR=d2, dH=d2, dw=dw2, accumulate=True)
    assert torch.equal(d2, dH)
    assert torch.equal(dw2, 1.0 + dw)
    ws = bn.Workspace(bn.load().bitnet_rmsnorm_grad_workspace_size(T, K))
    ws.buf.fill_(255)                                # what a workspace holds does not matter
    d3, dw3 = bn.bitnet_rmsnorm_grad(*a, w=wd, dR=dev(dR, torch.bfloat16), ws=ws)
    assert torch.equal(d3, dH) and torch.equal(dw3, dw)


def test_empty_batch(bn):
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    dw = torch.full((64,), 3.0, device="cuda")
    bn.bitnet_rmsnorm_grad(e, e, torch.empty(0, device="cuda"), dw=dw, accumulate=True)
    assert bool((dw == 3.0).all())
    bn.bitnet_rmsnorm_grad(e, e, torch.empty(0, device="cuda"), dw=dw)
    assert not dw.any()


def test_captured_and_replayed(bn):
    dY, H, rinv, w, dR = inputs(65, 2560, torch.float32, torch.bfloat16, True, True, 11)
    x = [dev(dY, torch.float32), dev(H, torch.bfloat16), dev(rinv, torch.float32)]
    kw = dict(w=dev(w, torch.float32), dR=dev(dR, torch.bfloat16))
    ws = bn.Workspace(bn.load().bitnet_rmsnorm_grad_workspace_size(65, 2560))
    dH, dw = torch.empty_like(x[1]), torch.empty(2560, device="cuda")
    ref = bn.bitnet_rmsnorm_grad(*x, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bn.bitnet_rmsnorm_grad(*x, **kw, dH=dH, dw=dw, ws=ws)
    for _ in range(2):
        dH.zero_(), dw.zero_()
        g.replay()
        assert torch.equal(dH, ref[0]) and torch.equal(dw, ref[1])


def test_refusals(bn):
    H = torch.zeros((4, 512), dtype=torch.bfloat16, device="cuda")
    r = torch.ones(4, device="cuda")
    with pytest.raises(AssertionError):
        bn.bitnet_rmsnorm_grad(H[:3], H, r)
    with pytest.raises(AssertionError):
        bn.bitnet_rmsnorm_grad(H, H, r, dR=H, dH=torch.empty((4, 512), device="cuda"))
    with pytest.raises(bn.BitnetError):
        bn.bitnet_rmsnorm_grad(H.clone(), H, r, dH=H)
    with pytest.raises(bn.BitnetError):
        bn.bitnet_rmsnorm_grad(H.clone(), H, r, ws=bn.Workspace(256))


@pytest.mark.parametrize("T,K", [(40, 3200), (300, 12288), (300, 12296)])
@pytest.mark.parametrize("residual", [True, False])
def test_without_the_weight_gradient(bn, T, K, residual):
    """The longest row of the register form and the shortest beyond it: dH is the same with dw and without."""
    dY, H, rinv, w, dR = inputs(T, K, torch.float32, torch.bfloat16, True, residual, K)
    a = (dev(dY, torch.float32), dev(H, torch.bfloat16), dev(rinv, torch.float32))
    kw = dict(w=dev(w, torch.float32), dR=dev(dR, torch.bfloat16) if residual else None)
    dH, dw = bn.bitnet_rmsnorm_grad(*a, **kw)
    alone, none = bn.bitnet_rmsnorm_grad(*a, **kw, need_dw=False)
    assert none is None and torch.equal(alone, dH)
    ref, bound, dw_ref, dw_bound = formula(dY, H, rinv, w, dR)
    check(dH, ref, bound, torch.bfloat16)
    check(dw, dw_ref, dw_bound, torch.float32)
    with pytest.raises(AssertionError):
        bn.bitnet_rmsnorm_grad(*a, **kw, dw=dw, need_dw=False)
