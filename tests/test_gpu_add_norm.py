"""GPU parity of the residual addition fused with RMSNorm and the per-token
quantisation: the new residual stream, codes, absmax and norm factor bit-exact
against the oracle's rmsnorm and quant_act of bf16(X + R).

"BitNet b1.58: Ternary Weights for 1.58-bit LLMs", "What this paper explains"
(LLaMA-alike pre-norm blocks) and "The mechanism" (per-token absmax int8
activations).
"""
import numpy as np
import pytest

import oracle
from sparse_linear_layers_bitnet_b200 import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def bn(cuda_device):
    import sparse_linear_layers_bitnet_b200 as m
    m.load()
    return m


def bf16_dev(a_f32):
    bits = synth.to_bf16_bits(a_f32)
    return torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16), synth.bf16_bits_to_f32(bits)


def _sum_bits(X, R):
    """bf16 bits of the exact sum: fp64 holds every sum of two bf16 values whose
    exponents are less than 45 apart, and further apart the larger one is the
    rounded sum; fp64 to bf16 goes through fp32 rounded to odd, so that the
    result is rounded once."""
    s = X.astype(np.float64) + R.astype(np.float64)
    f = s.astype(np.float32)
    up = np.abs(f.astype(np.float64)) > np.abs(s)          # truncate towards zero, then set the sticky bit
    u = f.view(np.uint32).copy()
    u[up] -= 1
    inexact = u.view(np.float32).astype(np.float64) != s
    u[inexact] |= 1
    return synth.to_bf16_bits(u.view(np.float32))


def _rows(T, K, seed):
    r = np.random.default_rng(seed)
    X = r.normal(size=(T, K)).astype(np.float32)
    R = (r.normal(size=(T, K)) * np.where(r.random(K) < 0.02, 20.0, 1.0)).astype(np.float32)
    if T > 2:
        R[1] = -X[1]                                        # the sum vanishes: absmax is the floor
        X[2] *= np.float32(2.0) ** r.integers(-60, 60, K).astype(np.float32)     # far exponents, ties of the addition
        R[2] *= np.float32(2.0) ** r.integers(-60, 60, K).astype(np.float32)
    if T > 4:
        X[3] *= 1e-30
        R[3] *= 1e-38                                       # subnormal summands
        X[4, ::2] = 0.0
        R[4] = 0.0
    return X, R


@pytest.mark.parametrize("T,K,weighted", [(1, 8, False), (1, 2560, True), (7, 264, True), (33, 3200, True), (5, 4096, False),
                                          (6, 8640, True), (5, 16384, True), (5, 20000, True), (5, 32768, True),
                                          (5, 40000, True), (5, 65536, False), (300, 3200, True), (2400, 264, False)])
def test_add_rmsnorm_quant_matches_the_oracle(bn, T, K, weighted):
    Xf, Rf = _rows(T, K, T * 7 + K)
    Xd, X = bf16_dev(Xf)
    Rd, R = bf16_dev(Rf)
    w = (1 + 0.1 * np.random.default_rng(K).normal(size=K)).astype(np.float32) if weighted else None
    wd = torch.from_numpy(w).cuda() if weighted else None
    Hb = _sum_bits(X, R)
    Hf = synth.bf16_bits_to_f32(Hb)
    xn, r = oracle.rmsnorm(Hf, 1e-6, w, return_r=True)
    q, a = oracle.quant_act(xn, 1e-5)
    H, Xq, am, rinv = bn.bitnet_add_rmsnorm_quant(Xd, Rd, w=wd)
    torch.cuda.synchronize()
    assert np.array_equal(H.view(torch.int16).cpu().numpy().view(np.uint16), Hb)
    assert np.array_equal(rinv.cpu().numpy(), r)
    assert np.array_equal(am.cpu().numpy(), a)
    assert np.array_equal(Xq.cpu().numpy(), q)


@pytest.mark.parametrize("K", [512, 3200, 24576, 40960])
@pytest.mark.parametrize("into", ["X", "R"])
def test_the_sum_may_go_into_an_input(bn, K, into):
    Xd, _ = bf16_dev(synth.activations(9, K, seed=K))
    Rd, _ = bf16_dev(synth.activations(9, K, seed=K + 1, outlier_p=0.01))
    ref = bn.bitnet_add_rmsnorm_quant(Xd, Rd)
    other = Rd.clone() if into == "X" else Xd.clone()
    got = bn.bitnet_add_rmsnorm_quant(Xd, Rd, H=Xd if into == "X" else Rd)
    torch.cuda.synchronize()
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    assert torch.equal(Rd if into == "X" else Xd, other)


@pytest.mark.parametrize("K", [2560, 32776])
def test_a_weight_off_16_bytes_gives_the_same(bn, K):
    Xd, _ = bf16_dev(synth.activations(4, K, seed=1))
    Rd, _ = bf16_dev(synth.activations(4, K, seed=2))
    w = torch.rand(K + 1, device="cuda") + 0.5
    ref = bn.bitnet_add_rmsnorm_quant(Xd, Rd, w=w[1:].clone())
    got = bn.bitnet_add_rmsnorm_quant(Xd, Rd, w=w[1:])
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_same_as_rmsnorm_quant_of_the_sum(bn):
    Xd, _ = bf16_dev(synth.activations(300, 3200, seed=3))
    Rd, _ = bf16_dev(synth.activations(300, 3200, seed=4, outlier_p=0.01))
    w = torch.rand(3200, device="cuda") + 0.5
    H, Xq, am, rinv = bn.bitnet_add_rmsnorm_quant(Xd, Rd, w=w)
    r2 = torch.empty(300, device="cuda")
    Xq2, am2 = bn.bitnet_rmsnorm_quant(H, w, rinv=r2)
    assert torch.equal(H, Xd + Rd)
    assert torch.equal(Xq, Xq2) and torch.equal(am, am2) and torch.equal(rinv, r2)


def test_empty_batch_and_another_stream(bn):
    e = torch.empty((0, 512), dtype=torch.bfloat16, device="cuda")
    assert bn.bitnet_add_rmsnorm_quant(e, e)[1].shape == (0, 512)
    Xd, _ = bf16_dev(synth.activations(64, 2560, seed=5))
    Rd, _ = bf16_dev(synth.activations(64, 2560, seed=6))
    ref = bn.bitnet_add_rmsnorm_quant(Xd, Rd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = bn.bitnet_add_rmsnorm_quant(Xd, Rd, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_refusals(bn):
    X = torch.zeros((4, 512), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(AssertionError):
        bn.bitnet_add_rmsnorm_quant(X, X[:2])
    with pytest.raises(AssertionError):
        bn.bitnet_add_rmsnorm_quant(X.float(), X)
    with pytest.raises(AssertionError):
        bn.bitnet_add_rmsnorm_quant(X, X, w=torch.ones(512, device="cuda", dtype=torch.bfloat16))
    buf = torch.zeros((6, 512), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(bn.BitnetError):   # overlaps X by two rows
        bn.bitnet_add_rmsnorm_quant(buf[:4], X, H=buf[2:])


def _not_finite(bn, T, K, weighted, off, fused):
    """Rows with Inf, -Inf, NaN, both infinities, squares that overflow fp32, a weight of NaN; against the definition:
    ms is Inf or NaN, r = 1 / sqrt(ms) 0 or NaN, absmax the largest |x r w| with NaN where one is, and no codes then."""
    r = np.random.default_rng(K)
    X, R = (r.normal(size=(T, K)).astype(np.float32) for _ in range(2))
    X[1, K // 2], X[2, K - 1], X[3, 0] = np.inf, -np.inf, np.nan
    X[4, 5], X[4, K - 8] = np.inf, -np.inf
    X[5, 1], X[5, 2] = np.nan, np.inf
    X[6] *= np.float32(2.0 ** 66)                           # finite, mean square above the fp32 range
    X[7, 3], R[7, 3] = 3e38, 3e38                           # the sum overflows
    if not fused:
        R[:] = 0.0
        X[7, 3] = np.inf
    Xd, Xh = bf16_dev(X)
    Rd, Rh = bf16_dev(R)
    wd = (torch.rand(K + 1, device="cuda") + 0.5)[1 if off else 0:][:K] if weighted else None
    with np.errstate(all="ignore"):
        if fused:
            H, Xq, am, rinv = bn.bitnet_add_rmsnorm_quant(Xd, Rd, w=wd)
        else:
            rinv = torch.empty(T, device="cuda")
            Xq, am = bn.bitnet_rmsnorm_quant(Xd, wd, rinv=rinv)
            H = Xd
        h = (Xh + Rh).astype(np.float32) if fused else Xh
        hb = synth.bf16_bits_to_f32(synth.to_bf16_bits(np.where(np.isnan(h), np.float32(0), h)))
        hb[np.isnan(h)] = np.nan
        got = H.float().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(hb)) and np.array_equal(got[~np.isnan(hb)], hb[~np.isnan(hb)])
        ms = (hb.astype(np.float64) ** 2).mean(1).astype(np.float32)
        rr = (1 / np.sqrt(ms + np.float32(1e-6))).astype(np.float32)
        a = np.abs(hb * rr[:, None] * (1 if wd is None else wd.cpu().numpy())).max(1)
    bad = [1, 2, 3, 4, 5, 7]
    am, rinv, Xq = am.cpu().numpy(), rinv.cpu().numpy(), Xq.cpu().numpy()
    assert np.isnan(a[bad]).all() and np.isnan(am[bad]).all()
    assert np.array_equal(np.isnan(rinv), np.isnan(rr)) and np.isnan(rr[[3, 5]]).all()
    assert not rinv[[1, 2, 4, 6, 7]].any() and not rr[[1, 2, 4, 6, 7]].any()
    assert not Xq[bad + [6]].any() and am[6] == np.float32(1e-5)
    fine = np.setdiff1d(np.arange(T), bad + [6])            # the other rows are the oracle's, bit for bit
    xn, ro = oracle.rmsnorm(hb[fine], 1e-6, None if wd is None else wd.cpu().numpy(), return_r=True)
    q, ao = oracle.quant_act(xn, 1e-5)
    assert np.array_equal(rinv[fine], ro) and np.array_equal(am[fine], ao) and np.array_equal(Xq[fine], q)
    if wd is not None:                                      # a weight of NaN, or of Inf, is seen as well
        for v in (float("nan"), float("inf")):
            wd[K - 3] = v
            _, Xq, am, rinv = bn.bitnet_add_rmsnorm_quant(Xd, Rd, w=wd)
            assert not bool(torch.isfinite(am).any()) and not Xq.any() and np.array_equal(rinv.cpu().numpy()[fine], ro)


@pytest.mark.parametrize("K,weighted,off", [(40000, True, False), (40000, False, False), (2560, True, True), (33000, True, True)])
@pytest.mark.parametrize("fused", [True, False])
def test_rows_that_are_not_finite_in_the_general_form(bn, K, weighted, off, fused):
    _not_finite(bn, 9, K, weighted, off, fused)


@pytest.mark.parametrize("T,K,weighted", [(9, 32, False), (9, 264, True), (9, 2560, True), (9, 3200, False), (9, 8640, True), (9, 16384, False),
                                          (9, 32768, True), (2500, 32, False), (2500, 264, True), (2500, 2560, True), (2500, 3200, False)])
@pytest.mark.parametrize("fused", [True, False])
def test_rows_that_are_not_finite(bn, T, K, weighted, fused):
    """Every width of the register form, and many rows, which take fewer threads each."""
    _not_finite(bn, T, K, weighted, False, fused)
