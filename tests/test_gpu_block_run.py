"""The block operators together, as a decode step and as a training step use
them: each stage's result against the definition on the stage's own inputs, and
a captured step replayed over growing caches against the same calls one by one.

"BitNet b1.58 ...", section "What this paper explains" (LLaMA-alike blocks);
"Sparse-BitNet" (gist.science), section 2 "Training Strategie" (straight-through
gradients).
"""
import numpy as np
import pytest

import oracle
from sparse_linear_layers_bitnet_b200 import synth
from tests.test_gpu_norm_grad import formula
from tests.test_gpu_rope import bf16, host, table_ref, turn, up

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF16, F32 = torch.bfloat16, torch.float32
HID, HEADS, KV, D, FFN, PAGE = 512, 4, 2, 128, 1024, 16


@pytest.fixture(scope="module")
def bn(cuda_device):
    import sparse_linear_layers_bitnet_b200 as m
    m.load()
    return m


def packed(bn, n_out, k, seed):
    pw = bn.PackedWeights(n_out, k)
    bn.bitnet_pack_nm(torch.from_numpy(synth.master_weights(n_out, k, 0.02, seed=seed)).cuda(), pw)
    return pw


class Block:
    """One pre-norm block's weights, cache and buffers for a batch of one-token sequences."""

    def __init__(self, bn, B, seed=0):
        self.bn, self.B = bn, B
        self.qkv = packed(bn, (HEADS + 2 * KV) * D, HID, seed + 1)
        self.o = packed(bn, HID, HEADS * D, seed + 2)
        self.gate_up = packed(bn, 2 * FFN, HID, seed + 3)
        self.down = packed(bn, HID, FFN, seed + 4)
        self.w1, self.w2 = (up(1 + 0.1 * np.random.default_rng(seed + 5 + i).normal(size=HID).astype(np.float32)) for i in range(2))
        most = 4
        self.K, self.V = bn.kv_cache(B * most + 1, KV, PAGE, D), bn.kv_cache(B * most + 1, KV, PAGE, D)
        self.pages = up(np.random.default_rng(seed).permutation(B * most).reshape(B, most), torch.int32)
        self.table = bn.rope_table(PAGE * most, D)
        self.ws = bn.Workspace(bn.load().bitnet_paged_attn_workspace_size(B, HEADS, KV, D))
        self.lin_ws = bn.Workspace(max(bn.load().bitnet_linear_workspace_size(),
                                       bn.load().bitnet_quant_linear_workspace_size(B, HEADS * D)))

    def step(self, x, delta, pos, lens):
        """The residual stream x plus the previous block's delta goes in; returns all that the step makes."""
        bn, s = self.bn, {}
        s["h1"], s["q1"], s["a1"], s["r1"] = bn.bitnet_add_rmsnorm_quant(delta, x, w=self.w1)
        s["qkv"] = bn.bitnet_sparse_linear(s["q1"], s["a1"], self.qkv, ws=self.lin_ws)
        s["q"] = bn.bitnet_rope_append(s["qkv"], pos, self.table, self.K, self.V, self.pages, ws=self.ws)
        s["att"] = bn.bitnet_paged_attn(s["q"], self.K, self.V, self.pages, lens, ws=self.ws)
        s["oout"] = bn.bitnet_quant_linear(s["att"], self.o, ws=self.lin_ws)
        s["h2"], s["q2"], s["a2"], s["r2"] = bn.bitnet_add_rmsnorm_quant(s["oout"], s["h1"], w=self.w2)
        s["gu"] = bn.bitnet_sparse_linear(s["q2"], s["a2"], self.gate_up, ws=self.lin_ws)
        s["qf"], s["af"] = bn.bitnet_swiglu_quant(s["gu"], FFN)
        s["out"] = bn.bitnet_sparse_linear(s["qf"], s["af"], self.down, ws=self.lin_ws)
        return s


def check_norm(x, delta, w, h, q, a):
    ref_h = bf16((host(delta) + host(x)).astype(np.float32))
    xn = oracle.rmsnorm(ref_h, 1e-6, host(w).astype(np.float32))
    rq, ra = oracle.quant_act(xn, 1e-5)
    assert np.array_equal(host(h), ref_h) and np.array_equal(q.cpu().numpy(), rq) and np.array_equal(a.cpu().numpy(), ra)


@pytest.mark.parametrize("B", [1, 3, 8, 33])   # the decode products and, above eight tokens, the tensor-core GEMM
def test_decode_steps(bn, B):
    blk = Block(bn, B)
    r = np.random.default_rng(B)
    start = r.integers(0, 40, B)
    for b in range(B):   # what the sequences hold already
        n = int(start[b])
        if n:
            qkv = up(r.normal(size=(n, (HEADS + 2 * KV) * D)).astype(np.float32), BF16)
            bn.bitnet_rope_append(qkv, up(np.arange(n), torch.int32), blk.table, blk.K, blk.V, blk.pages,
                                  seq=torch.full((n,), b, dtype=torch.int32, device="cuda"), ws=blk.ws)
    K0, V0 = host(blk.K), host(blk.V)
    tab = table_ref(PAGE * 4, D)
    pages = blk.pages.cpu().numpy()
    pos, lens = up(start, torch.int32), up(start + 1, torch.int32)
    x = up(r.normal(size=(B, HID)).astype(np.float32), BF16)
    delta = up(r.normal(size=(B, HID)).astype(np.float32), BF16)
    x0, d0, made = x.clone(), delta.clone(), []
    for step in range(4):
        s = blk.step(x, delta, pos, lens)
        assert bn.bitnet_read_device_status(blk.ws) == 0
        check_norm(x, delta, blk.w1, s["h1"], s["q1"], s["a1"])
        check_norm(s["h1"], s["oout"], blk.w2, s["h2"], s["q2"], s["a2"])
        at = start + step
        heads = host(s["qkv"]).reshape(B, -1, D).astype(np.float32)
        qk = bf16(turn(heads[:, :HEADS + KV], tab[at], False))
        assert np.array_equal(host(s["q"]).reshape(B, HEADS, D), qk[:, :HEADS])
        for b in range(B):
            page, row = pages[b, at[b] // PAGE], at[b] % PAGE
            K0[page, :, row], V0[page, :, row] = qk[b, HEADS:], heads[b, HEADS + KV:]
        assert np.array_equal(host(blk.K), K0) and np.array_equal(host(blk.V), V0)
        for b in range(B):
            n = at[b] + 1
            k = K0[pages[b]].transpose(1, 0, 2, 3).reshape(KV, -1, D)[:, :n].astype(np.float64)
            v = V0[pages[b]].transpose(1, 0, 2, 3).reshape(KV, -1, D)[:, :n].astype(np.float64)
            z = np.einsum("hgd,hnd->hgn", qk[b, :HEADS].reshape(KV, -1, D).astype(np.float64), k) * D ** -0.5
            p = np.exp(z - z.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            ref, size = np.einsum("hgn,hnd->hgd", p, v).reshape(-1), np.einsum("hgn,hnd->hgd", p, np.abs(v)).reshape(-1)
            # sum |q k| scale stays below 4 here: the scores are within 132 2^-23 4 of theirs, the weights within twice
            # that, 2^-12; 2^-11 also covers the weights' own 2^-17 and the sums.  Then one rounding to bf16.
            assert np.einsum("hgd,hnd->hgn", np.abs(qk[b, :HEADS].reshape(KV, -1, D)), np.abs(k)).max() * D ** -0.5 < 4
            assert np.all(np.abs(host(s["att"])[b] - ref) <= 2.0 ** -11 * size + 2.0 ** -8 * (np.abs(ref) + 2.0 ** -11 * size))
        made.append({k: s[k].clone() for k in ("out", "h2")})
        x, delta = s["h2"], s["out"]
        pos.add_(1)
        lens.add_(1)

    # the same steps captured once and replayed, on a cache that holds what it held at the start
    again = Block(bn, B)
    again.K.copy_(up(K0, BF16)), again.V.copy_(up(V0, BF16))
    pos, lens = up(start, torch.int32), up(start + 1, torch.int32)
    gx, gd = x0.clone(), d0.clone()
    again.step(gx, gd, pos, lens)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s = again.step(gx, gd, pos, lens)
        gx.copy_(s["h2"])
        gd.copy_(s["out"])
        pos.add_(1)
        lens.add_(1)
    gx.copy_(x0), gd.copy_(d0)
    for step in range(4):
        g.replay()
        assert torch.equal(gx, made[step]["h2"]) and torch.equal(gd, made[step]["out"])


def test_training_step(bn):
    """Forward to the rotated heads, and back: the inverse rotation, the product's input gradient (fp32), the norm's."""
    T, r = 200, np.random.default_rng(1)
    blk = Block(bn, 1, seed=40)
    x, o = (up(r.normal(size=(T, HID)).astype(np.float32), BF16) for _ in range(2))
    h, q, a, rinv = bn.bitnet_add_rmsnorm_quant(o, x, w=blk.w1)
    check_norm(x, o, blk.w1, h, q, a)
    qkv = bn.bitnet_sparse_linear(q, a, blk.qkv)
    pos = up(np.arange(T) % 64, torch.int32)
    before = host(qkv).astype(np.float32)
    bn.bitnet_rope(qkv, pos, blk.table, HEADS + KV, D, Y=qkv)
    tab = table_ref(64, D)
    want = before.reshape(T, -1, D).copy()
    want[:, :HEADS + KV] = bf16(turn(want[:, :HEADS + KV], tab[np.arange(T) % 64], False))
    assert np.array_equal(host(qkv), want.reshape(T, -1))

    g = up((0.01 * r.normal(size=(T, (HEADS + 2 * KV) * D))).astype(np.float32), BF16)   # from attention's backward
    g0 = host(g).astype(np.float32).reshape(T, -1, D)
    up_grad = up((0.01 * r.normal(size=(T, HID))).astype(np.float32), BF16)              # the residual stream's
    bn.bitnet_rope(g, pos, blk.table, HEADS + KV, D, inverse=True, Y=g)
    g0[:, :HEADS + KV] = bf16(turn(g0[:, :HEADS + KV], tab[np.arange(T) % 64], False, True))
    assert np.array_equal(host(g), g0.reshape(T, -1))
    dy = bn.bitnet_dgrad(g, blk.qkv, dx_dtype=F32)
    dh, dw = bn.bitnet_rmsnorm_grad(dy, h, rinv, w=blk.w1, dR=up_grad)
    ref, bound, dw_ref, dw_bound = formula(host(dy), host(h), host(rinv), host(blk.w1), host(up_grad))
    assert np.all(np.abs(host(dh) - ref) <= bound + 2.0 ** -8 * (np.abs(ref) + bound))
    assert np.all(np.abs(host(dw) - dw_ref) <= dw_bound)


@pytest.mark.parametrize("B", [1, 8, 33])
def test_captured_decode_steps_write_the_cache(bn, B):
    """Four steps one by one, and the same captured and replayed on a cache that holds NaN behind what the sequences held
    at the start: every replay has to write its own keys and values before it reads them."""
    r = np.random.default_rng(100 + B)
    start = r.integers(0, 40, B)
    blk = Block(bn, B, seed=B)
    blk.K.fill_(float("nan")), blk.V.fill_(float("nan"))
    for b in range(B):
        n = int(start[b])
        if n:
            qkv = up(r.normal(size=(n, (HEADS + 2 * KV) * D)).astype(np.float32), BF16)
            bn.bitnet_rope_append(qkv, up(np.arange(n), torch.int32), blk.table, blk.K, blk.V, blk.pages,
                                  seq=torch.full((n,), b, dtype=torch.int32, device="cuda"), ws=blk.ws)
    first = [t.clone() for t in (blk.K, blk.V)]
    pos, lens = up(start, torch.int32), up(start + 1, torch.int32)
    x0, d0 = (up(r.normal(size=(B, HID)).astype(np.float32), BF16) for _ in range(2))
    x, delta, made = x0, d0, []
    for _ in range(4):
        s = blk.step(x, delta, pos, lens)
        x, delta = s["h2"], s["out"]
        assert not bool(torch.isnan(x.float()).any() or torch.isnan(delta.float()).any())
        made.append((x.clone(), delta.clone()))
        pos.add_(1), lens.add_(1)
    last = [t.clone() for t in (blk.K, blk.V)]
    assert int(torch.isnan(first[0].float()).sum() - torch.isnan(last[0].float()).sum()) == 4 * B * KV * D

    gx, gd = x0.clone(), d0.clone()
    pos, lens = up(start, torch.int32), up(start + 1, torch.int32)
    blk.step(gx, gd, pos, lens)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s = blk.step(gx, gd, pos, lens)
        gx.copy_(s["h2"]), gd.copy_(s["out"])
        pos.add_(1), lens.add_(1)
    blk.K.copy_(first[0]), blk.V.copy_(first[1])
    gx.copy_(x0), gd.copy_(d0)
    pos.copy_(up(start, torch.int32)), lens.copy_(up(start + 1, torch.int32))
    for x, delta in made:
        g.replay()
        assert torch.equal(gx, x) and torch.equal(gd, delta)
    for got, want in zip((blk.K, blk.V), last):
        assert torch.equal(torch.nan_to_num(got, nan=3.0), torch.nan_to_num(want, nan=3.0))
    assert bn.bitnet_read_device_status(blk.ws) == 0
