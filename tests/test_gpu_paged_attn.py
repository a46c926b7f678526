"""GPU one-token attention over the paged cache against the softmax in 64 bits.

Bound per output, with u = 2^-24, x_j = scale q . k_j, p_j its softmax weight
and n keys:
  * a score is an fp32 sum of head_dim exact products (factor 2 for a tensor
    core that truncates instead of rounding) times a rounded constant:
    |dx_j| <= scale (head_dim + 4) 2 u sum_i |q_i k_ij| + 4 u |x_j| =: e_j; a
    weight and the sum of weights then move by at most exp(2 max e) - 1;
  * 2^x has a relative error of 2^-22 and a weight keeps 17 bits in its two
    parts (2^-17 relative);
  * sums over n keys, with one rescaling or joining step for each tile, warp and
    range: (2 n + 64) u of sum_j p_j |v_j|, again times 2;
  * one rounding to the output's type.
"""
import numpy as np
import pytest

from sparse_linear_layers_bitnet_b200 import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def bn(cuda_device):
    import sparse_linear_layers_bitnet_b200 as m
    m.load()
    return m


def bf16(x):
    return synth.bf16_bits_to_f32(synth.to_bf16_bits(x))


def up(x, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dtype)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


class Case:
    """A cache whose every unused place (rows behind a length, other pages, columns behind head_dim) is NaN."""

    def __init__(self, lens, heads, kv, d, page, layout="heads first", seed=0, spread=1.0, extra=2):
        r = np.random.default_rng(seed)
        self.lens, self.heads, self.kv, self.d, self.page = lens, heads, kv, d, page
        B, ld = len(lens), -(-d // 8) * 8
        counts = [-(-n // page) for n in lens]
        n_pages = sum(counts) + extra
        order = r.permutation(n_pages)
        self.pages = np.full((B, max(1, max(counts))), -1, np.int32)
        at = 0
        for b, c in enumerate(counts):
            self.pages[b, :c] = order[at:at + c]
            at += c
        shape = (n_pages, kv, page, ld) if layout == "heads first" else (n_pages, page, kv, ld)
        base = np.full((2,) + shape, np.nan, np.float32)
        view = base if layout == "heads first" else base.transpose(0, 1, 3, 2, 4)
        self.k, self.v = [], []
        for b, n in enumerate(lens):
            k, v = (bf16((r.normal(size=(kv, n, d)) * spread).astype(np.float32)) for _ in range(2))
            self.k.append(k)
            self.v.append(v)
            for j in range(counts[b]):
                part = slice(j * page, min(n, (j + 1) * page))
                rows = part.stop - part.start
                view[0, self.pages[b, j], :, :rows, :d] = k[:, part]
                view[1, self.pages[b, j], :, :rows, :d] = v[:, part]
        dev = up(base, BF16)
        if layout != "heads first":
            dev = dev.permute(0, 1, 3, 2, 4)
        self.K, self.V = dev[0][..., :d], dev[1][..., :d]
        self.q = bf16((r.normal(size=(B, heads * d)) * spread).astype(np.float32))
        self.scale = d ** -0.5

    def args(self):
        return up(self.q, BF16), self.K, self.V, up(self.pages, torch.int32), up(np.array(self.lens), torch.int32)

    def ref(self):
        B, G = len(self.lens), self.heads // self.kv
        O, bound = np.zeros((2, B, self.heads, self.d))
        lse, lbound = np.full((B, self.heads), -np.inf), np.zeros((B, self.heads))
        for b, n in enumerate(self.lens):
            if n == 0:
                continue
            q = self.q[b].reshape(self.kv, G, self.d).astype(np.float64)
            k, v = self.k[b].astype(np.float64), self.v[b].astype(np.float64)
            x = np.einsum("hgd,hnd->hgn", q, k) * self.scale
            e = abs(self.scale) * (self.d + 4) * 2 * U * np.einsum("hgd,hnd->hgn", np.abs(q), np.abs(k)) + 4 * U * np.abs(x)
            top = x.max(-1, keepdims=True)
            p = np.exp(x - top)
            s = p.sum(-1, keepdims=True)
            p /= s
            e = e.max(-1, keepdims=True)
            rel = np.expm1(2 * e) + 2.0 ** -22 + 2.0 ** -17 + 2 * (2 * n + 64) * U
            O[b] = np.einsum("hgn,hnd->hgd", p, v).reshape(self.heads, self.d)
            bound[b] = (rel * np.einsum("hgn,hnd->hgd", p, np.abs(v))).reshape(self.heads, self.d)
            lse[b] = (top + np.log(s)).reshape(-1)
            lbound[b] = (e + 2.0 ** -22 + 2 * (2 * n + 64) * U).reshape(-1) + 8 * U * (np.abs(lse[b]) + 1)
        return O.reshape(B, -1), bound.reshape(B, -1), lse, lbound


def check(got, ref, bound, dtype):
    step = 2.0 ** -8 if dtype == BF16 else U
    got = host(got)
    assert np.all(np.isfinite(got))
    err = np.abs(got - ref) - (bound + step * (np.abs(ref) + bound) + 1e-37)
    assert np.all(err <= 0), float(err.max())


def run(bn, c, dtype=BF16, **kw):
    lse = torch.full((len(c.lens), c.heads), float("nan"), device="cuda")
    q, K, V, pages, lens = c.args()
    n = bn.load().bitnet_paged_attn_workspace_size(len(c.lens), c.heads, c.kv, c.d)
    ws = bn.Workspace(n)
    ws.buf[256:].fill_(255)      # what a workspace holds behind its status word does not matter
    O = bn.bitnet_paged_attn(q, K, V, pages, lens, scale=c.scale, o_dtype=dtype, lse=lse, ws=ws, **kw)
    assert bn.bitnet_read_device_status(ws) == 0
    return O, lse


def check_case(bn, c, dtype=BF16):
    O, lse = run(bn, c, dtype)
    ref, bound, lref, lbound = c.ref()
    check(O, ref, bound, dtype)
    got = host(lse)
    none = np.isneginf(lref)
    assert np.array_equal(np.isneginf(got), none)
    assert np.all(np.abs(got[~none] - lref[~none]) <= lbound[~none])
    return O, lse


# lengths around the ends of 8-key half tiles, 16-key tiles, 64-key units, pages, and with idle slots among them
LENS = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 0, 127, 128, 129, 200, 1000]


@pytest.mark.parametrize("heads,kv,d", [(1, 1, 8), (20, 5, 128), (32, 32, 100), (8, 1, 256), (18, 2, 256), (16, 16, 64), (64, 4, 128),
                                        (40, 2, 64), (12, 4, 80), (9, 1, 96), (6, 2, 65), (4, 2, 1), (5, 5, 200)])
@pytest.mark.parametrize("page,layout,dtype", [(16, "heads first", BF16), (8, "rows first", F32), (256, "rows first", BF16)])
def test_against_the_softmax(bn, heads, kv, d, page, layout, dtype):
    check_case(bn, Case(LENS, heads, kv, d, page, layout, seed=heads + d + page), dtype)


@pytest.mark.parametrize("lens", [[1], [64], [65], [5000], [30011], [0, 0, 0], [0, 20000, 1, 300]])
@pytest.mark.parametrize("heads,kv,d", [(20, 5, 128), (4, 4, 100)])
def test_few_sequences(bn, lens, heads, kv, d):
    check_case(bn, Case(lens, heads, kv, d, 32, seed=len(lens)))


def test_many_sequences(bn):
    """More sequences than a CTA has threads, more units than CTAs, every length from 0 up."""
    r = np.random.default_rng(0)
    check_case(bn, Case([int(x) for x in r.permutation(np.arange(300) % 90)], 4, 2, 64, 16, seed=3))


@pytest.mark.parametrize("n,longest,heads,kv,d", [(60, 300, 32, 32, 64), (130, 400, 32, 32, 24), (128, 700, 48, 16, 40), (150, 260, 40, 1, 128)])
def test_many_short_heads(bn, n, longest, heads, kv, d):
    """More than four units per CTA: ranges that begin inside heads, at their ends and at their beginnings."""
    r = np.random.default_rng(n)
    check_case(bn, Case([int(x) for x in r.integers(0, longest + 1, n)], heads, kv, d, 16, seed=n))


def test_peaked_scores(bn):
    """Scores of both signs up to hundreds: weights that underflow, a maximum that moves late."""
    c = Case([777, 64, 129], 8, 2, 128, 16, seed=4, spread=4.0)
    for k in c.k:
        assert k.shape[0] == 2
    check_case(bn, c, F32)


def test_split_does_not_show(bn):
    """The same sequence alone (cut over many CTAs) and in a crowded batch (cut over few) within the bound;
    the same call twice gives the same bits."""
    c = Case([3001] * 40, 20, 5, 128, 16, seed=5)
    O, lse = check_case(bn, c)
    again, lse2 = run(bn, c)
    assert torch.equal(O, again) and torch.equal(lse, lse2)
    q, K, V, pages, lens = c.args()
    one = bn.bitnet_paged_attn(q[7:8], K, V, pages[7:8], lens[7:8], scale=c.scale)
    ref, bound, _, _ = c.ref()
    check(one, ref[7:8], bound[7:8], BF16)


def test_offsets_past_32_bits(bn):
    """Pages that lie more than 2^32 elements into the pool."""
    d, page, kv = 128, 64, 2
    stride = 1 << 26
    n_pages = 66                                             # 66 * 2^26 > 2^32 elements, 8.9 GB
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    pool = torch.empty(n_pages * stride, dtype=BF16, device="cuda")
    K = pool.as_strided((n_pages, kv, page, d), (stride, page * d, d, 1))
    V = pool[kv * page * d:].as_strided((n_pages, kv, page, d), (stride, page * d, d, 1))
    c = Case([150], 4, kv, d, page, seed=6)
    ids = [65, 0, 64]
    for j, at in enumerate(ids):
        K[at].copy_(c.K[c.pages[0, j]])
        V[at].copy_(c.V[c.pages[0, j]])
    O = bn.bitnet_paged_attn(up(c.q, BF16), K, V, up(np.array([ids]), torch.int32), up(np.array([150]), torch.int32), scale=c.scale)
    assert torch.equal(O, run(bn, c)[0])
    T = 3                                                    # and the write of new rows there
    qkv = torch.randn(T, (4 + 2 * kv) * d, device="cuda").to(BF16)
    bn.bitnet_rope_append(qkv, up(np.array([5, 70, 150]), torch.int32), None, K, V, up(np.array([ids]), torch.int32),
                          seq=torch.zeros(T, dtype=torch.int32, device="cuda"))
    for t, (at, row) in enumerate([(65, 5), (0, 6), (64, 22)]):
        assert torch.equal(K[at, :, row].reshape(-1), qkv[t, 4 * d:6 * d]) and torch.equal(V[at, :, row].reshape(-1), qkv[t, 6 * d:])


def test_bad_pages_and_lengths_are_reported_and_left_out(bn):
    c = Case([100, 64, 40], 4, 2, 64, 16, seed=7)
    q, K, V, pages, lens = c.args()
    bad = pages.clone()
    bad[0, 2] = 10 ** 6                                      # keys 32 .. 47
    bad[1, 0] = -7                                           # keys 0 .. 15
    bad[2, :] = -1                                           # all keys
    for b, gone in ((0, slice(32, 48)), (1, slice(0, 16)), (2, slice(0, 40))):
        c.k[b], c.v[b] = np.delete(c.k[b], gone, 1), np.delete(c.v[b], gone, 1)
    c.lens = [84, 48, 0]
    ws = bn.Workspace(bn.load().bitnet_paged_attn_workspace_size(3, 4, 2, 64))
    lse = torch.empty((3, 4), device="cuda")
    O = bn.bitnet_paged_attn(q, K, V, bad, lens, scale=c.scale, ws=ws, lse=lse)
    assert bn.bitnet_read_device_status(ws) == bn._abi.BITNET_ERR_INVALID_ARG
    ref, bound, lref, lbound = c.ref()
    check(O, ref, bound, BF16)
    assert bool(torch.isneginf(lse[2]).all()) and np.all(np.abs(host(lse)[:2] - lref[:2]) <= lbound[:2])
    c = Case([112, 50], 4, 2, 64, 16, seed=8)                # lists of 7 pages: 112 keys at most
    q, K, V, pages, lens = c.args()
    for trouble in (200, 2 ** 31 - 1):
        O = bn.bitnet_paged_attn(q, K, V, pages, up(np.array([trouble, 50]), torch.int32), scale=c.scale, ws=ws)
        assert bn.bitnet_read_device_status(ws) == bn._abi.BITNET_ERR_INVALID_ARG
        check(O, *c.ref()[:2], BF16)
    O = bn.bitnet_paged_attn(q, K, V, pages, up(np.array([-4, 50]), torch.int32), scale=c.scale, ws=ws)
    assert bn.bitnet_read_device_status(ws) == bn._abi.BITNET_ERR_INVALID_ARG
    assert not O[0].any() and bn.bitnet_read_device_status(ws) == 0


def test_captured_with_lengths_that_grow(bn):
    """Two graphs on one workspace, replayed in turn while the lengths on the device change."""
    c = Case([900, 1300, 700], 20, 5, 128, 16, seed=9)
    q, K, V, pages, lens = c.args()
    ws = bn.Workspace(bn.load().bitnet_paged_attn_workspace_size(3, 20, 5, 128))
    out = [torch.empty_like(q) for _ in range(2)]
    graphs = []
    bn.bitnet_paged_attn(q, K, V, pages, lens, O=out[0], ws=ws)
    torch.cuda.synchronize()
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            bn.bitnet_paged_attn(q, K, V, pages, lens, O=out[i], ws=ws)
    for now in ([1, 0, 64], [65, 1300, 3], [900, 1300, 700]):
        lens.copy_(up(np.array(now), torch.int32))
        graphs[0].replay()
        graphs[1].replay()
        ref = bn.bitnet_paged_attn(q, K, V, pages, lens)
        assert torch.equal(out[0], ref) and torch.equal(out[1], ref)


def test_another_stream_and_strided_rows(bn):
    c = Case([500, 33], 8, 2, 128, 16, seed=10)
    q, K, V, pages, lens = c.args()
    ref = bn.bitnet_paged_attn(q, K, V, pages, lens, scale=c.scale)
    wide = torch.zeros((2, 3 * q.shape[1] + 2), dtype=BF16, device="cuda")
    mid = wide[:, 2:2 + q.shape[1]]                          # rows off 16 bytes
    mid.copy_(q)
    out = torch.full_like(wide, 7.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    O = bn.bitnet_paged_attn(mid, K, V, pages, lens, scale=c.scale, O=out[:, 1:1 + q.shape[1]], stream=s)
    got = bn.bitnet_paged_attn(q, K, V, pages, lens, scale=c.scale, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, ref) and torch.equal(O, ref)
    assert bool((out[:, 0] == 7.0).all()) and bool((out[:, 1 + q.shape[1]:] == 7.0).all())


def test_refusals(bn):
    c = Case([20, 3], 4, 2, 64, 16)
    q, K, V, pages, lens = c.args()
    with pytest.raises(AssertionError):
        bn.bitnet_paged_attn(q.float(), K, V, pages, lens)
    with pytest.raises(AssertionError):
        bn.bitnet_paged_attn(q, K, V, pages, lens.long())
    with pytest.raises(AssertionError):
        bn.bitnet_paged_attn(q, K, V, pages[:1], lens)
    with pytest.raises(bn.BitnetError):
        bn.bitnet_paged_attn(q[:, :192], K, V, pages, lens)  # three heads over two key-value heads
    with pytest.raises(bn.BitnetError):
        bn.bitnet_paged_attn(q, K, V, pages, lens, O=q)
    with pytest.raises(bn.BitnetError):
        bn.bitnet_paged_attn(q, K, V, pages, lens, scale=float("inf"))
    with pytest.raises(bn.BitnetError):
        bn.bitnet_paged_attn(q, K, V, pages, lens, ws=bn.Workspace(256))
    e = bn.bitnet_paged_attn(q[:0], K, V, pages[:0], lens[:0])
    assert e.shape == (0, 256)


def test_long_sums_are_rounded_not_cut(bn):
    """Equal weights, and in feature f one value of 1 at key 2048 f among values of 2^-28: 32 of those are one step of
    fp32 at 1.  A chain of 16 key products that cuts off instead of rounding loses every 16 of them.

    Bound of O n (n = 2^18 keys, so weights are 2^-18 and n O is 1 + 2^-10): the 32 keys around the 1 lose less than
    2^-23, every other step of 32 keys adds a multiple of 2^-23 exactly; the joins of four warps and of at most 74
    ranges per head (a quarter of them in one warp) are 4 + 19 + 4 rounded additions; a reciprocal, a product and a
    rounding to fp32: 32 u in all, and 2^-10 of them."""
    n, d, page, kv, B = 1 << 18, 128, 64, 2, 4
    K = torch.zeros((n // page, kv, page, d), dtype=BF16, device="cuda")
    V = torch.full((n // page, page, d), 2.0 ** -28, device="cuda")
    V.view(n, d)[2048 * torch.arange(d, device="cuda"), torch.arange(d, device="cuda")] = 1.0
    V = V.to(BF16)[:, None].expand(-1, kv, -1, -1).contiguous()
    pages = torch.arange(n // page, dtype=torch.int32, device="cuda").repeat(B, 1)
    q = torch.ones((B, 4 * kv * d), dtype=BF16, device="cuda")
    O = bn.bitnet_paged_attn(q, K, V, pages, torch.full((B,), n, dtype=torch.int32, device="cuda"), o_dtype=F32)
    err = np.abs(host(O) * n - (1 + (n - 1) * 2.0 ** -28))
    assert err.max() <= 32 * U * (1 + 2.0 ** -9), err.max() / U


def test_weights_keep_24_bits(bn):
    """Two keys of one feature, q = 1 and scale 1: x = k, the first key's value 0 and its score the larger, the second's
    value 1, so O = p / (1 + p) with p = 2^(x log2 e - m).  Roundings of p: log2 e (u |x|), the maximum (u, |m| <= 1.45,
    which cancels in p only where it is the same for both keys: it is), the exponent (u |x - m| <= 2.9 u, times ln 2) and
    2^-22 of the power: 2^-22 + 4.5 u; three parts of 8 bits hold p without a further one.  Then the sum, its reciprocal
    and the product: 4 u."""
    B, kv = 64, 32
    r = np.random.default_rng(0)
    x = np.stack([np.ones((B, kv)), r.uniform(-1, 1, (B, kv))], -1).astype(np.float32)
    x = bf16(x)
    K, V = (bn.kv_cache(B, kv, 8, 1) for _ in range(2))
    K[:, :, :2, 0] = up(x, BF16)
    V[:, :, 1] = 1.0
    pages = torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
    O = bn.bitnet_paged_attn(torch.ones((B, kv), dtype=BF16, device="cuda"), K, V, pages.contiguous(),
                             torch.full((B,), 2, dtype=torch.int32, device="cuda"), scale=1.0, o_dtype=F32)
    p = np.exp(x[..., 1].astype(np.float64) - 1.0)
    ref = p / (1 + p)
    assert np.all(np.abs(host(O) - ref) <= ref * (2.0 ** -22 + 8.5 * U))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,kv,d", [(4, 2, 128), (32, 2, 64), (3, 3, 100), (8, 1, 256)])
def test_infinities_and_nan_in_keys_and_values(bn, heads, kv, d, dtype):
    """A value of Inf gives Inf whatever its weight's bits are (1 and 1/2 among them), both signs or NaN give NaN, in that
    feature only; a key whose score is minus infinity counts nothing, one of plus infinity or NaN makes its head NaN."""
    lens = [40, 300, 5, 7, 64, 200]
    c = Case(lens, heads, kv, d, 16, seed=11)
    c.q[:] = np.where(np.arange(heads * d) % d == 0, 1.0, 0.0)     # scores come from feature 0
    for b in range(len(lens)):
        c.k[b][:, :, 0] = -np.arange(lens[b])[None] % 4              # weights 1, e^(-scale), ... : some of them bare powers
    c.k[4][:, 3, 0] = -np.inf                                        # left out
    c.k[5][:, 9, 0] = np.inf
    c.v[0][:, 4, 1], c.v[0][:, 8, 2], c.v[0][:, 1, 3] = np.inf, -np.inf, np.inf
    c.v[0][:, 2, 4], c.v[0][:, 6, 4] = np.inf, -np.inf
    c.v[1][:, 299, d - 1], c.v[1][:, 0, 5], c.v[1][:, 150, 6] = np.inf, np.nan, -np.inf
    for b, n in enumerate(lens):                                     # into the pages
        for j in range(-(-n // 16)):
            rows = slice(16 * j, min(n, 16 * j + 16))
            c.K[c.pages[b, j], :, :rows.stop - rows.start].copy_(up(c.k[b][:, rows], BF16))
            c.V[c.pages[b, j], :, :rows.stop - rows.start].copy_(up(c.v[b][:, rows], BF16))
    O, lse = run(bn, c, dtype)
    got, got_l = host(O).reshape(len(lens), heads, d), host(lse)
    assert np.isnan(got[5]).all() and np.isnan(got_l[5]).all()
    x = [np.einsum("hgd,hnd->hgn", np.ones((kv, heads // kv, 1)), c.k[b][:, :, :1].astype(np.float64)) * c.scale for b in range(5)]
    p = [np.exp(s - s.max(-1, keepdims=True)) for s in x]
    with np.errstate(invalid="ignore"):
        ref = np.stack([np.einsum("hgn,hnd->hgd", w / w.sum(-1, keepdims=True), c.v[b].astype(np.float64)).reshape(heads, d)
                        for b, w in enumerate(p)])
    got = got[:5]
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(np.isposinf(got), np.isposinf(ref)) and np.array_equal(np.isneginf(got), np.isneginf(ref))
    assert np.isposinf(ref[0, :, 1]).all() and np.isnan(ref[0, :, 4]).all() and np.isfinite(ref[4]).all()
    size = np.stack([np.einsum("hgn,hnd->hgd", w / w.sum(-1, keepdims=True), np.abs(np.nan_to_num(c.v[b].astype(np.float64), posinf=0, neginf=0)))
                     .reshape(heads, d) for b, w in enumerate(p)])
    # scores are exact up to u |x|, |x| < 4: the weights within 2^-17 + 2^-21, twice that with their sum, then the rounding of O
    ok = np.isfinite(ref)
    bound = 2 * (2.0 ** -17 + 2.0 ** -20) * size
    bound += (2.0 ** -8 if dtype == BF16 else U) * (np.abs(np.where(ok, ref, 0)) + bound)
    assert np.all(np.abs(got[ok] - ref[ok]) <= bound[ok])


@pytest.mark.parametrize("n,heads,d", [(60000, 5, 128), (45000, 16, 100), (45000, 3, 256)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_head_over_more_ranges_than_a_join_takes_at_once(bn, n, heads, d, dtype):
    """One sequence and one key-value head cut over more than 128 ranges: the join's warps take their partials in several
    rounds, and the largest scores come near the end, so that what they have is rescaled."""
    c = Case([n], heads, 1, d, 64, seed=n + d)
    late = int(0.97 * n)
    for j in range(late, late + 3):
        c.k[0][0, j] = c.q[0, :d]
    for j in range(-(-n // 64)):
        rows = slice(64 * j, min(n, 64 * j + 64))
        c.K[c.pages[0, j], :, :rows.stop - rows.start].copy_(up(c.k[0][:, rows], BF16))
    check_case(bn, c, dtype)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 3.0])
@pytest.mark.parametrize("heads,kv,d", [(20, 5, 128), (7, 7, 100)])
def test_scales(bn, scale, heads, kv, d):
    """No scale at all (every key counts the same, what lies behind a length still nothing), a negative and a large one."""
    c = Case(LENS, heads, kv, d, 16, seed=13)
    c.scale = scale
    check_case(bn, c, F32)
