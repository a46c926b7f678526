"""GPU rotary positions and the paged key-value cache write, bit for bit against
the definition in NumPy: every step one rounded fp32 operation, then one
rounding to the output's type; cache rows, padding rows and rows that no call
writes compared as bits.

"BitNet b1.58: Ternary Weights for 1.58-bit LLMs", "What this paper explains"
(LLaMA-alike blocks).
"""
import numpy as np
import pytest

from sparse_linear_layers_bitnet_b200 import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bn(cuda_device):
    import sparse_linear_layers_bitnet_b200 as m
    m.load()
    return m


def bf16(x):
    return synth.bf16_bits_to_f32(synth.to_bf16_bits(x))


def table_ref(n_pos, rot, base=10000.0):
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    a = np.arange(n_pos, dtype=np.float64)[:, None] * f
    return np.stack((np.cos(a), np.sin(a)), -1).astype(np.float32)


def turn(x, cs, interleaved, inverse=False):
    """x [T, heads, d] fp32, cs [T, rot / 2, 2] fp32; NumPy's fp32 operations round once each."""
    n = cs.shape[1]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1] * np.float32(-1 if inverse else 1)
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    u, v = a * c - b * s, b * c + a * s
    y = x.copy()
    if interleaved:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = u, v
    else:
        y[..., :n], y[..., n:2 * n] = u, v
    return y


def up(x, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dtype)


def host(t):
    return t.float().cpu().numpy()


# head sizes: every vector width (8, 4, 2, 1), partial rotation, an odd count of copied vectors
@pytest.mark.parametrize("heads,d,rot", [(1, 2, 2), (5, 128, 128), (64, 100, 100), (3, 80, 32), (7, 96, 50), (2, 256, 256),
                                         (4, 65, 10), (3, 24, 16), (9, 64, 0), (33, 72, 64)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_bits(bn, heads, d, rot, dtype, interleaved):
    r = np.random.default_rng(heads * d + rot)
    T, n_pos = 37, 500
    x = r.normal(size=(T, heads * d)).astype(np.float32)
    if dtype == BF16:
        x = bf16(x)
    pos = r.integers(0, n_pos, T).astype(np.int32)
    tab = table_ref(n_pos, rot) if rot else np.zeros((n_pos, 0, 2), np.float32)
    for inverse in (False, True):
        ref = turn(x.reshape(T, heads, d), tab[pos], interleaved, inverse).reshape(T, -1)
        if dtype == BF16:
            ref = bf16(ref)
        ws = bn.Workspace(256)
        got = bn.bitnet_rope(up(x, dtype), up(pos, torch.int32), up(tab), heads, interleaved=interleaved, inverse=inverse, ws=ws)
        assert np.array_equal(host(got).view(np.uint32), ref.view(np.uint32))
        assert bn.bitnet_read_device_status(ws) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [128, 100])
def test_rope_in_place_on_the_query_and_key_heads(bn, dtype, d):
    """Strided rows (the value heads behind stay), padding rows stay, the inverse is the gradient."""
    T, heads, kv = 19, 6, 2
    r = np.random.default_rng(d)
    x = r.normal(size=(T, (heads + 2 * kv) * d)).astype(np.float32)
    x = bf16(x) if dtype == BF16 else x
    pos = r.integers(0, 64, T).astype(np.int32)
    pos[[3, 7]] = -1
    tab = table_ref(64, d)
    ref = turn(x.reshape(T, -1, d)[:, :heads + kv], tab[np.maximum(pos, 0)], False)
    want = x.copy().reshape(T, -1, d)
    want[pos >= 0, :heads + kv] = (bf16(ref) if dtype == BF16 else ref)[pos >= 0]
    xd = up(x, dtype)
    out = bn.bitnet_rope(xd, up(pos, torch.int32), up(tab), heads + kv, d, Y=xd)
    assert out is xd
    assert np.array_equal(host(xd).view(np.uint32), want.reshape(T, -1).view(np.uint32))


def test_rope_gradient_against_differences(bn):
    """The map is linear: <g, R(v)> = <R^T(g), v> for the inverse as R^T.  Both sides are fp32 results
    summed in 64 bits: each element carries at most 3 roundings of terms no larger than |a| + |b|."""
    r = np.random.default_rng(0)
    T, heads, d = 11, 3, 64
    v, g = (r.normal(size=(T, heads * d)).astype(np.float32) for _ in range(2))
    pos, tab = up(r.integers(0, 4096, T).astype(np.int32), torch.int32), up(table_ref(4096, 48))
    for interleaved in (False, True):
        fwd = host(bn.bitnet_rope(up(v), pos, tab, heads, interleaved=interleaved)).astype(np.float64)
        bwd = host(bn.bitnet_rope(up(g), pos, tab, heads, interleaved=interleaved, inverse=True)).astype(np.float64)
        a, b = (g.astype(np.float64) * fwd).sum(), (bwd * v.astype(np.float64)).sum()
        assert abs(a - b) <= 3 * 2.0 ** -24 * 2 * np.abs(g).max() * np.abs(v).max() * 2 * v.size


def test_a_position_behind_the_table_is_reported_and_its_row_left(bn):
    x = torch.randn(4, 128, device="cuda")
    y = torch.full((4, 128), 7.0, device="cuda")
    tab = up(table_ref(16, 64))
    ws = bn.Workspace(256)
    bn.bitnet_rope(x, up(np.array([0, 16, -5, 2 ** 31 - 1], np.int32), torch.int32), tab, 2, Y=y, ws=ws)
    assert bn.bitnet_read_device_status(ws) == bn._abi.BITNET_ERR_INVALID_ARG
    assert bn.bitnet_read_device_status(ws) == 0           # cleared by the read
    assert bool((y[1:] == 7.0).all()) and torch.equal(y[0], x[0])


@pytest.mark.parametrize("scaling", [None, {"type": "linear", "factor": 4}, {"type": "base", "factor": 8},
                                     {"type": "parts", "factor": 16, "original": 512}])
def test_table_far_positions(bn, scaling):
    """Angles in 64 bits: 2^20 positions away fp32 angles would be off by whole hundredths.  Each entry is
    one rounding of amplitude * cos: 2^-24 of it, plus 2^-52 * 2^20 of the angle."""
    n, rot = 1 << 20, 8
    t = bn.rope_table(n, rot, 10000.0, scaling).cpu().numpy().astype(np.float64)
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    amp = 1.0
    if scaling and scaling["type"] == "linear":
        f = f / 4
    elif scaling and scaling["type"] == "base":
        f = (10000.0 * 8 ** (rot / (rot - 2))) ** (-np.arange(0, rot, 2) / rot)
        assert abs(f[0] - 1) < 1e-15 and abs(f[-1] * 8 / 10000.0 ** (-(rot - 2) / rot) - 1) < 1e-12
    elif scaling:
        keep = np.clip((512 * f / (2 * np.pi) - 1) / 31, 0, 1)
        assert keep[0] == 1 and keep[-1] == 0
        f, amp = f * keep + f * (1 - keep) / 16, 0.1 * np.log(16) + 1
    p = np.array([0, 1, 77777, n - 1])
    a = p[:, None] * f
    bound = 2.0 ** -23 * amp + 2.0 ** -30
    assert np.all(np.abs(t[p, :, 0] - amp * np.cos(a)) <= bound)
    assert np.all(np.abs(t[p, :, 1] - amp * np.sin(a)) <= bound)


def _append_case(bn, heads, kv, d, rot, dtype, interleaved, page, lens, new, layout, seed):
    """A cache of sequences that hold lens keys and get new more each, in pages in shuffled order."""
    r = np.random.default_rng(seed)
    B = len(lens)
    counts = [-(-(n + new) // page) for n in lens]
    n_pages = sum(counts) + 2
    order = r.permutation(n_pages)
    pages = np.full((B, max(counts)), -1, np.int32)
    at = 0
    for b, c in enumerate(counts):
        pages[b, :c] = order[at:at + c]
        at += c
    T = B * new
    x = r.normal(size=(T, (heads + 2 * kv) * d)).astype(np.float32)
    x = bf16(x) if dtype == BF16 else x
    pos = np.concatenate([np.arange(n, n + new) for n in lens]).astype(np.int32)
    seq = np.repeat(np.arange(B), new).astype(np.int32)
    tab = table_ref(max(lens) + new, rot) if rot else None
    if layout == "heads first":
        K, V = bn.kv_cache(n_pages, kv, page, d), bn.kv_cache(n_pages, kv, page, d)
    else:   # pages of rows that hold all heads
        K, V = (bn.kv_cache(n_pages, page, kv, d).permute(0, 2, 1, 3) for _ in range(2))
    K.copy_(torch.randn(K.shape, device="cuda"))
    V.copy_(torch.randn(V.shape, device="cuda"))
    return x, pos, seq, pages, tab, K, V


def _append_ref(x, pos, seq, pages, tab, K, V, heads, kv, d, interleaved):
    T, page = len(pos), K.shape[2]
    h = x.reshape(T, heads + 2 * kv, d)
    live = (pos >= 0) & (seq >= 0)
    qk = h[:, :heads + kv] if tab is None else turn(h[:, :heads + kv], tab[np.maximum(pos, 0)], interleaved)
    Kr, Vr = host(K).copy(), host(V).copy()
    for t in np.flatnonzero(live):
        at, row = pages[seq[t], pos[t] // page], pos[t] % page
        Kr[at, :, row] = bf16(qk[t, heads:])
        Vr[at, :, row] = bf16(h[t, heads + kv:])
    return bf16(qk[:, :heads]).reshape(T, -1), Kr, Vr


@pytest.mark.parametrize("heads,kv,d,rot", [(20, 5, 128, 128), (32, 32, 100, 100), (4, 1, 80, 24), (2, 2, 64, 0), (3, 3, 65, 10),
                                            (8, 1, 256, 256)])
@pytest.mark.parametrize("dtype,interleaved", [(BF16, False), (F32, True)])
@pytest.mark.parametrize("layout,page,new", [("heads first", 16, 1), ("rows first", 8, 13)])
def test_append_bits(bn, heads, kv, d, rot, dtype, interleaved, layout, page, new):
    x, pos, seq, pages, tab, K, V = _append_case(bn, heads, kv, d, rot, dtype, interleaved, page, [0, 7, 8, 41], new, layout, d + new)
    Qr, Kr, Vr = _append_ref(x, pos, seq, pages, tab, K, V, heads, kv, d, interleaved)
    ws = bn.Workspace(256)
    Q = bn.bitnet_rope_append(up(x, dtype), up(pos, torch.int32), None if tab is None else up(tab), K, V, up(pages, torch.int32),
                              seq=None if new == 1 else up(seq, torch.int32), interleaved=interleaved, ws=ws)
    assert bn.bitnet_read_device_status(ws) == 0
    assert np.array_equal(host(Q), Qr) and np.array_equal(host(K), Kr) and np.array_equal(host(V), Vr)


def test_append_padding_rows_and_bad_indexes(bn):
    heads, kv, d, page = 4, 2, 64, 16
    x, pos, seq, pages, tab, K, V = _append_case(bn, heads, kv, d, d, BF16, False, page, [5, 20], 3, "heads first", 1)
    pages = np.concatenate([pages, np.array([[10 ** 6, -1]], np.int32)])          # a third sequence with bad pages
    pos = np.concatenate([pos, [3, 17, 2, 0, 10 ** 6, 1]]).astype(np.int32)       # the row's own trouble, in order:
    seq = np.concatenate([seq, [2, 2, 3, -1, 0, 1]]).astype(np.int32)             # page, page, sequence, (padding), position, (fine)
    pos[-1], tail = 30, len(pos)
    x = bf16(np.random.default_rng(2).normal(size=(tail, x.shape[1])).astype(np.float32))
    tab = table_ref(64, d)
    good = np.ones(tail, bool)
    good[6:11] = False
    safe = np.where(good, pos, -1)
    Qr, Kr, Vr = _append_ref(x, safe, seq, pages, tab, K, V, heads, kv, d, False)
    Q = torch.full((tail, heads * d), 7.0, dtype=BF16, device="cuda")
    ws = bn.Workspace(256)
    bn.bitnet_rope_append(up(x, BF16), up(pos, torch.int32), up(tab), K, V, up(pages, torch.int32), seq=up(seq, torch.int32), Q=Q, ws=ws)
    assert bn.bitnet_read_device_status(ws) == bn._abi.BITNET_ERR_INVALID_ARG
    assert np.array_equal(host(K), Kr) and np.array_equal(host(V), Vr)
    assert np.array_equal(host(Q)[good], Qr[good]) and bool((Q[torch.from_numpy(~good).cuda()] == 7.0).all())
    ws = bn.Workspace(256)
    only_pad = np.array([-1, -3], np.int32)
    bn.bitnet_rope_append(up(x[:2], BF16), up(only_pad, torch.int32), up(tab), K, V, up(pages, torch.int32), seq=up(only_pad, torch.int32), ws=ws)
    assert bn.bitnet_read_device_status(ws) == 0 and np.array_equal(host(K), Kr)


def test_append_captured_and_replayed(bn):
    heads, kv, d, page = 20, 5, 128, 16
    x, pos, seq, pages, tab, K, V = _append_case(bn, heads, kv, d, d, BF16, False, page, [9, 30], 1, "heads first", 5)
    xd, pd, td, pg = up(x, BF16), up(pos, torch.int32), up(tab), up(pages, torch.int32)
    Q, ws = torch.empty((2, heads * d), dtype=BF16, device="cuda"), bn.Workspace(256)
    bn.bitnet_rope_append(xd, pd, td, K, V, pg, Q=Q, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bn.bitnet_rope_append(xd, pd, td, K, V, pg, Q=Q, ws=ws)
    x2 = bf16(np.random.default_rng(9).normal(size=x.shape).astype(np.float32))
    xd.copy_(up(x2, BF16))
    pd.sub_(3)                                             # other rows of the same pages
    Qr, Kr, Vr = _append_ref(x2, pos - 3, seq, pages, tab, K, V, heads, kv, d, False)
    g.replay()
    assert np.array_equal(host(Q), Qr) and np.array_equal(host(K), Kr) and np.array_equal(host(V), Vr)


def test_refusals(bn):
    x, tab = torch.zeros((4, 256), device="cuda"), up(table_ref(8, 64))
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(AssertionError):
        bn.bitnet_rope(x, pos.long(), tab, 4)
    with pytest.raises(AssertionError):
        bn.bitnet_rope(x.half(), pos, tab, 4)
    with pytest.raises(bn.BitnetError):                    # the table turns more features than a head has
        bn.bitnet_rope(x, pos, tab, 8)
    with pytest.raises(bn.BitnetError):                    # Y over a part of X
        bn.bitnet_rope(x[:2], pos[:2], tab, 4, Y=x[1:3])
    K, V = bn.kv_cache(4, 1, 16, 64), bn.kv_cache(4, 1, 16, 64)
    pages = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(bn.BitnetError):                    # four rows, two sequences, no seq
        bn.bitnet_rope_append(x, pos, tab, K, V, pages)
    with pytest.raises(AssertionError):
        bn.bitnet_rope_append(x, pos, tab, K, V[:3], pages)
    with pytest.raises(bn.BitnetError):                    # rows that do not lie on 16 bytes
        W = torch.zeros((2, 4, 1, 16, 68), dtype=BF16, device="cuda")[..., :64]
        bn.bitnet_rope_append(x[:2], pos[:2], tab, W[0], W[1], pages)


@pytest.mark.parametrize("heads,kv,d,rot", [(32, 32, 100, 100), (20, 5, 128, 128), (6, 2, 40, 24), (2, 1, 72, 0), (4, 4, 36, 20),
                                            (40, 12, 128, 128), (60, 20, 128, 64)])
@pytest.mark.parametrize("dtype,interleaved,layout", [(BF16, False, "heads first"), (F32, True, "rows first"), (BF16, True, "rows first")])
def test_append_of_many_rows(bn, heads, kv, d, rot, dtype, interleaved, layout):
    """Enough rows for several per persistent CTA, with padding rows and rows of bad indexes among them."""
    new = 701
    x, pos, seq, pages, tab, K, V = _append_case(bn, heads, kv, d, rot, dtype, interleaved, 32, [3, 500], new, layout, d)
    r = np.random.default_rng(d)
    odd = r.choice(len(pos), 40, replace=False)
    pos[odd[:10]] = -1
    seq[odd[10:20]] = -2
    seq[odd[20:30]] = 2 + r.integers(0, 1000, 10)
    pos[odd[30:]] = 10 ** 6 + r.integers(0, 1000, 10)
    good = np.ones(len(pos), bool)
    good[odd] = False
    Qr, Kr, Vr = _append_ref(x, np.where(good, pos, -1), np.where(good, seq, 0), pages, tab, K, V, heads, kv, d, interleaved)
    Q = torch.full((len(pos), heads * d), 7.0, dtype=BF16, device="cuda")
    ws = bn.Workspace(256)
    bn.bitnet_rope_append(up(x, dtype), up(pos, torch.int32), None if tab is None else up(tab), K, V, up(pages, torch.int32),
                          seq=up(seq, torch.int32), interleaved=interleaved, Q=Q, ws=ws)
    assert bn.bitnet_read_device_status(ws) == bn._abi.BITNET_ERR_INVALID_ARG
    assert np.array_equal(host(Q)[good], Qr[good]) and bool((Q[torch.from_numpy(~good).cuda()] == 7.0).all())
    assert np.array_equal(host(K), Kr) and np.array_equal(host(V), Vr)


@pytest.mark.parametrize("d,rot,heads", [(100, 100, 8), (100, 36, 8), (128, 128, 8), (50, 20, 8), (128, 128, 64), (128, 64, 70)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rope_of_many_rows_in_place(bn, d, rot, heads, dtype):
    T = 1500
    r = np.random.default_rng(d + rot)
    x = r.normal(size=(T, heads * d)).astype(np.float32)
    x = bf16(x) if dtype == BF16 else x
    pos = r.integers(-3, 2000, T).astype(np.int32)
    tab = table_ref(2000, rot)
    ref = turn(x.reshape(T, heads, d), tab[np.maximum(pos, 0)], False).reshape(T, -1)
    ref = np.where(pos[:, None] >= 0, bf16(ref) if dtype == BF16 else ref, x)
    xd = up(x, dtype)
    bn.bitnet_rope(xd, up(pos, torch.int32), up(tab), heads, Y=xd)
    assert np.array_equal(host(xd).view(np.uint32), ref.view(np.uint32))


def test_without_a_workspace_a_bad_index_raises(bn):
    """Nobody could read the status word of a workspace that the call made for itself."""
    x, tab = torch.randn(4, 128, device="cuda"), up(table_ref(16, 64))
    fine = up(np.array([0, 15, -5, 3], np.int32), torch.int32)
    bn.bitnet_rope(x, fine, tab, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    bad = up(np.array([0, 16, -5, 3], np.int32), torch.int32)
    torch.cuda.synchronize()
    for stream in (None, s):
        with pytest.raises(bn.BitnetError, match="out of range"):
            bn.bitnet_rope(x, bad, tab, 2, stream=stream)
    K, V = bn.kv_cache(4, 1, 16, 64), bn.kv_cache(4, 1, 16, 64)
    qkv = torch.randn(2, 4 * 64, device="cuda").to(BF16)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    pages = up(np.array([[0], [4]], np.int32), torch.int32)          # page 4 of four
    with pytest.raises(bn.BitnetError, match="out of range"):
        bn.bitnet_rope_append(qkv, pos, tab, K, V, pages)
    with pytest.raises(bn.BitnetError, match="out of range"):
        bn.bitnet_paged_attn(qkv[:, :64].contiguous(), K, V, pages, pos + 1)
    pages.zero_()
    q = bn.bitnet_rope_append(qkv[:1], pos[:1], tab, K, V, pages[:1])
    bn.bitnet_paged_attn(q, K, V, pages[:1], pos[:1] + 1)
    assert bn.bitnet_rope(x[:0], fine[:0], tab, 2).shape == (0, 128)


def test_a_captured_call_needs_a_workspace(bn):
    x, tab = torch.randn(4, 128, device="cuda"), up(table_ref(16, 64))
    pos, y, ws = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.empty(4, 128, device="cuda"), bn.Workspace(256)
    bn.bitnet_rope(x, pos, tab, 2, Y=y, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bn.bitnet_rope(x, pos, tab, 2, Y=y, ws=ws)
        with pytest.raises(bn.BitnetError, match="workspace"):
            bn.bitnet_rope(x, pos, tab, 2, Y=y)
    pos.fill_(16)
    g.replay()
    assert bn.bitnet_read_device_status(ws) == bn._abi.BITNET_ERR_INVALID_ARG
    pos.fill_(0)
    g.replay()
    assert bn.bitnet_read_device_status(ws) == 0 and torch.equal(y, x)


def test_rows_of_more_than_the_heads_need_head_dim(bn):
    """Five heads of 64 and two more behind them: 448 / 5 is no head's size."""
    x, tab = torch.randn(3, 448, device="cuda"), up(table_ref(16, 64))
    pos = torch.ones(3, dtype=torch.int32, device="cuda")
    with pytest.raises(AssertionError, match="head_dim"):
        bn.bitnet_rope(x, pos, tab, 5)
    y = bn.bitnet_rope(x, pos, tab, 5, 64)
    assert y.shape == (3, 320) and torch.equal(y, bn.bitnet_rope(x[:, :320].contiguous(), pos, tab, 5))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T", [21, 1500])
def test_odd_row_strides_and_a_table_off_16_bytes(bn, dtype, interleaved, T):
    """Rows an odd number of elements apart that start off the vectors' alignment, a table on 8 bytes only."""
    heads, d, rot, n_pos = 5, 64, 48, 300
    r = np.random.default_rng(T)
    x = r.normal(size=(T, heads * d)).astype(np.float32)
    x = bf16(x) if dtype == BF16 else x
    pos = r.integers(0, n_pos, T).astype(np.int32)
    tab = table_ref(n_pos, rot)
    flat = torch.zeros(2 + tab.size, device="cuda")
    flat[2:] = up(tab).reshape(-1)
    td = flat[2:].view(n_pos, rot // 2, 2)
    assert td.data_ptr() % 16 == 8
    ref = turn(x.reshape(T, heads, d), tab[pos], interleaved).reshape(T, -1)
    ref = bf16(ref) if dtype == BF16 else ref
    aligned = up(x, dtype)
    assert np.array_equal(host(bn.bitnet_rope(aligned, up(pos, torch.int32), td, heads, interleaved=interleaved)).view(np.uint32), ref.view(np.uint32))
    wide, out = (torch.full((T, heads * d + 7), 9.0, dtype=dtype, device="cuda") for _ in range(2))
    xv, yv = wide[:, 3:3 + heads * d], out[:, 1:1 + heads * d]
    xv.copy_(aligned)
    bn.bitnet_rope(xv, up(pos, torch.int32), td, heads, d, interleaved=interleaved, Y=yv)
    assert np.array_equal(host(yv).view(np.uint32), ref.view(np.uint32))
    assert bool((out[:, 0] == 9.0).all()) and bool((out[:, 1 + heads * d:] == 9.0).all())
    bn.bitnet_rope(xv, up(pos, torch.int32), td, heads, d, interleaved=interleaved, Y=xv)      # in place
    assert np.array_equal(host(xv).view(np.uint32), ref.view(np.uint32))
    K, V = bn.kv_cache(-(-T // 16), 1, 16, d), bn.kv_cache(-(-T // 16), 1, 16, d)
    xv.copy_(aligned)                                                 # three query heads, a key and a value head
    Q = bn.bitnet_rope_append(xv, up(np.arange(T) % n_pos if T < n_pos else np.arange(T), torch.int32), td if T < n_pos else None,
                              K, V, torch.arange(-(-T // 16), dtype=torch.int32, device="cuda")[None].contiguous(),
                              seq=torch.zeros(T, dtype=torch.int32, device="cuda"), interleaved=interleaved)
    h = x.reshape(T, heads, d)
    qk = turn(h[:, :4], tab[np.arange(T)], interleaved) if T < n_pos else h[:, :4]
    assert np.array_equal(host(Q), bf16(qk[:, :3]).reshape(T, -1))
    assert np.array_equal(host(K)[:, 0].reshape(-1, d)[:T], bf16(qk[:, 3])) and np.array_equal(host(V)[:, 0].reshape(-1, d)[:T], bf16(h[:, 4]))


def test_a_workspace_that_held_anything_is_cleared_by_a_read(bn):
    x, tab = torch.randn(4, 128, device="cuda"), up(table_ref(16, 64))
    pos, ws = torch.zeros(4, dtype=torch.int32, device="cuda"), bn.Workspace(256)
    ws.buf.fill_(255)
    assert bn.bitnet_read_device_status(ws) != 0
    bn.bitnet_rope(x, pos, tab, 2, ws=ws)
    assert bn.bitnet_read_device_status(ws) == 0
