"""The operators between the BitLinear products of a decoder block, as cases to
be measured: what a block runs besides its ternary products, in training and in
serving.

  add_norm   residual addition, RMSNorm and per-token int8 codes in one pass
  norm_grad  the gradient of that step for its input, the residual stream and
             the norm weight
  rope       rotary positions on the query and key heads of a QKV row (forward,
             and its backward, the inverse rotation)
  append     rotary positions and the write of keys and values into a paged
             key-value cache
  attn       attention of one new token per sequence over that cache

`run` takes each in elementary torch operations, or, where `own` is true,
through the calls of this package.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}
EPS_NORM, EPS_ACT = 1e-6, 1e-5


# ------------------------------------------------------------------ cases

def _add_norm(T, K, **kw):
    return dict(op="add_norm", T=T, K=K, **kw)


def _norm_grad(T, K, dy, residual, **kw):
    return dict(op="norm_grad", T=T, K=K, dy=dy, residual=residual, **kw)


def _rope(T, heads, d, rot, interleaved, inverse, dtype, n_pos, **kw):
    return dict(op="rope", T=T, heads=heads, d=d, rot=rot, interleaved=interleaved, inverse=inverse, dtype=dtype,
                n_pos=n_pos, **kw)


def _append(seqs, new, heads, kv_heads, d, rot, interleaved, dtype, page, context, **kw):
    return dict(op="append", seqs=seqs, new=new, heads=heads, kv_heads=kv_heads, d=d, rot=rot, interleaved=interleaved,
                dtype=dtype, page=page, context=context, **kw)


def _attn(seqs, shortest, longest, heads, kv_heads, d, page, **kw):
    return dict(op="attn", seqs=seqs, shortest=shortest, longest=longest, heads=heads, kv_heads=kv_heads, d=d, page=page,
                **kw)


def listed():
    return [
        # one decoded token of the 2B model (hidden 2560): latency only
        _add_norm(1, 2560, name="add_norm 1x2560"),
        # a training step's block of the 3B model (hidden 3200)
        _add_norm(2048, 3200, name="add_norm 2048x3200"),
        # a long prefill at the 7B width, a token count that divides nothing
        _add_norm(16381, 4096, name="add_norm 16381x4096"),
        # the 3B block's backward: bf16 gradient from the input-gradient product, and the residual stream's
        _norm_grad(2048, 3200, "bf16", True, name="norm_grad 2048x3200"),
        # 7B width, many tokens, fp32 gradient from the product, no residual branch (the model's last norm)
        _norm_grad(8191, 4096, "f32", False, name="norm_grad 8191x4096 f32"),
        # the 3B block's query and key heads (32 + 32 heads of 100), halves layout, whole head
        _rope(2048, 64, 100, 100, False, False, "bf16", 4096, name="rope 2048x64x100"),
        # backward at the 7B width with interleaved pairs on half of the head, fp32 rows, far positions
        _rope(4095, 64, 128, 64, True, True, "f32", 131072, name="rope back 4095x64x128 f32"),
        # one decode step of eight sequences of the 2B model (20 query and 5 key-value heads of 128)
        _append(8, 1, 20, 5, 128, 128, False, "bf16", 16, 4000, name="append 8x1"),
        # chunks of prompts of the 3B model going into the cache
        _append(4, 1021, 32, 32, 100, 100, False, "bf16", 64, 2000, name="append 4x1021"),
        # one sequence of the 2B model at a middle length: too few heads to fill the GPU without a split
        _attn(1, 4001, 4001, 20, 5, 128, 16, name="attn 1x4001"),
        # a ragged serving batch of the 3B model (32 heads of 100, no sharing), one idle slot
        _attn(24, 0, 4096, 32, 32, 100, 64, name="attn 24x..4096 d100"),
        # long contexts of the 2B model, grouped heads
        _attn(8, 65536, 131072, 20, 5, 128, 16, name="attn 8x..131072"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["add_norm", "norm_grad", "rope", "append", "attn", "attn"])
    heads, kv_heads, d = rng.choice([(20, 5, 128), (32, 32, 100), (32, 32, 128), (32, 8, 128), (64, 4, 128), (8, 1, 256),
                                     (16, 16, 64), (12, 4, 80), (24, 8, 96), (7, 7, 64)])
    rot = d if rng.random() < 0.6 else max(2, 2 * int(d * rng.uniform(0.2, 0.5)))
    interleaved = rng.random() < 0.5
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    if op in ("add_norm", "norm_grad"):
        K = 8 * _log_int(rng, 32, 1080)
        T = min(_log_int(rng, 1, 16384), 16381 * 4096 // (2 * K))
        if op == "add_norm":
            return _add_norm(T, K)
        return _norm_grad(T, K, dtype, rng.random() < 0.7)
    if op == "rope":
        T = min(_log_int(rng, 1, 8192), 4095 * 64 * 128 // (2 * heads * d))
        return _rope(T, heads + kv_heads, d, rot, interleaved, rng.random() < 0.5, dtype, _log_int(rng, 2048, 131072))
    if op == "append":
        new = 1 if rng.random() < 0.5 else _log_int(rng, 2, 2000)
        seqs = _log_int(rng, 1, 128) if new == 1 else rng.randint(1, 4)
        return _append(seqs, new, heads, kv_heads, d, rot, interleaved, dtype, page, _log_int(rng, 1, 8000))
    seqs = _log_int(rng, 1, 128)
    most = 6 * 2**28 // (seqs * kv_heads * d * 4)   # keys per sequence that keep the cache below 1.6 GB
    longest = min(_log_int(rng, 1, 131072), max(1, most))
    return _attn(seqs, rng.choice([0, longest // 2, longest]), longest, heads, kv_heads, d, page)


def _lens(case):
    """The sequences' lengths: the case's own, the same for every seed."""
    r = random.Random("%d %d %d" % (case["seqs"], case["shortest"], case["longest"]))
    n = [r.randint(case["shortest"], case["longest"]) for _ in range(case["seqs"])]
    n[0] = case["longest"]
    if case["shortest"] == 0 and len(n) > 1:
        n[-1] = 0   # a slot of the batch that no request holds
    return n


def _starts(case):
    """How many keys each sequence of an append case holds already."""
    r = random.Random("%d %d" % (case["seqs"], case["context"]))
    return [r.randint(case["context"] // 2, case["context"]) for _ in range(case["seqs"])]


# ------------------------------------------------------------------ inputs

def _table(n_pos, rot, base):
    """cos and sin of every position and frequency, [n_pos, rot / 2, 2] fp32: angles in 64 bits."""
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(n_pos, dtype=torch.float64, device=DEV)[:, None] * freq
    return torch.stack((a.cos(), a.sin()), dim=-1).to(F32).contiguous()


def _cache(g, n_pages, kv_heads, page, d):
    """One of keys and values: [pages, heads, page, d], every row on 16 bytes."""
    ld = -(-d // 8) * 8
    c = torch.randn((n_pages, kv_heads, page, ld), generator=g, device=DEV, dtype=BF16)
    return c[..., :d]


def _pages(g, counts, extra):
    """Pages of every sequence in shuffled order, -1 behind its last: [seqs, most] int32, and the pool's size."""
    n = sum(counts) + extra
    order = torch.randperm(n, generator=g, device=DEV).to(torch.int32).tolist()
    most = max(1, max(counts))
    rows, at = [], 0
    for c in counts:
        rows.append(order[at:at + c] + [-1] * (most - c))
        at += c
    return torch.tensor(rows, dtype=torch.int32, device=DEV), n


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def randn(*shape, dtype=F32, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV, dtype=F32) * scale).to(dtype)

    def outliers(x):   # residual streams have a few features far above the others
        hot = torch.rand(x.shape[-1], generator=g, device=DEV) < 0.01
        return torch.where(hot, x * 20, x)

    op, s = case["op"], {"case": case}
    if op == "add_norm":
        T, K = case["T"], case["K"]
        s |= dict(X=randn(T, K, dtype=BF16), R=outliers(randn(T, K)).to(BF16), w=1 + randn(K, scale=0.1))
    elif op == "norm_grad":
        T, K = case["T"], case["K"]
        H = outliers(randn(T, K)).to(BF16)
        rinv = 1 / (H.double().square().mean(-1) + EPS_NORM).sqrt()
        s |= dict(dY=randn(T, K, dtype=DTYPES[case["dy"]], scale=0.01), H=H, rinv=rinv.to(F32), w=1 + randn(K, scale=0.1),
                  dR=randn(T, K, dtype=BF16, scale=0.01) if case["residual"] else None)
    elif op == "rope":
        T = case["T"]
        # packed training sequences: positions restart, the farthest ones are in use
        length = min(T, case["n_pos"])
        pos = (torch.arange(T, device=DEV) % length + (case["n_pos"] - length)).to(torch.int32)
        s |= dict(X=randn(T, case["heads"] * case["d"], dtype=DTYPES[case["dtype"]]), pos=pos,
                  table=_table(case["n_pos"], case["rot"], 10000.0))
    elif op == "append":
        heads, kv, d, page = case["heads"], case["kv_heads"], case["d"], case["page"]
        starts, new = _starts(case), case["new"]
        table, n = _pages(g, [-(-(a + new) // page) for a in starts], 3)
        T = case["seqs"] * new
        pos = torch.tensor(starts, device=DEV)[:, None] + torch.arange(new, device=DEV)
        s |= dict(QKV=randn(T, (heads + 2 * kv) * d, dtype=DTYPES[case["dtype"]]), pos=pos.reshape(-1).to(torch.int32),
                  seq=torch.arange(case["seqs"], device=DEV, dtype=torch.int32).repeat_interleave(new),
                  k=_cache(g, n, kv, page, d), v=_cache(g, n, kv, page, d), pages=table,
                  table=_table(max(starts) + new, case["rot"], 500000.0))
    else:
        heads, kv, d, page = case["heads"], case["kv_heads"], case["d"], case["page"]
        lens = _lens(case)
        table, n = _pages(g, [-(-a // page) for a in lens], 3)
        s |= dict(Q=randn(case["seqs"], heads * d, dtype=BF16, scale=2.0), k=_cache(g, n, kv, page, d),
                  v=_cache(g, n, kv, page, d), pages=table, lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                  scale=d ** -0.5)
    if own:
        import sparse_linear_layers_bitnet_b200 as bn
        # what a serving or training loop holds: the output buffers and the workspace
        s["bn"] = bn
        if op == "add_norm":
            s["out"] = dict(H=torch.empty_like(s["X"]), Xq=torch.empty(s["X"].shape, dtype=torch.int8, device=DEV),
                            absmax=torch.empty(T, device=DEV), rinv=torch.empty(T, device=DEV))
        elif op == "norm_grad":
            s["out"] = dict(dH=torch.empty_like(s["H"]), dw=torch.empty(K, device=DEV))
            s["ws"] = bn.Workspace(bn.load().bitnet_rmsnorm_grad_workspace_size(T, K))
        elif op == "rope":
            s["out"], s["ws"] = dict(Y=torch.empty_like(s["X"])), bn.Workspace(256)
        elif op == "append":
            s["out"], s["ws"] = dict(Q=torch.empty((T, heads * d), dtype=BF16, device=DEV)), bn.Workspace(256)
        else:
            s["out"] = dict(O=torch.empty_like(s["Q"]), lse=torch.empty((case["seqs"], heads), device=DEV))
            s["ws"] = bn.Workspace(bn.load().bitnet_paged_attn_workspace_size(case["seqs"], heads, kv, d))
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if own:
        return _RUN_OWN[c["op"]](s, c)
    return _RUN[c["op"]](s, c)


def _run_add_norm_own(s, c):
    H, Xq, a, r = s["bn"].bitnet_add_rmsnorm_quant(s["X"], s["R"], w=s["w"], eps_norm=EPS_NORM, eps_act=EPS_ACT, **s["out"])
    return {"H": H, "codes": Xq, "absmax": a, "rinv": r}


def _run_norm_grad_own(s, c):
    dH, dw = s["bn"].bitnet_rmsnorm_grad(s["dY"], s["H"], s["rinv"], w=s["w"], dR=s["dR"], ws=s["ws"], **s["out"])
    return {"dH": dH, "dw": dw}


def _run_rope_own(s, c):
    return s["bn"].bitnet_rope(s["X"], s["pos"], s["table"], c["heads"], interleaved=c["interleaved"], inverse=c["inverse"],
                               ws=s["ws"], **s["out"])


def _run_append_own(s, c):
    Q = s["bn"].bitnet_rope_append(s["QKV"], s["pos"], s["table"], s["k"], s["v"], s["pages"], seq=s["seq"],
                                   interleaved=c["interleaved"], ws=s["ws"], **s["out"])
    return {"Q": Q, "k": s["k"], "v": s["v"]}


def _run_attn_own(s, c):
    O = s["bn"].bitnet_paged_attn(s["Q"], s["k"], s["v"], s["pages"], s["lens"], scale=s["scale"], ws=s["ws"], **s["out"])
    return {"O": O, "lse": s["out"]["lse"]}


def _run_add_norm(s, c):
    H = (s["X"].float() + s["R"].float()).to(BF16)
    x = H.float()
    ms = x.double().square().mean(-1, keepdim=True).float()   # the definition rounds the exact mean square once
    r = (ms + EPS_NORM).sqrt().reciprocal()
    y = x * r * s["w"]
    a = y.abs().amax(-1, keepdim=True).clamp(min=EPS_ACT)
    # (a tensor over a tensor: one rounded division, where a number over a tensor is a reciprocal and a product)
    q = (y * (torch.full_like(a, 127.0) / a)).round().clamp(-127, 127).to(torch.int8)   # codes: whole numbers, fixed bit for bit
    return {"H": H, "codes": q, "absmax": a[:, 0], "rinv": r[:, 0]}


def _run_norm_grad(s, c):
    h, g, r = s["H"].float(), s["dY"].float(), s["rinv"][:, None]
    xh = h * r
    gw = g * s["w"]
    d = r * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    if s["dR"] is not None:
        d = d + s["dR"].float()
    return {"dH": d.to(BF16), "dw": (g * xh).sum(0)}


def _rotate(x, cs, interleaved, inverse):
    """x [T, heads, d] fp32 with its first 2 * cs.shape[1] features rotated; cs [T, rot / 2, 2]."""
    n = cs.shape[1]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    if inverse:
        sin = -sin
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((y, x[..., 2 * n:]), -1)


def _run_rope(s, c):
    x = s["X"].float().view(c["T"], c["heads"], c["d"])
    y = _rotate(x, s["table"][s["pos"].long()], c["interleaved"], c["inverse"])
    return y.reshape(c["T"], -1).to(s["X"].dtype)


def _run_append(s, c):
    heads, kv, d, page = c["heads"], c["kv_heads"], c["d"], c["page"]
    x = s["QKV"].float().view(-1, heads + 2 * kv, d)
    pos = s["pos"].long()
    qk = _rotate(x[:, :heads + kv], s["table"][pos], c["interleaved"], False).to(BF16)
    at = s["pages"].long()[s["seq"].long(), pos // page]
    s["k"][at, :, pos % page] = qk[:, heads:]
    s["v"][at, :, pos % page] = x[:, heads + kv:].to(BF16)
    return {"Q": qk[:, :heads].reshape(-1, heads * d), "k": s["k"], "v": s["v"]}


def _run_attn(s, c):
    B, heads, kv, d = c["seqs"], c["heads"], c["kv_heads"], c["d"]
    at = s["pages"].long().clamp(min=0)
    n = at.shape[1] * c["page"]
    live = torch.arange(n, device=DEV) < s["lens"][:, None, None, None]
    q = s["Q"].float().view(B, kv, heads // kv, d)
    k = s["k"][at].permute(0, 2, 1, 3, 4).reshape(B, kv, n, d).float()
    x = ((q @ k.transpose(-1, -2)) * s["scale"]).masked_fill(~live, -math.inf)
    del k
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    v = s["v"][at].permute(0, 2, 1, 3, 4).reshape(B, kv, n, d).float()
    o = (p @ v) / torch.where(total > 0, total, 1.0)
    return {"O": o.reshape(B, heads * d).to(BF16), "lse": (top + total.log())[..., 0].reshape(B, heads)}


_RUN = dict(add_norm=_run_add_norm, norm_grad=_run_norm_grad, rope=_run_rope, append=_run_append, attn=_run_attn)
_RUN_OWN = dict(add_norm=_run_add_norm_own, norm_grad=_run_norm_grad_own, rope=_run_rope_own, append=_run_append_own,
                attn=_run_attn_own)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "add_norm":
        n = case["T"] * case["K"]
        return {"bytes": 7 * n + 4 * case["K"] + 8 * case["T"], "flops": 8 * n}
    if op == "norm_grad":
        n = case["T"] * case["K"]
        each = (2 if case["dy"] == "bf16" else 4) + 2 + 2 + (2 if case["residual"] else 0)
        return {"bytes": each * n + 8 * case["K"] + 4 * case["T"], "flops": 10 * n}
    size = 4 if case.get("dtype") == "f32" else 2
    if op == "rope":
        n = case["T"] * case["heads"]
        used = min(case["T"], case["n_pos"])
        return {"bytes": 2 * size * n * case["d"] + 4 * case["T"] + 4 * used * case["rot"], "flops": 3 * n * case["rot"]}
    if op == "append":
        T, heads, kv, d = case["seqs"] * case["new"], case["heads"], case["kv_heads"], case["d"]
        rows = T * (heads + 2 * kv) * d
        return {"bytes": (size + 2) * rows + T * (12 + 4 * case["rot"]), "flops": 3 * T * (heads + kv) * case["rot"]}
    keys, B, heads, kv, d = sum(_lens(case)), case["seqs"], case["heads"], case["kv_heads"], case["d"]
    return {"bytes": 4 * keys * kv * d + 4 * B * heads * d + 4 * B * heads + 4 * B + 4 * (keys // case["page"]),
            "flops": 4 * keys * heads * d}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "add_norm":
        # the codes' definition: every step rounded once to fp32, in this order
        f = lambda v: v.float().double()   # noqa: E731
        H = (s["X"].double() + s["R"].double()).float().to(BF16).double()
        r = f(1 / f(torch.sqrt(f(f((H * H).sum(1) / case["K"]) + f(torch.tensor(EPS_NORM, dtype=torch.float64))))))
        y = f(f(H * r[:, None]) * s["w"].double())
        a = torch.maximum(y.abs().max(1).values, f(torch.tensor(EPS_ACT, dtype=torch.float64)).to(y.device))
        q = torch.round(f(y * f(torch.full_like(a, 127.0) / a)[:, None]))
        return {"H": H, "codes": q.to(torch.int8), "absmax": a, "rinv": r}
    if op == "norm_grad":
        h, g, r, w = s["H"].double(), s["dY"].double(), s["rinv"].double()[:, None], s["w"].double()
        dot = (g * w * h).sum(1, keepdim=True)
        d = r * w * g - r ** 3 / case["K"] * dot * h
        if case["residual"]:
            d = d + s["dR"].double()
        return {"dH": d, "dw": torch.einsum("tk,tk,t->k", g, h, r[:, 0])}
    if op == "rope":
        return _turned(s["X"].double().view(case["T"], case["heads"], case["d"]), s["table"].double()[s["pos"].long()],
                       case["interleaved"], -1 if case["inverse"] else 1).flatten(1)
    if op == "append":
        heads, kv, page = case["heads"], case["kv_heads"], case["page"]
        x = s["QKV"].double().view(-1, heads + 2 * kv, case["d"])
        x[:, :heads + kv] = _turned(x[:, :heads + kv], s["table"].double()[s["pos"].long()], case["interleaved"], 1)
        k, v = s["k"].double(), s["v"].double()
        page_of = torch.stack([s["pages"][b, p // page] for b, p in zip(s["seq"].tolist(), s["pos"].tolist())]).long()
        row = s["pos"].long() % page
        k[page_of, :, row] = x[:, heads:heads + kv]
        v[page_of, :, row] = x[:, heads + kv:]
        return {"Q": x[:, :heads].flatten(1), "k": k, "v": v}
    heads, kv, d = case["heads"], case["kv_heads"], case["d"]
    out = torch.zeros(case["seqs"], heads, d, dtype=torch.float64, device=DEV)
    lse = torch.full((case["seqs"], heads), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(_lens(case)):
        if n == 0:
            continue
        used = s["pages"][b, :-(-n // case["page"])].long()
        for j in range(kv):
            k = s["k"][used, j].flatten(0, 1)[:n].double()
            v = s["v"][used, j].flatten(0, 1)[:n].double()
            mine = slice(j * heads // kv, (j + 1) * heads // kv)
            z = s["Q"].double().view(case["seqs"], heads, d)[b, mine] @ k.T * s["scale"]
            lse[b, mine] = torch.logsumexp(z, 1)
            out[b, mine] = torch.exp(z - lse[b, mine][:, None]) @ v
    return {"O": out.flatten(1), "lse": lse}


def _turned(x, cs, interleaved, sign):
    """Complex rotation of the pairs of x [T, heads, d] by sign times the angles of cs [T, rot / 2, 2]."""
    n = cs.shape[1]
    turn = torch.complex(cs[..., 0], sign * cs[..., 1])[:, None]
    y = x.clone()
    if interleaved:
        z = torch.complex(x[..., 0:2 * n:2], x[..., 1:2 * n:2]) * turn
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :n], x[..., n:2 * n]) * turn
        y[..., :n], y[..., n:2 * n] = z.real, z.imag
    return y
