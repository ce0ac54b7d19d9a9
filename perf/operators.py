"""Measured cases of the operators around and inside an FP8 pre-norm MoE block.

Four operators, each in its plain form (elementary torch operations in 32
bits, rounded once at the end) and through the framework's entry points:

* ``product``  matrix products grouped by expert on 8-bit operands: activations
  quantised to E4M3 with one fp32 scale per 1 x 128 block, weights held as E4M3
  codes with one fp32 scale per 128 x 128 tile.  ``grad`` false: C = A W^T with
  W [E, n, k]; true: the data gradient C = A W with W [E, k, n].
* ``experts``  the expert layer on those products: dispatch, w1 | w3 with
  SwiGLU, h quantised per 1 x 128 block, w2, combine.
* ``norm``     layer norm; with ``train`` its backward too (residual gradient
  added, weight and bias gradients reduced over the tokens).
* ``dropout``  combine of the expert outputs, dropout from a counter-based
  generator and the residual sum; with ``train`` the backward mask as well.
"""
import math

import torch

own = False

BF16, F32, F64, I32, U8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8
E4M3 = torch.float8_e4m3fn
EPS = 1e-5


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one token through eight of sixteen experts' up projections: weight bytes and latency
        dict(name="product_decode", op="product", groups=16, rows=8, n=2048, k=7168, grad=False, skew=0.0),
        # a micro-batch of a small layer: odd rows, ragged groups, partial tiles on both sides
        dict(name="product_ragged", op="product", groups=16, rows=3109, n=464, k=592, grad=False, skew=1.0),
        # up projection of a full batch on eight large experts: tensor rate
        dict(name="product_large", op="product", groups=8, rows=8192, n=14336, k=4096, grad=False, skew=0.3),
        # data gradient through the up projection of fine-grained experts, about 128 rows each
        dict(name="product_grad", op="product", groups=64, rows=8192, n=7168, k=2048, grad=True, skew=0.5),
        # a decoding step of four tokens, top-8 of sixteen experts
        dict(name="experts_decode", op="experts", tokens=4, d=7168, f=2048, experts=16, top_k=8),
        # a prefill chunk on the same experts, about 128 rows each
        dict(name="experts_chunk", op="experts", tokens=257, d=7168, f=2048, experts=16, top_k=8),
        # a full training or prefill batch on eight large experts
        dict(name="experts_large", op="experts", tokens=4096, d=4096, f=14336, experts=8, top_k=2),
        # the norm of one decoded token
        dict(name="norm_decode", op="norm", tokens=1, d=7168, wide=False, train=False),
        # a training step's norm with an fp32 residual stream, odd token count
        dict(name="norm_odd", op="norm", tokens=1777, d=2560, wide=True, train=True),
        # a training step's norm at full size
        dict(name="norm_large", op="norm", tokens=4096, d=7168, wide=False, train=True),
        # the block's end on a small layer
        dict(name="dropout_small", op="dropout", tokens=777, d=512, top_k=4, shared=True, wide=True, p=0.1, train=True),
        # the block's end at full size
        dict(name="dropout_large", op="dropout", tokens=4096, d=7168, top_k=8, shared=True, wide=False, p=0.1,
             train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _not_listed(v, step):
    return v + step if v == 3072 else v


def draw(rng):
    op = rng.choice(["product", "experts", "norm", "dropout"])
    if op == "product":
        groups = rng.choice([1, 3, 8, 16, 40, 64])
        n = _not_listed(16 * _log(rng, 16, 448), 16)
        k = _not_listed(16 * _log(rng, 16, 448), 16)
        rows = _log(rng, 1, 8192)
        while groups * n * k > 1_000_000_000:
            groups = max(1, groups // 2)
        while 2 * rows * n * k > 9.6e11:
            rows = rows // 2
        return dict(op=op, groups=groups, rows=rows, n=n, k=k, grad=rng.random() < 0.5,
                    skew=round(rng.uniform(0.0, 1.2), 3))
    if op == "experts":
        experts = rng.choice([4, 8, 12, 16, 32])
        d = _not_listed(64 * _log(rng, 4, 112), 64)
        f = _not_listed(64 * _log(rng, 4, 64), 64)
        top_k = rng.choice([1, 2, 4])
        tokens = _log(rng, 1, 4096)
        while experts * d * f > 500_000_000:
            experts //= 2
        while 6 * tokens * top_k * d * f > 2.8e12:
            tokens //= 2
        return dict(op=op, tokens=tokens, d=d, f=f, experts=experts, top_k=min(top_k, experts))
    d = _not_listed(64 * _log(rng, 1, 112), 64)
    tokens = _log(rng, 1, 4096)
    if op == "norm":
        return dict(op=op, tokens=tokens, d=d, wide=rng.random() < 0.4, train=rng.random() < 0.7)
    return dict(op=op, tokens=tokens, d=d, top_k=rng.choice([1, 2, 4, 8]), shared=rng.random() < 0.5,
                wide=rng.random() < 0.4, p=rng.choice([0.0, 0.05, 0.1, 0.3]), train=rng.random() < 0.7)


# ------------------------------------------------------------------ the inputs
def _normal(g, shape, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device="cuda", dtype=F32) * std).to(dtype)


def _weight(g, groups, rows, cols, std=0.02):
    """E4M3 codes [groups, rows, cols] and fp32 scales of their 128 x 128 tiles."""
    codes = torch.empty(groups, rows, cols, device="cuda", dtype=U8)
    tr, tc = -(-rows // 128), -(-cols // 128)
    scales = torch.empty(groups, tr, tc, device="cuda", dtype=F32)
    for e in range(groups):
        w = torch.zeros(tr * 128, tc * 128, device="cuda", dtype=F32)
        w[:rows, :cols] = torch.randn(rows, cols, generator=g, device="cuda", dtype=F32) * std
        t = w.view(tr, 128, tc, 128)
        s = t.abs().amax(dim=(1, 3)) / 448.0
        scales[e] = s
        q = (t / s[:, None, :, None]).view(tr * 128, tc * 128)[:rows, :cols]
        codes[e] = q.to(E4M3).view(U8)
    return codes, scales


def _routing(tokens, experts, top_k, seed):
    """Top-k of uneven random logits: expert indices, weights and the offsets of each expert's rows."""
    c = torch.Generator().manual_seed(seed)
    lg = torch.randn(tokens, experts, generator=c) + 0.5 * torch.randn(experts, generator=c)
    top, idx = lg.topk(top_k, dim=1)
    w = torch.softmax(top, dim=1)
    counts = torch.bincount(idx.flatten(), minlength=experts)
    off = torch.zeros(experts + 1, dtype=torch.int64)
    off[1:] = counts.cumsum(0)
    return idx.to(I32), w, off


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "product":
        e, rows, n, k = case["groups"], case["rows"], case["n"], case["k"]
        c = torch.Generator().manual_seed(seed)
        share = torch.softmax(case["skew"] * torch.randn(e, generator=c), 0)
        pick = torch.multinomial(share, rows, replacement=True, generator=c)
        s["off"] = [0] + torch.bincount(pick, minlength=e).cumsum(0).tolist()
        s["offsets"] = torch.tensor(s["off"], dtype=I32, device="cuda")
        s["a"] = _normal(g, (rows, k))
        s["w"], s["w_scale"] = _weight(g, e, *((k, n) if case["grad"] else (n, k)))
        s["out"] = torch.empty(rows, n, device="cuda", dtype=BF16)
        s["ld"] = -(-(-(-k // 128)) // 4) * 4
        s["codes"] = torch.empty(rows, k, device="cuda", dtype=U8)
        s["scales"] = torch.empty(rows, s["ld"], device="cuda", dtype=F32)
    elif op == "experts":
        t, d, f, e, k = case["tokens"], case["d"], case["f"], case["experts"], case["top_k"]
        idx, w, off = _routing(t, e, k, seed)
        order = torch.sort(idx.flatten().long(), stable=True).indices
        s["off"] = off.tolist()
        s["copy_of_row"] = order.cuda()
        s["x"] = _normal(g, (t, d))
        s["topk_idx"], s["topk_w"], s["offsets"] = idx.cuda(), w.cuda(), off.to(I32).cuda()
        for key, r, c in (("w1", f, d), ("w3", f, d), ("w2", d, f)):
            s[key], s[key + "_scale"] = _weight(g, e, r, c)
    elif op == "norm":
        t, d = case["tokens"], case["d"]
        kind = F32 if case["wide"] else BF16
        s["x"] = (torch.randn(t, d, generator=g, device="cuda") * 1.5
                  + 0.1 * torch.randn(t, 1, generator=g, device="cuda") + 0.7).to(kind)
        s["gamma"] = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
        s["beta"] = 0.1 * torch.randn(d, generator=g, device="cuda")
        s["dy"], s["dres"] = _normal(g, (t, d)), _normal(g, (t, d), 1.0, kind)
    else:
        t, d, k = case["tokens"], case["d"], case["top_k"]
        kind = F32 if case["wide"] else BF16
        perm = torch.randperm(t * k, generator=torch.Generator().manual_seed(seed))
        s["row_of_copy"] = perm.to(I32).cuda()
        s["y_perm"] = _normal(g, (t * k, d))
        s["topk_w"] = torch.softmax(torch.randn(t, k, generator=g, device="cuda"), 1)
        s["y_shared"] = _normal(g, (t, d)) if case["shared"] else None
        s["resid"], s["dout"] = _normal(g, (t, d), 1.0, kind), _normal(g, (t, d), 1.0, kind)
        s["rng"] = torch.tensor([(seed * 7919 + 13) % (1 << 62), (seed * 104729) % (1 << 40)], dtype=torch.int64,
                                device="cuda")
    if own:
        _own_state(s)
    return s


# --------------------------------------------------------------- the plain form
def _quantised(x):
    """The values that 1 x 128 blocks of x stand for in E4M3 with an fp32 scale, in fp32."""
    rows, cols = x.shape
    nb = -(-cols // 128)
    t = torch.nn.functional.pad(x.float(), (0, nb * 128 - cols)).view(rows, nb, 128)
    amax = t.abs().amax(dim=2, keepdim=True)
    s = amax / 448.0
    s = torch.where(s > 0, s, torch.ones_like(s))
    # the quotient in 64 bits: a 32-bit one can land on a border between two codes; odd in its last bit where
    # 32 bits do not hold it, so that the conversion rounds the exact quotient once
    q = t.double() / s.double()
    r = q.float()
    bits = r.view(torch.int32)
    toward = torch.where(r.double().abs() > q.abs(), bits - 1, bits)
    r = torch.where(r.double() == q, bits, toward | 1).view(F32)
    return (r.to(E4M3).float() * s).view(rows, nb * 128)[:, :cols]


def _weights(codes, scales):
    """fp32 values of one matrix of E4M3 codes with 128 x 128 tile scales."""
    r, c = codes.shape
    full = scales.repeat_interleave(128, 0)[:r].repeat_interleave(128, 1)[:, :c]
    return codes.view(E4M3).float() * full


def _plain_product(s):
    a = _quantised(s["a"])
    out = torch.empty(s["rows"], s["n"], device="cuda", dtype=BF16)
    for e in range(s["groups"]):
        lo, hi = s["off"][e], s["off"][e + 1]
        if hi > lo:
            w = _weights(s["w"][e], s["w_scale"][e])
            out[lo:hi] = a[lo:hi] @ (w if s["grad"] else w.t())
    return out


def _plain_experts(s):
    k = s["top_k"]
    x = _quantised(s["x"])
    row = s["copy_of_row"]
    acc = torch.zeros(s["tokens"] * k, s["d"], device="cuda", dtype=F32)
    for e in range(s["experts"]):
        lo, hi = s["off"][e], s["off"][e + 1]
        if hi > lo:
            xe = x[row[lo:hi] // k]
            a1 = xe @ _weights(s["w1"][e], s["w1_scale"][e]).t()
            a3 = xe @ _weights(s["w3"][e], s["w3_scale"][e]).t()
            h = _quantised(a1 / (1 + torch.exp(-a1)) * a3)
            acc[row[lo:hi]] = h @ _weights(s["w2"][e], s["w2_scale"][e]).t()
    return (acc.view(s["tokens"], k, s["d"]) * s["topk_w"][:, :, None]).sum(1).to(BF16)


def _plain_norm(s):
    x, gamma = s["x"].float(), s["gamma"]
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    xhat = c * rstd
    y = (xhat * gamma + s["beta"]).to(BF16)
    if not s["train"]:
        return y, mean[:, 0], rstd[:, 0]
    dy = s["dy"].float()
    gy = dy * gamma
    dx = rstd * (gy - gy.mean(1, keepdim=True) - xhat * (gy * xhat).mean(1, keepdim=True))
    dx = (dx + s["dres"].float()).to(s["x"].dtype)
    return y, mean[:, 0], rstd[:, 0], dx, (dy * xhat).sum(0), dy.sum(0)


def _keep(rng, n, p):
    """True where an element stays: Philox-4x32 with ten rounds (Salmon et al., "Parallel random numbers: as easy
    as 1, 2, 3", 2011), key rng[0], counter rng[1] + i // 4, word i % 4 of each block against p * 2^32."""
    low = 0xFFFFFFFF
    ctr = torch.arange(-(-n // 4), device="cuda", dtype=torch.int64) + rng[1]
    c0, c1 = ctr & low, (ctr >> 32) & low
    c2, c3 = torch.zeros_like(c0), torch.zeros_like(c0)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack([c0, c1, c2, c3], 1).flatten()[:n] >= int(p * 4294967296.0 + 0.5)


def _plain_dropout(s):
    t, d, k, p = s["tokens"], s["d"], s["top_k"], s["p"]
    y = s["y_perm"][s["row_of_copy"].long()].float().view(t, k, d)
    y = (y * s["topk_w"][:, :, None]).sum(1)
    if s["y_shared"] is not None:
        y = y + s["y_shared"].float()
    mask = _keep(s["rng"], t * d, p).view(t, d).float() * (1 / (1 - p))
    out = (s["resid"].float() + mask * y).to(s["resid"].dtype)
    if not s["train"]:
        return out
    return out, (mask * s["dout"].float()).to(BF16)


# ---------------------------------------------------- the framework's operators
def _own_state(s):
    """The descriptor, workspace and buffers that a user's program keeps."""
    from ragged_grouped_gemm_gb300 import api
    from ragged_grouped_gemm_gb300.inputs import MoEConfig

    empty = lambda *shape, dt=BF16: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    op = s["op"]
    if op == "product":
        need = api.moe_grouped_gemm_fp8_workspace_size(s["groups"], s["rows"], s["n"], s["k"])
    else:
        if op == "experts":
            cfg = MoEConfig("case", s["tokens"], s["d"], s["f"], s["experts"], s["top_k"], precision="fp8b")
        else:
            k = s.get("top_k", 1)
            cfg = MoEConfig("case", s["tokens"], s["d"], 64, max(8, k), k)
        s["desc"] = api.make_desc(cfg)
        need = api.moe_workspace_size(s["desc"])[0 if op == "experts" else 1]
        t, d = s["tokens"], s["d"]
    s["ws"] = torch.empty(need, dtype=U8, device="cuda")
    api.moe_workspace_init(s["ws"])
    if op == "experts":
        r, f = t * s["top_k"], s["f"]
        s.update(row_of=empty(r, dt=I32), copy_of=empty(r, dt=I32), xq=empty(r, d, dt=U8),
                 xs=empty(r, api.fp8_scale_ld(d), dt=F32), y_rows=empty(r, d), out=empty(t, d))
        s["wq"] = {key: s[key] for w in ("w1", "w3", "w2") for key in (w, w + "_scale")}
    elif op == "norm":
        s.update(y=empty(t, d), mean=empty(t, dt=F32), rstd=empty(t, dt=F32))
        if s["train"]:
            s.update(dx=torch.empty_like(s["x"]), dgamma=empty(d, dt=F32), dbeta=empty(d, dt=F32))
    elif op == "dropout":
        s.update(out=torch.empty_like(s["resid"]), dmoe=empty(t, d))


def _own_run(s):
    from ragged_grouped_gemm_gb300 import api

    op = s["op"]
    if op == "product":
        api.moe_quantize_fp8_rows(s["a"], s["codes"], s["scales"])
        api.moe_grouped_gemm_fp8(s["codes"], s["scales"], s["offsets"], s["w"], s["w_scale"], s["out"], s["ws"],
                                 b_mn=s["grad"])
        return s["out"]
    if op == "experts":
        api.moe_permute_fp8b(s["desc"], s["x"], s["topk_idx"], s["offsets"], s["row_of"], s["copy_of"], None,
                             s["xq"], s["xs"], None, None, s["ws"])
        api.moe_grouped_ffn_fp8b(s["desc"], s["xq"], s["xs"], s["offsets"], None, None, s["wq"], {}, s["y_rows"],
                                 None, s["ws"])
        api.moe_combine(s["desc"], s["y_rows"], s["row_of"], s["topk_w"], None, s["out"])
        return s["out"]
    if op == "norm":
        api.moe_layernorm(s["desc"], s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"], eps=EPS)
        if not s["train"]:
            return s["y"], s["mean"], s["rstd"]
        api.moe_layernorm_backward(s["desc"], s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["dres"], s["dx"],
                                   s["dgamma"], s["dbeta"], s["ws"])
        return s["y"], s["mean"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"]
    api.moe_combine_dropout(s["desc"], s["y_perm"], s["row_of_copy"], s["topk_w"], s["y_shared"], s["resid"],
                            s["rng"], s["p"], s["out"])
    if not s["train"]:
        return s["out"]
    api.moe_dropout_backward(s["desc"], s["dout"], s["rng"], s["p"], s["dmoe"])
    return s["out"], s["dmoe"]


def run(state):
    if own:
        return _own_run(state)
    return {"product": _plain_product, "experts": _plain_experts, "norm": _plain_norm,
            "dropout": _plain_dropout}[state["op"]](state)


# ------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "product":
        e, r, n, k = case["groups"], case["rows"], case["n"], case["k"]
        hit = min(e, r) if r < e else e
        tiles = -(-n // 128) * -(-k // 128)
        return {"bytes": 2 * r * k + hit * (n * k + 4 * tiles) + 2 * r * n + 4 * (e + 1), "flops": 2 * r * n * k}
    if op == "experts":
        t, d, f, e, k = (case[c] for c in ("tokens", "d", "f", "experts", "top_k"))
        r = t * k
        # experts that r evenly spread copies leave without a row
        hit = e * (1 - (1 - k / e) ** t)
        return {"bytes": 2 * t * d * 2 + 8 * r + hit * 3 * d * f, "flops": 6 * r * d * f}
    t, d = case["tokens"], case["d"]
    sx = 4 if case["wide"] else 2
    if op == "norm":
        b = t * d * (sx + 2) + 8 * t + 8 * d
        if case["train"]:
            b += t * d * (2 + 2 * sx) + 8 * d   # dy, dres, dx; x is read once and its row is at hand
        return {"bytes": b, "flops": t * d * (24 if case["train"] else 8)}
    k = case["top_k"]
    b = t * k * d * 2 + 8 * t * k + t * d * 2 * sx + (t * d * 2 if case["shared"] else 0)
    if case["train"]:
        b += t * d * (sx + 2)
    return {"bytes": b, "flops": t * d * (2 * k + 30)}


# ------------------------------------------------------------- from 64 bits
def _blocks64(x):
    """x [rows, cols] in 64 bits -> the values of its 1 x 128 blocks in E4M3, by rounding to the grid of the code."""
    rows, cols = x.shape
    out = torch.empty_like(x)
    for c in range(0, cols, 128):
        b = x[:, c:c + 128]
        top = b.abs().max(dim=1, keepdim=True).values
        scale = torch.where(top > 0, (top.float() / 448.0), torch.ones_like(top, dtype=F32)).double()
        q = (b / scale).clamp(-448.0, 448.0)
        # spacing of the grid: 2^(e - 3) with e the exponent, at least -6
        e = torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6)))
        step = torch.exp2(e - 3)
        out[:, c:c + 128] = torch.round(q / step) * step * scale
    return out


def _matrix64(codes, scales):
    """A matrix of E4M3 codes and tile scales, bit by bit in 64 bits."""
    b = codes.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).double()), m * 2.0 ** -9)
    v = torch.where(b > 127, -v, v)
    rows, cols = torch.arange(b.shape[0], device=b.device) // 128, torch.arange(b.shape[1], device=b.device) // 128
    return v * scales.double()[rows][:, cols]


def _random32(key, ctr):
    """The four 32-bit words of each counter, in Python's own integers' steps on 16-bit halves."""
    low, half = 0xFFFFFFFF, 0xFFFF

    def wide(x, m):   # high and low words of the 64-bit product of two 32-bit numbers
        xl, xh, ml, mh = x & half, x >> 16, m & half, m >> 16
        mid = xh * ml + ((xl * ml) >> 16)
        mid2 = xl * mh + (mid & half)
        return (xh * mh + (mid >> 16) + (mid2 >> 16)) & low, ((mid2 << 16) | ((xl * ml) & half)) & low

    w = [ctr & low, (ctr >> 32) & low, torch.zeros_like(ctr), torch.zeros_like(ctr)]
    for r in range(10):
        ka, kb = (key + r * 0x9E3779B9) & low, ((key >> 32) + r * 0xBB67AE85) & low
        h0, l0 = wide(w[0], 0xD2511F53)
        h1, l1 = wide(w[2], 0xCD9E8D57)
        w = [h1 ^ w[1] ^ ka, l1, h0 ^ w[3] ^ kb, l0]
    return w


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "product":
        a = _blocks64(s["a"].double())
        out = torch.zeros(case["rows"], case["n"], device="cuda", dtype=F64)
        for e, (lo, hi) in enumerate(zip(s["off"], s["off"][1:])):
            if lo < hi:
                w = _matrix64(s["w"][e], s["w_scale"][e])
                out[lo:hi] = torch.mm(a[lo:hi], w) if case["grad"] else torch.mm(a[lo:hi], w.T)
        return out
    if op == "experts":
        x = _blocks64(s["x"].double())
        k, out = case["top_k"], torch.zeros(case["tokens"], case["d"], device="cuda", dtype=F64)
        for e in range(case["experts"]):
            token, rank = torch.where(s["topk_idx"] == e)
            if token.numel():
                up = torch.mm(x[token], _matrix64(s["w1"][e], s["w1_scale"][e]).T)
                gate = torch.mm(x[token], _matrix64(s["w3"][e], s["w3_scale"][e]).T)
                h = _blocks64(up * torch.sigmoid(up) * gate)
                y = torch.mm(h, _matrix64(s["w2"][e], s["w2_scale"][e]).T)
                out.index_add_(0, token, y * s["topk_w"][token, rank].double()[:, None])
        return out
    if op == "norm":
        x, ga = s["x"].double(), s["gamma"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + EPS).rsqrt()
        xhat = (x - mean[:, None]) * rstd[:, None]
        y = xhat * ga + s["beta"].double()
        if not case["train"]:
            return y, mean, rstd
        dy = s["dy"].double()
        v = dy * ga
        d = case["d"]
        dx = rstd[:, None] / d * (d * v - v.sum(1)[:, None] - xhat * (v * xhat).sum(1)[:, None]) + s["dres"].double()
        return y, mean, rstd, dx, torch.einsum("td,td->d", dy, xhat), dy.sum(0)
    t, d, k = case["tokens"], case["d"], case["top_k"]
    key, first = s["rng"].tolist()
    count = torch.arange((t * d + 3) // 4, device="cuda", dtype=torch.int64) + first
    words = torch.stack(_random32(key, count), dim=-1).reshape(-1)[:t * d].view(t, d)
    p = case["p"]
    kept = words >= round(p * 2 ** 32)
    y = torch.zeros(t, d, device="cuda", dtype=F64) if s["y_shared"] is None else s["y_shared"].double()
    rows = s["row_of_copy"].view(t, k).long()
    for j in range(k):
        y = y + s["topk_w"][:, j, None].double() * s["y_perm"][rows[:, j]].double()
    none = torch.zeros((), device="cuda", dtype=F64)
    out = s["resid"].double() + torch.where(kept, y / (1.0 - p), none)
    if not case["train"]:
        return out
    return out, torch.where(kept, s["dout"].double() / (1.0 - p), none)
