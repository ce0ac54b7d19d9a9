"""Measured cases of a training step's operators: router balance and 8-bit activation checkpoints.

Four operators, each in its plain form (elementary torch operations in 32 or
64 bits, rounded once at the end) and through the framework's entry points:

* ``balance``  the load-balancing loss over ragged sequences with the router's
  z-loss: expert counts per sequence, both losses and the logits' gradient.
* ``router``   what that dense gradient gives behind the logits: the input
  gradient dx + dlogits W_g and the router's weight gradient dW + dlogits^T x.
* ``swiglu``   the experts' backward through w2 and the SwiGLU from a1, a3 kept
  in 8 bits (E4M3, one power-of-two scale per 32 elements of a row): da1, da3,
  the weighted h that w2's gradient needs, and the gradient of the row weights.
* ``weights``  the experts' weight gradient dy^T x per expert from token rows x
  kept in the same 8 bits, read in expert order.
"""
import math

import torch

own = False

BF16, F32, F64, I32, U8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8
E4M3 = torch.float8_e4m3fn
COEF, ZCOEF = 0.01, 0.001


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # the router of a micro-batch: one short sequence, latency
        dict(name="balance_small", op="balance", tokens=256, experts=8, top_k=2, seqs=1, gate="softmax", pad=0.0),
        # packed documents of uneven lengths, empty ones among them, a padded tail, a number of experts off 32
        dict(name="balance_ragged", op="balance", tokens=3109, experts=60, top_k=4, seqs=37, gate="sigmoid", pad=0.1),
        # the router of a full training batch of fine-grained experts
        dict(name="balance_large", op="balance", tokens=16384, experts=256, top_k=8, seqs=8, gate="sigmoid", pad=0.0),
        # the dense router gradient of a small layer, odd token count
        dict(name="router_small", op="router", tokens=257, d=512, experts=16),
        # a full batch, few experts: the traffic of x and dx
        dict(name="router_few", op="router", tokens=4096, d=4096, experts=8),
        # a full batch, many experts
        dict(name="router_large", op="router", tokens=4096, d=7168, experts=256),
        # a micro-batch of a small layer: ragged groups, partial tiles
        dict(name="swiglu_small", op="swiglu", rows=3108, d=512, f=256, experts=16, skew=1.0),
        # fine-grained experts, about 128 rows each
        dict(name="swiglu_fine", op="swiglu", rows=8192, d=7168, f=2048, experts=64, skew=0.5),
        # a full batch on eight large experts: tensor rate
        dict(name="swiglu_large", op="swiglu", rows=8192, d=4096, f=14336, experts=8, skew=0.3),
        # weight gradients of a micro-batch of a small layer
        dict(name="weights_small", op="weights", tokens=777, top_k=4, m=256, k=512, experts=16, skew=1.0),
        # the up projection's gradient of fine-grained experts: fp32 output traffic
        dict(name="weights_fine", op="weights", tokens=1024, top_k=8, m=2048, k=7168, experts=64, skew=0.5),
        # the up projection's gradient of eight large experts: tensor rate
        dict(name="weights_large", op="weights", tokens=4096, top_k=2, m=14336, k=4096, experts=8, skew=0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "router", "swiglu", "weights"])
    if op == "balance":
        experts = _log(rng, 2, 512)
        tokens = _log(rng, 1, 32768)
        while tokens * experts > 16384 * 256:
            tokens //= 2
        return dict(op=op, tokens=tokens, experts=experts, top_k=min(experts, rng.choice([1, 2, 4, 6, 8])),
                    seqs=min(tokens, _log(rng, 1, 400)), gate=rng.choice(["softmax", "sigmoid"]),
                    pad=rng.choice([0.0, 0.0, 0.05, 0.5]))
    d = 64 * _log(rng, 2, 112)
    if op == "router":
        return dict(op=op, tokens=_log(rng, 1, 4096), d=d, experts=_log(rng, 2, 256))
    experts = rng.choice([1, 3, 8, 16, 40, 64])
    f = 64 * _log(rng, 2, 224)
    rows = _log(rng, 1, 8192)
    while experts * d * f > 900_000_000:
        experts = max(1, experts // 2)
    while 2 * rows * d * f > 9.6e11:
        rows //= 2
    skew = round(rng.uniform(0.0, 1.2), 3)
    if op == "swiglu":
        return dict(op=op, rows=rows, d=d, f=f, experts=experts, skew=skew)
    top_k = min(experts, rng.choice([1, 2, 4, 8]))
    m, k = rng.choice([(d, f), (f, d)])
    return dict(op=op, tokens=max(1, rows // top_k), top_k=top_k, m=m, k=k, experts=experts, skew=skew)


# ------------------------------------------------------------------ the inputs
def _normal(g, shape, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device="cuda", dtype=F32) * std).to(dtype)


def _kept(v):
    """fp32 rows [rows, cols] kept in 8 bits: E4M3 codes and, per 32 elements of a row, the exponent byte
    127 + floor(log2(largest)) - 8 of a power-of-two scale, [cols / 32, rows rounded up to 16]."""
    rows, cols = v.shape
    b = v.view(rows, cols // 32, 32)
    top = b.abs().amax(2)
    e = (torch.frexp(top).exponent - 9).clamp(-127, 127)
    e = torch.where(top > 0, e, torch.full_like(e, -127))
    codes = torch.ldexp(b, -e[:, :, None]).clamp(-448, 448).to(E4M3).view(U8).view(rows, cols)
    scales = torch.zeros(cols // 32, -(-rows // 16) * 16, dtype=U8, device=v.device)
    scales[:, :rows] = (e + 127).to(U8).t()
    return codes, scales


def _lengths(total, parts, c):
    """Uneven lengths that sum to ``total``; about one in eight is empty where there are many."""
    share = torch.rand(parts, generator=c) + 0.2
    if parts >= 8:
        share[torch.rand(parts, generator=c) < 0.125] = 0.0
        share[0] = 1.0
    cut = torch.round(share.cumsum(0) / share.sum() * total).long()
    return [0] + cut.tolist()


def _groups(rows, experts, skew, c):
    share = torch.softmax(skew * torch.randn(experts, generator=c), 0)
    pick = torch.multinomial(share, rows, replacement=True, generator=c)
    return [0] + torch.bincount(pick, minlength=experts).cumsum(0).tolist()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.Generator().manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "balance":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        used = t - int(t * case["pad"])
        s["seq"] = _lengths(used, case["seqs"], c)
        s["seq_offsets"] = torch.tensor(s["seq"], dtype=I32, device="cuda")
        s["logits"] = _normal(g, (t, e), 1.3, F32) + 0.7 * torch.randn(e, generator=g, device="cuda")
        bias = 0.3 * torch.randn(e, generator=g, device="cuda")
        s["topk_idx"] = (s["logits"] + bias).topk(k, dim=1).indices.to(I32)
    elif op == "router":
        t, d, e = case["tokens"], case["d"], case["experts"]
        row = torch.exp(0.5 * torch.randn(t, 1, generator=g, device="cuda"))
        row[torch.rand(t, 1, generator=g, device="cuda") < 0.05] = 0.0   # padding tokens
        s["dlogits"] = _normal(g, (t, e), 1e-2, F32) * row
        s["x"], s["w_gate"] = _normal(g, (t, d)), _normal(g, (e, d), 0.02)
        s["dx_in"], s["dw_in"] = _normal(g, (t, d), 1e-2), _normal(g, (e, d), 0.1, F32)
    elif op == "swiglu":
        r, d, f, e = case["rows"], case["d"], case["f"], case["experts"]
        s["off"] = _groups(r, e, case["skew"], c)
        s["offsets"] = torch.tensor(s["off"], dtype=I32, device="cuda")
        s["dy"] = _normal(g, (r, d))
        s["row_w"] = torch.rand(r, generator=g, device="cuda") * 0.8 + 0.1
        s["w2"] = torch.empty(e, d, f, device="cuda", dtype=BF16)
        for i in range(e):
            s["w2"][i] = _normal(g, (d, f), 0.02)
        for key in ("a1", "a3"):
            s[key], s[key + "_scale"] = _kept(_normal(g, (r, f), 1.2, F32))
    else:
        t, k, e = case["tokens"], case["top_k"], case["experts"]
        r = t * k
        s["off"] = _groups(r, e, case["skew"], c)
        s["offsets"] = torch.tensor(s["off"], dtype=I32, device="cuda")
        s["copy_of_row"] = torch.randperm(r, generator=c).to(I32).cuda()
        s["dy"] = _normal(g, (r, case["m"]), 0.1)
        s["x"], s["x_scale"] = _kept(_normal(g, (t, case["k"]), 1.0, F32))
    if own:
        _own_state(s)
    return s


# --------------------------------------------------------------- the plain form
def _values(codes, scales):
    """What kept rows stand for, in fp32."""
    rows, cols = codes.shape
    e = scales[:, :rows].t().to(torch.int32) - 127
    return torch.ldexp(codes.view(E4M3).float().view(rows, cols // 32, 32), e[:, :, None]).view(rows, cols)


def _plain_balance(s):
    t, e, k, n = s["tokens"], s["experts"], s["top_k"], s["seqs"]
    counts = torch.zeros(n, e, device="cuda", dtype=I32)
    grad = torch.zeros(t, e, device="cuda", dtype=F32)
    off = s["seq_offsets"].long()
    row = torch.arange(t, device="cuda")
    seq = torch.searchsorted(off, row, right=True) - 1   # the last sequence that starts at or before a token
    inside = (row >= off[0]) & (row < off[-1])
    seq = seq.clamp(0, n - 1)
    hit = (seq[:, None] * e + s["topk_idx"].long())[inside].flatten()
    counts.view(-1).index_add_(0, hit, torch.ones_like(hit, dtype=I32))
    length = (off[1:] - off[:-1])
    full = (length > 0).sum()
    used = inside.sum()
    lg = s["logits"]
    top = lg.max(1, keepdim=True).values
    ex = torch.exp(lg - top)
    z = ex.sum(1, keepdim=True)
    soft = ex / z
    lse = (top + torch.log(z))[:, 0]
    if s["gate"] == "softmax":
        q = dq = soft
    else:
        sg = 1 / (1 + torch.exp(-lg))
        total = sg.sum(1, keepdim=True)
        q, dq = sg / total, sg * (1 - sg) / total
    span = length[seq].float()[:, None].clamp_min(1)
    share = counts[seq].float() / span
    inner = (share * q).sum(1, keepdim=True)
    factor = COEF * e / (full.float().clamp_min(1) * span)
    g = factor * dq * (share - inner) + (2 * ZCOEF / used.float().clamp_min(1)) * lse[:, None] * soft
    grad[inside] = g[inside]
    balance = (factor * inner)[inside].double().sum()
    square = (lse[inside].double() ** 2).sum() * (ZCOEF / used.double().clamp_min(1))
    return counts, torch.stack([balance, square]).float(), grad


def _plain_router(s):
    dl = s["dlogits"]
    dx = s["dx_in"].float() + dl @ s["w_gate"].float()
    return dx.to(BF16), s["dw_in"] + dl.t() @ s["x"].float()


def _plain_swiglu(s):
    r, f = s["rows"], s["f"]
    da1, da3, h = (torch.empty(r, f, device="cuda", dtype=BF16) for _ in range(3))
    dw = torch.empty(r, device="cuda", dtype=F32)
    a1, a3 = _values(s["a1"], s["a1_scale"]), _values(s["a3"], s["a3_scale"])
    for e in range(s["experts"]):
        lo, hi = s["off"][e], s["off"][e + 1]
        if hi > lo:
            dh = s["dy"][lo:hi].float() @ s["w2"][e].float()
            u, v, w = a1[lo:hi], a3[lo:hi], s["row_w"][lo:hi, None]
            sg = 1 / (1 + torch.exp(-u))
            act = u * sg
            da3[lo:hi] = w * dh * act
            da1[lo:hi] = w * dh * v * (sg + act * (1 - sg))
            h[lo:hi] = w * act * v
            dw[lo:hi] = (dh * act * v).sum(1)
    return da1, da3, h, dw


def _plain_weights(s):
    dw = torch.zeros(s["experts"], s["m"], s["k"], device="cuda", dtype=F32)
    x = _values(s["x"], s["x_scale"])
    token = (s["copy_of_row"] // s["top_k"]).long()
    for e in range(s["experts"]):
        lo, hi = s["off"][e], s["off"][e + 1]
        if hi > lo:
            dw[e] = s["dy"][lo:hi].float().t() @ x[token[lo:hi]]
    return dw


# ---------------------------------------------------- the framework's operators
def _own_state(s):
    """The descriptor, workspace and buffers that a user's program keeps."""
    from ragged_grouped_gemm_gb300 import api
    from ragged_grouped_gemm_gb300.inputs import MoEConfig

    empty = lambda *shape, dt=BF16: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    op, e = s["op"], s["experts"]
    if op == "balance":
        t = s["tokens"]
        s["desc"] = api.make_desc(MoEConfig("case", t, 64, 64, e, s["top_k"], gate=s["gate"]))
        need = api.moe_workspace_size(s["desc"])[0]
        s.update(counts=empty(s["seqs"], e, dt=I32), loss=empty(2, dt=F32), grad=empty(t, e, dt=F32))
    elif op == "router":
        t, d = s["tokens"], s["d"]
        s["desc"] = api.make_desc(MoEConfig("case", t, d, 64, e, 1))
        need = api.moe_workspace_size(s["desc"])[1]
        s.update(dx=empty(t, d), dw=empty(e, d, dt=F32))
    elif op == "swiglu":
        r, f = s["rows"], s["f"]
        need = api.moe_swiglu_backward_ckpt_workspace_size(e, r, s["d"], f)
        s.update(da1=empty(r, f), da3=empty(r, f), h=empty(r, f), dg=empty(r, dt=F32))
    else:
        need = api.moe_grouped_wgrad_ckpt_workspace_size(e, s["tokens"] * s["top_k"], s["m"], s["k"])
        s.update(dw=empty(e, s["m"], s["k"], dt=F32))
    s["ws"] = torch.empty(need, dtype=U8, device="cuda")
    api.moe_workspace_init(s["ws"])


def _own_run(s):
    from ragged_grouped_gemm_gb300 import api

    op = s["op"]
    if op == "balance":
        api.moe_balance_loss(s["desc"], s["logits"], s["topk_idx"], s["seq_offsets"], s["counts"], s["loss"],
                             s["grad"], s["ws"], coef=COEF, z_coef=ZCOEF)
        return s["counts"], s["loss"], s["grad"]
    if op == "router":
        api.moe_router_backward(s["desc"], s["dlogits"], s["x"], s["w_gate"], s["dx_in"], s["dx"], s["dw_in"],
                                s["dw"], s["ws"])
        return s["dx"], s["dw"]
    if op == "swiglu":
        api.moe_swiglu_backward_ckpt(s["dy"], s["offsets"], s["w2"], s["row_w"], s["a1"], s["a1_scale"], s["a3"],
                                     s["a3_scale"], s["da1"], s["da3"], s["h"], s["dg"], s["ws"])
        return s["da1"], s["da3"], s["h"], s["dg"]
    api.moe_grouped_wgrad_ckpt(s["dy"], s["x"], s["x_scale"], s["offsets"], s["copy_of_row"], s["top_k"], s["dw"],
                               s["ws"])
    return s["dw"]


def run(state):
    if own:
        return _own_run(state)
    return {"balance": _plain_balance, "router": _plain_router, "swiglu": _plain_swiglu,
            "weights": _plain_weights}[state["op"]](state)


# ------------------------------------------------------------------------- work
def work(case):
    op, e = case["op"], case["experts"]
    if op == "balance":
        t, k, n = case["tokens"], case["top_k"], case["seqs"]
        return {"bytes": 8 * t * e + 4 * t * k + 4 * (n + 1) + 4 * n * e + 8, "flops": 20 * t * e}
    if op == "router":
        t, d = case["tokens"], case["d"]
        return {"bytes": 4 * t * e + 6 * t * d + 2 * e * d + 8 * e * d, "flops": 4 * t * d * e}
    if op == "swiglu":
        r, d, f = case["rows"], case["d"], case["f"]
        hit = min(e, r)
        kept = 2 * r * f + 2 * r * f // 32
        return {"bytes": 2 * r * d + 2 * hit * d * f + kept + 6 * r * f + 8 * r + 4 * (e + 1),
                "flops": 2 * r * d * f + 20 * r * f}
    t, r, m, k = case["tokens"], case["tokens"] * case["top_k"], case["m"], case["k"]
    return {"bytes": 2 * r * m + t * k + t * k // 32 + 4 * r + 4 * e * m * k + 4 * (e + 1), "flops": 2 * r * m * k}


# ------------------------------------------------------------- from 64 bits
def _decoded64(codes, scales):
    """Kept rows bit by bit in 64 bits."""
    b = codes.to(torch.int64)
    ex, man = (b >> 3) & 15, (b & 7).double()
    v = torch.where(ex > 0, (8 + man) * torch.exp2((ex - 10).double()), man * 2.0 ** -9)
    v = torch.where(b > 127, -v, v)
    s = torch.exp2(scales[:, :codes.shape[0]].double() - 127)
    return v * s.t().repeat_interleave(32, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    op, e = case["op"], case["experts"]
    if op == "balance":
        seq, n = s["seq"], case["seqs"]
        lg = s["logits"].double()
        prob = torch.softmax(lg, 1)
        lse = torch.logsumexp(lg, 1)
        counts = torch.zeros(n, e, device="cuda", dtype=I32)
        grad = torch.zeros(case["tokens"], e, device="cuda", dtype=F64)
        spans = [(i, a, b) for i, (a, b) in enumerate(zip(seq, seq[1:])) if a < b]
        used = sum(b - a for _, a, b in spans)
        balance = torch.zeros((), device="cuda", dtype=F64)
        square = torch.zeros((), device="cuda", dtype=F64)
        for i, a, b in spans:
            counts[i] = torch.bincount(s["topk_idx"][a:b].flatten(), minlength=e).to(I32)
            f = counts[i].double() / (b - a)
            if case["gate"] == "softmax":
                q = prob[a:b]
                slope = q
            else:
                u = torch.sigmoid(lg[a:b])
                total = u.sum(1, keepdim=True)
                q, slope = u / total, u * torch.sigmoid(-lg[a:b]) / total
            scale = COEF * e / len(spans)
            balance += scale * torch.dot(f, q.mean(0))
            square += ZCOEF / used * torch.dot(lse[a:b], lse[a:b])
            grad[a:b] = (scale / (b - a) * slope * (f[None] - torch.mv(q, f)[:, None])
                         + 2 * ZCOEF / used * lse[a:b, None] * prob[a:b])
        return counts, torch.stack([balance, square]), grad
    if op == "router":
        dl = s["dlogits"].double()
        return (torch.addmm(s["dx_in"].double(), dl, s["w_gate"].double()),
                torch.addmm(s["dw_in"].double(), dl.T, s["x"].double()))
    if op == "swiglu":
        r, f = case["rows"], case["f"]
        da1, da3, h = (torch.empty(r, f, device="cuda", dtype=F64) for _ in range(3))
        dw = torch.empty(r, device="cuda", dtype=F64)
        for i, (lo, hi) in enumerate(zip(s["off"], s["off"][1:])):
            if lo < hi:
                rows = slice(lo, hi)
                dh = torch.mm(s["dy"][rows].double(), s["w2"][i].double())
                # the kept scales of these rows: columns lo .. hi
                u = _decoded64(s["a1"][rows], s["a1_scale"][:, rows])
                v = _decoded64(s["a3"][rows], s["a3_scale"][:, rows])
                w = s["row_w"][rows, None].double()
                up, down = torch.sigmoid(u), torch.sigmoid(-u)
                silu = torch.nn.functional.silu(u)
                h[rows] = w * silu * v
                da3[rows] = w * dh * silu
                da1[rows] = w * dh * v * up * (1 + u * down)
                dw[rows] = torch.einsum("rf,rf->r", dh, silu * v)
        return da1, da3, h, dw
    dw = torch.zeros(e, case["m"], case["k"], device="cuda", dtype=F64)
    x = _decoded64(s["x"], s["x_scale"])
    token = torch.div(s["copy_of_row"].long(), case["top_k"], rounding_mode="floor")
    for i, (lo, hi) in enumerate(zip(s["off"], s["off"][1:])):
        if lo < hi:
            torch.mm(s["dy"][lo:hi].double().T, x[token[lo:hi]], out=dw[i])
    return dw
