"""The operators around the expert FFN, as cases that can be timed and compared.

Four operators of one mixture-of-experts block: the routing gate (scores, top-k, weights, and its gradient), the
balance loss over the gate's choices (with the per-expert counts and its gradient), the norms before and after the
block with their gate and residual scale (and their gradients), and the 8-bit integer product of the dense expert
that runs beside the routed ones.

With `own` false, `run` computes them from elementary torch operations; with `own` true it calls this package.
`exact` gives the same results in 64 bits: the forward formulas written a second time, the gradients from
differentiating them.
"""
import math

import torch

own = False

SOFTMAX, SIGMOID, SQRT_SOFTPLUS = 0, 1, 2
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # the gate of one decode step of a serving batch: 64 tokens, 8 of 384 experts, softmax weights renormalized
        dict(name="gate_decode", kind="gate", T=64, E=384, k=8, score=SOFTMAX, bias=False, groups=1, top_groups=1,
             dtype="f32", masked=False),
        # the gate of a prefill batch: sigmoid scores, a selection bias, 4 of 8 expert groups, BF16 logits, some padding
        dict(name="gate_prefill_grouped", kind="gate", T=16384, E=256, k=8, score=SIGMOID, bias=True, groups=8,
             top_groups=4, dtype="bf16", masked=True),
        # a training step of the gate: choices and weights, then the gradient of the logits through the weights
        dict(name="gate_train", kind="gate_train", T=8192, E=384, k=8, score=SOFTMAX, bias=False, groups=1,
             top_groups=1, dtype="f32", masked=False),
        # balance loss of one short micro-batch of a small layer (odd numbers of tokens and experts)
        dict(name="balance_small", kind="balance", T=509, E=60, k=4, score=SOFTMAX, B=1, dtype="bf16", masked=True),
        # balance loss of a packed batch of sequences of all lengths, with its gradient
        dict(name="balance_packed", kind="balance", T=16384, E=384, k=8, score=SIGMOID, B=24, dtype="f32",
             masked=True),
        # the residual update and norms around the block in a decode step
        dict(name="norm_decode", kind="norm", T=64, H=7168, x="bf16", res="bf16", gate="channel", post=True),
        # the same for a prefill batch
        dict(name="norm_prefill", kind="norm", T=8192, H=7168, x="bf16", res="bf16", gate="channel", post=True),
        # backward of a training batch, every gradient
        dict(name="norm_train", kind="norm_backward", T=8192, H=7168, x="bf16", res="bf16", gate="channel",
             post=True),
        # backward with a float32 residual stream, a gate for each token, an odd number of tokens, a ragged width
        dict(name="norm_train_f32", kind="norm_backward", T=2047, H=2888, x="bf16", res="f32", gate="token",
             post=True),
        # the dense expert in a decode step: the weights are read once for 64 tokens
        dict(name="int8_decode", kind="int8_ffn", T=64, H=7168, I=2048),
        # one 8-bit projection of a ragged chunk, added to a residual
        dict(name="int8_ragged", kind="int8_linear", T=333, N=1000, K=1040),
        # the dense expert over a prefill batch, added to the routed experts' output
        dict(name="int8_prefill", kind="int8_ffn", T=8192, H=7168, I=2048),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["gate", "gate_train", "balance", "norm", "norm_backward", "int8_ffn", "int8_linear"])
    T = _log_int(rng, 1, 8192)
    if kind in ("gate", "gate_train", "balance"):
        groups = rng.choice([1, 1, 4, 8]) if kind != "balance" else 1
        E = groups * _log_int(rng, 8, 512 // groups)
        k = rng.randint(1, min(12, E // 2))
        case = dict(kind=kind, T=T, E=E, k=k, score=rng.choice([SOFTMAX, SIGMOID, SQRT_SOFTPLUS]),
                    dtype=rng.choice(["f32", "bf16"]), masked=rng.random() < 0.5)
        if kind == "balance":
            case["B"] = _log_int(rng, 1, 48)
        else:
            top = groups if groups == 1 else groups // 2
            case.update(k=min(k, top * (E // groups)), bias=rng.random() < 0.5, groups=groups, top_groups=top)
        return case
    if kind in ("norm", "norm_backward"):
        return dict(kind=kind, T=T, H=8 * _log_int(rng, 16, 1000), x=rng.choice(["bf16", "f32"]),
                    res=rng.choice(["bf16", "f32"]), gate=rng.choice(["none", "channel", "token"]),
                    post=rng.random() < 0.7)
    if kind == "int8_ffn":
        return dict(kind=kind, T=T, H=16 * _log_int(rng, 16, 448), I=16 * _log_int(rng, 8, 128))
    return dict(kind=kind, T=T, N=8 * _log_int(rng, 8, 896), K=16 * _log_int(rng, 4, 448))


# ------------------------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)

    def rand(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    s = {"case": case, "kind": case["kind"]}
    kind, T = case["kind"], case["T"]
    if kind in ("gate", "gate_train", "balance"):
        E, k = case["E"], case["k"]
        # logits as a trained gate has them: a popularity of each expert and the token's own preference
        logits = randn(E, scale=0.5)[None] + randn(T, E, scale=1.5)
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        s["mask"] = (rand(T) > 0.03).to(torch.uint8) if case["masked"] else None
        if kind == "balance":
            ids = torch.topk(s["logits"].float(), k, dim=1).indices.to(torch.int32)
            s["ids"] = ids.contiguous()
            cuts = torch.sort(torch.randint(0, T + 1, (case["B"] - 1,), device="cuda", generator=g)).values
            ends = torch.tensor([0, T], device="cuda")
            s["cu"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
            s["d_loss"] = torch.tensor([1e-2, 1e-3], device="cuda") * (0.5 + rand(2))
        else:
            s["bias"] = randn(E, scale=0.05) if case["bias"] else None
            if kind == "gate_train":
                s["d_w"] = randn(T, k, scale=0.1)
    elif kind in ("norm", "norm_backward"):
        H, xt, rt = case["H"], DTYPES[case["x"]], DTYPES[case["res"]]
        s["x"] = randn(T, H, dtype=xt, scale=0.7)
        s["residual"] = randn(T, H, dtype=rt, scale=2.0)
        s["w_pre"] = 1.0 + randn(H, scale=0.1)
        s["w_post"] = 0.5 + randn(H, scale=0.1) if case["post"] else None
        s["gate"] = (None if case["gate"] == "none" else
                     0.3 + randn(H, scale=0.1) if case["gate"] == "channel" else torch.sigmoid(randn(T, 1)))
        s["scale"] = 0.75
        if kind == "norm_backward":
            s["d_y"] = randn(T, H, dtype=xt, scale=0.02)
            s["d_res"] = randn(T, H, dtype=rt, scale=0.02)
    else:
        def weight(n, c):
            w = randn(n, c, scale=0.02)
            sc = w.abs().amax(1) / 127.0
            return torch.round(w / sc[:, None]).to(torch.int8), sc
        N, K = (2 * case["I"], case["H"]) if kind == "int8_ffn" else (case["N"], case["K"])
        s["x"] = randn(T, K, dtype=torch.bfloat16)
        s["w1"], s["w1_scale"] = weight(N, K)
        if kind == "int8_ffn":
            s["w2"], s["w2_scale"] = weight(case["H"], case["I"])
            if own:
                import nvfp4_quantized_moe_amd as nv
                s["weights"] = nv.Int8FFNWeights(s["w1"], s["w1_scale"], s["w2"], s["w2_scale"])
        s["add"] = randn(T, case["H"] if kind == "int8_ffn" else N, dtype=torch.bfloat16)
    return s


# -------------------------------------------------------------------------------------------------- plain forms

def _score(x, score):
    if score == SOFTMAX:
        e = torch.exp(x - x.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True)
    if score == SIGMOID:
        return 1.0 / (1.0 + torch.exp(-x))
    return torch.sqrt(torch.log1p(torch.exp(-x.abs())) + x.clamp(min=0))


def _plain_gate(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    logits = s["logits"]
    if s["bias"] is None and G == 1:
        key = logits.float()
    else:
        key = _score(logits.double(), c["score"])  # 64 bits: neighbouring sums may differ in the last bits of 32
        if s["bias"] is not None:
            key = key + s["bias"].double()
        if G > 1:
            by = key.view(T, G, E // G)
            two = torch.sort(by, dim=2, descending=True).values[:, :, :2].sum(2)
            best = torch.sort(two, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
            chosen = torch.zeros(T, G, dtype=torch.bool, device=key.device).scatter_(1, best, True)
            key = torch.where(chosen[:, :, None], by, -math.inf).view(T, E)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(_score(logits.float(), c["score"]), 1, ids)
    w = w / w.sum(1, keepdim=True) * 2.5
    ids = ids.to(torch.int32)
    if s["mask"] is not None:
        dead = s["mask"][:, None] == 0
        ids, w = ids.masked_fill(dead, -1), w.masked_fill(dead, 0.0)
    return ids, w


def _plain_gate_grad(s, ids):
    c = s["case"]
    x = s["logits"].float()
    p = _score(x, c["score"])
    at = ids.long().clamp(min=0)
    sel = torch.gather(p, 1, at)
    total = sel.sum(1, keepdim=True)
    dw = s["d_w"] * 2.5
    d_sel = (dw - (dw * sel).sum(1, keepdim=True) / total) / total
    dp = torch.zeros_like(p).scatter_(1, at, d_sel)
    if c["score"] == SOFTMAX:
        dx = p * (dp - (dp * p).sum(1, keepdim=True))
    elif c["score"] == SIGMOID:
        dx = dp * p * (1.0 - p)
    else:
        dx = dp * 0.5 / p / (1.0 + torch.exp(-x))
    if s["mask"] is not None:
        dx = dx.masked_fill(s["mask"][:, None] == 0, 0.0)
    return dx.to(s["logits"].dtype)


def _plain_balance(s):
    c = s["case"]
    T, E, k, B = c["T"], c["E"], c["k"], c["B"]
    x = s["logits"].float()
    live = torch.ones(T, device=x.device) if s["mask"] is None else (s["mask"] != 0).float()
    seq = torch.searchsorted(s["cu"][1:].long(), torch.arange(T, device=x.device), right=True)
    member = ((seq[None] == torch.arange(B, device=x.device)[:, None]) * live).double()  # [B, T]
    sc = _score(x, c["score"])
    total = sc.sum(1, keepdim=True)
    q = sc / total
    chosen = torch.zeros(T, E, device=x.device).scatter_(1, s["ids"].long(), 1.0)
    counts = (member.float() @ chosen).to(torch.int32)
    tokens = member.sum(1)
    sums = member @ q.double()
    n = tokens.clamp(min=1)[:, None]
    seqs = (tokens > 0).sum().clamp(min=1)
    f = counts.double() / (n * k)
    balance = E * (f * sums / n).sum() / seqs
    top = x.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(x - top).sum(1, keepdim=True))
    n_all = tokens.sum().clamp(min=1)
    z = (lse[:, 0].double().square() * live.double()).sum() / n_all
    # gradient: of each token's mean share, and of its squared log-sum
    dq = ((E / (seqs * n)) * f * s["d_loss"][0].double()).float()[seq]
    inner = (dq * q).sum(1, keepdim=True)
    if c["score"] == SOFTMAX:
        dx = q * (dq - inner)
    else:
        ds = (dq - inner) / total
        dx = ds * sc * (1.0 - sc) if c["score"] == SIGMOID else ds * 0.5 / sc / (1.0 + torch.exp(-x))
    dx = dx + (2.0 * s["d_loss"][1] / n_all.float()) * lse * torch.exp(x - lse)
    dx = dx * live[:, None]
    return torch.stack([balance, z]).float(), counts, dx.to(s["logits"].dtype)


def _plain_norm(s):
    x, r = s["x"].float(), s["residual"].float()
    if s["w_post"] is not None:
        x = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * s["w_post"]
    if s["gate"] is not None:
        x = x * s["gate"]
    r = (r + s["scale"] * x).to(s["residual"].dtype)
    f = r.float()  # the block reads the residual stream as it is kept
    y = f * torch.rsqrt((f * f).mean(1, keepdim=True) + EPS) * s["w_pre"]
    return r, y.to(s["x"].dtype)


def _plain_norm_grad(s):
    # here `residual` is the stream after the update, as the forward pass left it
    x, r, dy, dr = s["x"].float(), s["residual"].float(), s["d_y"].float(), s["d_res"].float()
    rho = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    rn = r * rho
    dn = dy * s["w_pre"]
    d_pre = (dy * rn).sum(0)
    dr = dr + rho * (dn - rn * (dn * rn).mean(1, keepdim=True))
    if s["w_post"] is not None:
        sig = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
        xn = x * sig
        n = xn * s["w_post"]
    else:
        n = x
    db = s["scale"] * dr
    d_gate = None
    if s["gate"] is not None:
        d_gate = (db * n).sum(0) if s["case"]["gate"] == "channel" else (db * n).sum(1, keepdim=True)
        db = db * s["gate"]
    d_post = None
    if s["w_post"] is not None:
        d_post = (db * xn).sum(0)
        dxn = db * s["w_post"]
        db = sig * (dxn - xn * (dxn * xn).mean(1, keepdim=True))
    out = {"d_x": db.to(s["x"].dtype), "d_residual": dr.to(s["residual"].dtype), "d_w_pre": d_pre}
    if d_post is not None:
        out["d_w_post"] = d_post
    if d_gate is not None:
        out["d_gate"] = d_gate
    return out


def _plain_linear(x, w, w_scale):
    x = x.float()
    sc = x.abs().amax(1, keepdim=True) / 127.0
    q = torch.round(x.double() / torch.where(sc > 0, sc, 1.0).double()).float()  # 64 bits: halves lie close by
    return (q @ w.float().t()) * sc * w_scale


def _plain_int8(s):
    if s["kind"] == "int8_linear":
        return (_plain_linear(s["x"], s["w1"], s["w1_scale"]) + s["add"].float()).to(torch.bfloat16)
    gu = _plain_linear(s["x"], s["w1"], s["w1_scale"])
    inter = gu.shape[1] // 2
    g, u = gu[:, :inter], gu[:, inter:]
    h = (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16)  # the second product's input is kept in BF16
    return (_plain_linear(h, s["w2"], s["w2_scale"]) + s["add"].float()).to(torch.bfloat16)


# ------------------------------------------------------------------------------------------------------- a pass

def run(s):
    kind, c = s["kind"], s["case"]
    if own:
        import nvfp4_quantized_moe_amd as nv
        if kind in ("gate", "gate_train"):
            ids, w = nv.moe_gate_topk(s["logits"], c["k"], score=c["score"], bias=s["bias"], token_mask=s["mask"],
                                      n_group=c["groups"], topk_group=c["top_groups"], renormalize=True, scale=2.5)
            if kind == "gate":
                return ids, w
            d = nv.moe_gate_backward(s["logits"], ids, score=c["score"], renormalize=True, scale=2.5,
                                     token_mask=s["mask"], d_topk_w=s["d_w"])
            return ids, w, d
        if kind == "balance":
            loss, counts, tokens = nv.moe_balance_loss(s["logits"], s["ids"], score=c["score"],
                                                       token_mask=s["mask"], cu_seqlens=s["cu"])
            d = nv.moe_gate_backward(s["logits"], s["ids"], score=c["score"], token_mask=s["mask"],
                                     d_loss=s["d_loss"], counts=counts, tokens=tokens, cu_seqlens=s["cu"])
            return loss, counts, d
        if kind == "norm":
            return nv.moe_block_norm(s["x"], s["residual"], s["w_pre"], w_post=s["w_post"], gate=s["gate"],
                                     scale=s["scale"], eps=EPS)
        if kind == "norm_backward":
            d = nv.moe_block_norm_backward(s["d_y"], s["d_res"], s["x"], s["residual"], s["w_pre"],
                                           w_post=s["w_post"], gate=s["gate"], scale=s["scale"], eps=EPS)
            return {n: v for n, v in d.items() if v is not None}
        if kind == "int8_linear":
            q, sc = nv.int8_quantize_rows(s["x"])
            return nv.int8_gemm(q, sc, s["w1"], s["w1_scale"], add=s["add"])
        return nv.int8_ffn_forward(s["weights"], s["x"], add=s["add"])
    if kind == "gate":
        return _plain_gate(s)
    if kind == "gate_train":
        ids, w = _plain_gate(s)
        return ids, w, _plain_gate_grad(s, ids)
    if kind == "balance":
        return _plain_balance(s)
    if kind == "norm":
        return _plain_norm(s)
    if kind == "norm_backward":
        return _plain_norm_grad(s)
    return _plain_int8(s)


def work(case):
    kind, T = case["kind"], case["T"]
    size = {"bf16": 2, "f32": 4}
    if kind in ("gate", "gate_train", "balance"):
        E, k, b = case["E"], case["k"], size[case["dtype"]]
        bytes_ = T * E * b + T * k * 8 + (T if case["masked"] else 0)  # logits in; ids and weights out
        if kind == "gate":
            return {"bytes": bytes_ + (4 * E if case["bias"] else 0), "flops": 8 * T * E}
        if kind == "gate_train":
            return {"bytes": bytes_ + T * E * b + T * k * 4 + (4 * E if case["bias"] else 0), "flops": 16 * T * E}
        return {"bytes": 2 * T * E * b + T * k * 4 + 4 * case["B"] * E + T * bool(case["masked"]),
                "flops": 24 * T * E}
    if kind in ("norm", "norm_backward"):
        H, x, r = case["H"], size[case["x"]], size[case["res"]]
        vec = 4 * H * (1 + case["post"] + (case["gate"] == "channel")) + 4 * T * (case["gate"] == "token")
        if kind == "norm":
            return {"bytes": 2 * T * H * (x + r) + vec, "flops": 10 * T * H}
        return {"bytes": T * H * (3 * x + 3 * r) + 2 * vec, "flops": 30 * T * H}
    if kind == "int8_ffn":
        H, I = case["H"], case["I"]
        return {"bytes": 3 * H * I + 4 * (2 * I + H) + 3 * 2 * T * H, "flops": 6 * T * H * I}
    N, K = case["N"], case["K"]
    return {"bytes": N * K + 4 * N + 2 * T * K + 4 * T * N, "flops": 2 * T * N * K}


# ------------------------------------------------------------------------------------------------ 64-bit results

def _exact_score(x, score):
    if score == SOFTMAX:
        return torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
    if score == SIGMOID:
        return torch.sigmoid(x)
    return torch.sqrt(torch.logaddexp(x, torch.zeros_like(x)))


def _exact_weights(x, ids, c, live):
    got = torch.gather(_exact_score(x, c["score"]), 1, ids.long().clamp(min=0))
    return got * (2.5 / got.sum(1, keepdim=True)) * live[:, None]


def _exact_gate(s, grad):
    c = s["case"]
    x = s["logits"].double().requires_grad_(grad)
    T, E, G = c["T"], c["E"], c["groups"]
    live = torch.ones(T, dtype=torch.float64, device=x.device) if s["mask"] is None else (s["mask"] != 0).double()
    with torch.no_grad():
        key = x.clone() if s["bias"] is None and G == 1 else _exact_score(x, c["score"])
        if s["bias"] is not None:
            key = key + s["bias"].double()
        if G > 1:
            per = E // G
            tops = torch.topk(key.view(T, G, per), min(2, per), dim=2).values.sum(2)
            # a group stays when fewer than top_groups others come before it
            ahead = (tops[:, None, :] > tops[:, :, None]).sum(2)
            order = torch.arange(G, device=x.device)
            ahead += ((tops[:, None, :] == tops[:, :, None]) & (order[None, None, :] < order[None, :, None])).sum(2)
            key = key.masked_fill((ahead >= c["top_groups"]).repeat_interleave(per, 1), -math.inf)
        picked = []
        for _ in range(c["k"]):
            best = (key == key.amax(1, keepdim=True)).to(torch.int8).argmax(1)  # the lowest index among equals
            picked.append(best)
            key = key.scatter(1, best[:, None], -math.inf)
        ids = torch.where(live[:, None] > 0, torch.stack(picked, 1), -1).to(torch.int32)
    w = _exact_weights(x, ids, c, live)
    if not grad:
        return ids, w
    (w * s["d_w"].double()).sum().backward()
    return ids, w.detach(), x.grad


def _exact_balance(s):
    c = s["case"]
    T, E, B, k = c["T"], c["E"], c["B"], c["k"]
    x = s["logits"].double().requires_grad_(True)
    live = torch.ones(T, dtype=torch.bool, device=x.device) if s["mask"] is None else s["mask"] != 0
    q = _exact_score(x, c["score"])
    q = q / q.sum(1, keepdim=True)
    cu = s["cu"].tolist()
    counts = torch.zeros(B, E, dtype=torch.int32, device=x.device)
    terms = []
    for b in range(B):
        on = live[cu[b]:cu[b + 1]]
        n = int(on.sum())
        if n == 0:
            continue
        got = torch.bincount(s["ids"][cu[b]:cu[b + 1]][on].reshape(-1).long(), minlength=E)
        counts[b] = got.to(torch.int32)
        share = q[cu[b]:cu[b + 1]][on].sum(0) / n
        terms.append(E * (got.double() / (n * k) * share).sum())
    if not terms:  # every token is padding
        return torch.zeros(2, device=x.device), counts, torch.zeros_like(x)
    balance = torch.stack(terms).mean()
    z = torch.logsumexp(x, 1)[live].square().mean()
    (balance * s["d_loss"][0].double() + z * s["d_loss"][1].double()).backward()
    return torch.stack([balance, z]).detach(), counts, x.grad


def _exact_rms(v, w):
    return v / torch.sqrt(v.pow(2).mean(1, keepdim=True) + EPS) * w


def _exact_branch(s, x, w_post, gate):
    b = x if w_post is None else _exact_rms(x, w_post)
    return b * s["scale"] if gate is None else b * gate * s["scale"]


def _exact_norm(s):
    d = {n: None if s[n] is None else s[n].double() for n in ("x", "residual", "w_pre", "w_post", "gate")}
    r = d["residual"] + _exact_branch(s, d["x"], d["w_post"], d["gate"])
    return r, _exact_rms(r.to(s["residual"].dtype).double(), d["w_pre"])


def _exact_norm_grad(s):
    d = {n: None if s[n] is None else s[n].double().requires_grad_(True)
         for n in ("x", "residual", "w_pre", "w_post", "gate")}
    (_exact_rms(d["residual"], d["w_pre"]) * s["d_y"].double()).sum().backward()
    d_res = d["residual"].grad + s["d_res"].double()
    (_exact_branch(s, d["x"], d["w_post"], d["gate"]) * d_res).sum().backward()
    out = {"d_x": d["x"].grad, "d_residual": d_res, "d_w_pre": d["w_pre"].grad}
    if s["w_post"] is not None:
        out["d_w_post"] = d["w_post"].grad
    if s["gate"] is not None:
        out["d_gate"] = d["gate"].grad
    return out


def _exact_linear(x, w, w_scale):
    sc = (x.float().abs().amax(1) / 127.0).double()  # the scale itself is a 32-bit number by definition
    q = torch.where(sc[:, None] > 0, torch.round(x.double() / sc[:, None].clamp(min=1e-300)), 0.0)
    return torch.matmul(q, w.double().t()) * sc[:, None] * w_scale.double()[None]


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind in ("gate", "gate_train"):
        return _exact_gate(s, kind == "gate_train")
    if kind == "balance":
        return _exact_balance(s)
    if kind == "norm":
        return _exact_norm(s)
    if kind == "norm_backward":
        return _exact_norm_grad(s)
    if kind == "int8_linear":
        return _exact_linear(s["x"], s["w1"], s["w1_scale"]) + s["add"].double()
    g, u = _exact_linear(s["x"], s["w1"], s["w1_scale"]).chunk(2, dim=1)
    h = (torch.nn.functional.silu(g) * u).to(torch.bfloat16)
    return _exact_linear(h, s["w2"], s["w2_scale"]) + s["add"].double()
