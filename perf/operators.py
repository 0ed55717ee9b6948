"""Cases of the operators around the LoRA projections: the projection whose rows belong to
different adapters (``multi_fwd``), the norms before and after a block with its gate and
residual scale (``block_norm_fwd`` / ``block_norm_bwd``) and the orthogonalised adapter
update (``orthogonalize`` / ``muon_step``).

With ``own`` false ``run`` computes the plain form in elementary torch operations; with
``own`` true it calls the package.  ``exact`` is the operator's definition in float64.
"""
import math

import torch

own = False

# widths of the Llama-3-8B block that the library's benchmark runs on
H8, I8, KV8 = 4096, 14336, 1024


def _layer_mats(r):
    """The adapters of one Llama-3-8B layer, by shape: (count, rows, cols)."""
    return [(6, H8, r), (1, I8, r), (3, r, H8), (2, r, KV8), (2, r, I8)]


def _text(groups):
    return ";".join("%dx%dx%d" % g for g in groups)


def _groups(case):
    return [tuple(int(v) for v in g.split("x")) for g in case["mats"].split(";")]


def listed():
    return [
        # one user's next token through q or o, its adapter among the few that are loaded
        dict(name="multi_decode_1", op="multi", dtype="bf16", T=1, K=H8, N=H8, r=16, n=8, rows="mixed", none=0.0),
        # a decode batch through the gate projection: a token of each of 67 requests, many
        # adapters, some requests on the base model
        dict(name="multi_decode_67", op="multi", dtype="bf16", T=67, K=H8, N=I8, r=16, n=32, rows="mixed", none=0.1),
        # a mixed batch through the down projection: chunks of prompts, rank 64
        dict(name="multi_chunks_777", op="multi", dtype="bf16", T=777, K=I8, N=H8, r=64, n=12, rows="runs", none=0.1),
        # a full prefill batch through q or o: long prompts of several users
        dict(name="multi_prefill_8192", op="multi", dtype="bf16", T=8192, K=H8, N=H8, r=16, n=16, rows="runs", none=0.1),
        # the small fp32 configuration, each row another adapter
        dict(name="multi_f32_128", op="multi", dtype="f32", T=128, K=256, N=704, r=8, n=5, rows="mixed", none=0.1),
        # residual add and the next block's norm for one token
        dict(name="norm_fwd_decode_1", op="norm_fwd", dtype="bf16", params="bf16", T=1, H=H8, post=False, gate="none", pre=True),
        # post-norm, learned gate, residual and the next pre-norm of a training batch
        dict(name="norm_fwd_8192", op="norm_fwd", dtype="bf16", params="bf16", T=8192, H=H8, post=True, gate="col", pre=True),
        # its backward pass
        dict(name="norm_bwd_8192", op="norm_bwd", dtype="bf16", params="bf16", T=8192, H=H8, post=True, gate="col", pre=True),
        # odd sizes in fp32, one gate value a token
        dict(name="norm_bwd_f32_1003", op="norm_bwd", dtype="f32", params="f32", T=1003, H=1001, post=True, gate="row", pre=True),
        # orthogonalised gradients of one layer's rank-16 adapters
        dict(name="orth_layer_r16", op="orth", dtype="bf16", mats=_text(_layer_mats(16)), nesterov=False),
        # the optimizer step of a whole rank-16 fine-tune: 32 layers, 448 adapter matrices
        dict(name="muon_model_r16", op="muon", dtype="f32", mats=_text([(32 * c, a, b) for c, a, b in _layer_mats(16)]), nesterov=True),
        # the optimizer step of one layer at the largest rank
        dict(name="muon_layer_r64", op="muon", dtype="f32", mats=_text(_layer_mats(64)), nesterov=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["multi", "multi", "norm_fwd", "norm_bwd", "orth", "muon"])
    if op == "multi":
        rows, none = rng.choice(["mixed", "runs"]), rng.choice([0.0, 0.1, 0.4])
        if rng.random() < 0.25:
            return dict(op=op, dtype="f32", T=_log(rng, 1, 700), K=_log(rng, 33, 1500), N=_log(rng, 33, 1500),
                        r=rng.randint(1, 64), n=_log(rng, 1, 40), rows=rows, none=none)
        return dict(op=op, dtype="bf16", T=_log(rng, 1, 4096), K=64 * _log(rng, 2, 112), N=64 * _log(rng, 2, 112),
                    r=8 * rng.randint(1, 8), n=_log(rng, 1, 64), rows=rows, none=none)
    if op in ("norm_fwd", "norm_bwd"):
        f32 = rng.random() < 0.3
        return dict(op=op, dtype="f32" if f32 else "bf16", params="f32" if f32 else rng.choice(["bf16", "f32"]),
                    T=_log(rng, 1, 8192), H=_log(rng, 30, 4000) if f32 else 64 * _log(rng, 1, 96),
                    post=rng.random() < 0.6, gate=rng.choice(["none", "col", "row", "elem"]), pre=rng.random() < 0.8)
    groups = []
    for _ in range(rng.randint(1, 5)):
        r, long = rng.choice([rng.randint(1, 64), 8, 16, 32]), _log(rng, 64, 12000)
        groups.append((_log(rng, 1, 24),) + rng.choice([(long, r), (r, long)]))
    return dict(op=op, dtype=rng.choice(["bf16", "f32"]), mats=_text(groups), nesterov=rng.random() < 0.7)


_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ALPHA = 32.0
NORM = dict(res_scale=1.0, branch_scale=0.75, eps=1e-6, unit_offset=True)
MUON = dict(lr=0.02, momentum=0.95, weight_decay=0.01)
COEFFS, EPS, STEPS = (3.4445, -4.7750, 2.0315), 1e-7, 5


class _Gen:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, shape, dtype, scale=1.0, shift=0.0):
        return torch.randn(shape, generator=self.g, device="cuda").mul_(scale).add_(shift).to(dtype)

    def uniform(self, shape):
        return torch.rand(shape, generator=self.g, device="cuda")


def _ids(g, case):
    """The adapter of each row, -1 for the base model alone: "mixed" draws every row by itself,
    "runs" gives each of about n requests a run of rows."""
    T, n = case["T"], case["n"]
    owner = torch.arange(T, device="cuda")
    if case["rows"] == "runs":
        cuts = torch.sort((g.uniform((max(1, min(n, T)),)) * T).long()).values
        owner = torch.searchsorted(cuts, owner, right=True)
    pick = (g.uniform((T + 1,)) * n).int().clamp_(max=n - 1)
    pick[g.uniform((T + 1,)) < case["none"]] = -1
    return pick[owner].contiguous()


def _gradients(g, count, rows, cols, dtype):
    """Matrices with a spectrum that falls off, as the gradients of adapters have."""
    r = min(rows, cols)
    q = g.normal((count, max(rows, cols), r), torch.float32, 1.0 / math.sqrt(max(rows, cols)))
    p = g.normal((count, r, r), torch.float32, 1.0 / math.sqrt(r))
    fall = torch.exp(-4.0 * torch.arange(r, device="cuda") / r)
    x = torch.bmm(q * fall, p) * 1e-2
    return (x if rows >= cols else x.transpose(1, 2)).contiguous().to(dtype)


def prepare(case, seed):
    g = _Gen(seed)
    s = dict(case=case, op=case["op"])
    dt = _DT[case["dtype"]]
    if case["op"] == "multi":
        T, K, N, r, n = (case[k] for k in ("T", "K", "N", "r", "n"))
        s["X"] = g.normal((T, K), dt)
        s["W"] = g.normal((K, N), dt, 1.0 / math.sqrt(K))
        s["A"] = g.normal((n, K, r), dt, 1.0 / math.sqrt(K))
        s["B"] = g.normal((n, r, N), dt, 0.5 / math.sqrt(r))
        s["scale"] = g.uniform((n,)) + ALPHA / 32
        s["ids"] = _ids(g, case)
        if own:
            import adapter_mlp_amd as lm

            s["pool"] = lm.AdapterPool(A=s["A"], B=s["B"], scale=s["scale"])
    elif case["op"] in ("norm_fwd", "norm_bwd"):
        T, H = case["T"], case["H"]
        pt = _DT[case["params"]]
        shape = {"none": None, "col": (H,), "row": (T, 1), "elem": (T, H)}[case["gate"]]
        s["R"] = g.normal((T, H), dt, 2.0)
        s["Y"] = g.normal((T, H), dt, 0.5)
        s["par"] = dict(w_pre=g.normal((H,), pt, 0.1) if case["pre"] else None,
                        w_post=g.normal((H,), pt, 0.1) if case["post"] else None,
                        gate=g.normal(shape, pt if case["gate"] == "col" else dt, 0.3, 0.5) if shape else None)
        s["dX"] = g.normal((T, H), dt) if case["pre"] else None
        s["dR"] = g.normal((T, H), dt)
    else:
        s["G"] = [_gradients(g, c, a, b, dt) for c, a, b in _groups(case)]
        if case["op"] == "muon":
            s["M"] = [_gradients(g, c, a, b, torch.float32) for c, a, b in _groups(case)]
            s["P"] = [g.normal((c, a, b), dt, 0.02) for c, a, b in _groups(case)]
            s["scale"] = [math.sqrt(max(1.0, b / a)) for _, a, b in _groups(case)]
    return s


def _multi(s):
    """Y = X W + scale[i] (X A[i]) B[i], i the row's adapter: every row times every adapter, the
    row's own kept, then one product with the stacked B."""
    x, (n, K, r) = s["X"].float(), s["A"].shape
    u = (x @ s["A"].float().permute(1, 0, 2).reshape(K, n * r)).view(-1, n, r)
    mine = s["ids"][:, None] == torch.arange(n, device=x.device, dtype=torch.int32)
    u = u * (mine * s["scale"])[:, :, None]
    y = x @ s["W"].float() + u.view(-1, n * r) @ s["B"].float().view(n * r, -1)
    return y.to(s["X"].dtype)


def _unit(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + NORM["eps"])


def _f(x):
    return None if x is None else x.float()


def _weights(par):
    w_pre, w_post, gate = (_f(par[k]) for k in ("w_pre", "w_post", "gate"))
    one = 1.0 if NORM["unit_offset"] else 0.0
    return None if w_pre is None else w_pre + one, None if w_post is None else w_post + one, 1.0 if gate is None else gate


def _norm_fwd(s):
    w_pre, w_post, gate = _weights(s["par"])
    y = s["Y"].float()
    p = y if w_post is None else y * _unit(y) * w_post
    out = NORM["res_scale"] * s["R"].float() + NORM["branch_scale"] * (gate * p)
    x = None if w_pre is None else (out * _unit(out) * w_pre).to(s["R"].dtype)
    return out.to(s["R"].dtype), x


def _norm_bwd(s):
    """Gradients of the block's output Y and residual R and of the weights, from those of the new
    residual and of its norm; s["R"] is the new residual here."""
    w_pre, w_post, gate = _weights(s["par"])
    dt, par, grads = s["R"].dtype, s["par"], {}
    d = s["dR"].float()
    if w_pre is not None:
        o, dx = s["R"].float(), s["dX"].float()
        u = _unit(o)
        o = o * u
        g = dx * w_pre
        d = d + u * (g - o * (g * o).mean(-1, keepdim=True))
        grads["w_pre"] = (dx * o).sum(0).to(par["w_pre"].dtype)
    y = s["Y"].float()
    v = None if w_post is None else _unit(y)
    yn = y if v is None else y * v
    p = yn if v is None else yn * w_post
    db = NORM["branch_scale"] * d
    if par["gate"] is not None:
        grads["gate"] = (db * p).sum_to_size(par["gate"].shape).to(par["gate"].dtype)
    dp = db * gate
    if v is not None:
        grads["w_post"] = (dp * yn).sum(0).to(par["w_post"].dtype)
        g = dp * w_post
        dp = v * (g - yn * (g * yn).mean(-1, keepdim=True))
    return (NORM["res_scale"] * d).to(dt), dp.to(dt), grads


def _newton_schulz(u):
    """STEPS steps of X <- a X + (b S + c S S) X, S = X X^T, on the short side, from U over its norm."""
    tall = u.shape[1] > u.shape[2]
    x = u.float().transpose(1, 2).contiguous() if tall else u.float()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    a, b, c = COEFFS
    for _ in range(STEPS):
        S = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * S + c * torch.bmm(S, S), x)
    return x.transpose(1, 2) if tall else x


def _muon(s, i):
    P, G, M, mu = s["P"][i], s["G"][i].float(), s["M"][i], MUON["momentum"]
    M.mul_(mu).add_(G)
    o = _newton_schulz(G + mu * M if s["case"]["nesterov"] else M)
    P.copy_(P.float() * (1.0 - MUON["lr"] * MUON["weight_decay"]) - MUON["lr"] * s["scale"][i] * o)
    return P, M


def run(s):
    op = s["op"]
    if own:
        import adapter_mlp_amd as lm

        if op == "multi":
            return lm.multi_fwd(s["X"], s["W"], s["pool"], s["ids"])
        if op == "norm_fwd":
            return lm.block_norm_fwd(s["R"], s["Y"], **s["par"], **NORM)
        if op == "norm_bwd":
            return lm.block_norm_bwd(s["dR"], s["dX"], s["R"], s["Y"], **s["par"], **NORM)
        if op == "orth":
            return lm.orthogonalize(s["G"], steps=STEPS, coeffs=COEFFS, eps=EPS)
        lm.muon_step(s["P"], s["G"], s["M"], scale=s["scale"], nesterov=s["case"]["nesterov"], steps=STEPS, coeffs=COEFFS,
                     eps=EPS, **MUON)
        return s["P"], s["M"]
    if op == "multi":
        return _multi(s)
    if op == "norm_fwd":
        return _norm_fwd(s)
    if op == "norm_bwd":
        return _norm_bwd(s)
    if op == "orth":
        return [_newton_schulz(G).to(G.dtype) for G in s["G"]]
    both = [_muon(s, i) for i in range(len(s["G"]))]
    return [p for p, _ in both], [m for _, m in both]


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "multi":
        T, K, N, r = (case[k] for k in ("T", "K", "N", "r"))
        used = min(case["n"], T)
        return {"bytes": es * (T * K + K * N + used * r * (K + N) + T * N) + 4 * T, "flops": 2 * T * K * N + 2 * T * r * (K + N)}
    if case["op"] in ("norm_fwd", "norm_bwd"):
        T, H = case["T"], case["H"]
        pre, post, gate = int(case["pre"]), int(case["post"]), case["gate"]
        gb = {"none": 0, "col": H, "row": T, "elem": T * H}[gate] * es
        pb = (pre + post) * H * (4 if case["params"] == "f32" else 2)
        if case["op"] == "norm_fwd":
            return {"bytes": es * T * H * (3 + pre) + gb + pb, "flops": T * H * (3 + 4 * pre + 4 * post)}
        reads = 1 + 2 * pre + (1 if gate != "none" or post else 0)
        return {"bytes": es * T * H * (reads + 2) + 2 * (gb + pb), "flops": T * H * (3 + 10 * pre + 10 * post)}
    total = sum(c * a * b for c, a, b in _groups(case))
    products = sum(4 * c * a * b * min(a, b) for c, a, b in _groups(case))
    if case["op"] == "orth":
        return {"bytes": 2 * es * total, "flops": products}
    return {"bytes": (3 * es + 8) * total, "flops": products + 8 * total}


def _exact_multi(s):
    y = torch.matmul(s["X"].double(), s["W"].double())
    for i in range(s["case"]["n"]):
        rows = torch.nonzero(s["ids"] == i).flatten()
        low = torch.matmul(s["X"][rows].double(), s["A"][i].double())
        y[rows] += torch.matmul(low, s["B"][i].double()) * float(s["scale"][i])
    return y


def _exact_norm(s):
    """The forward in float64, differentiated by torch for the backward case."""
    case, off = s["case"], 1.0 if NORM["unit_offset"] else 0.0
    par = {k: None if v is None else v.double().requires_grad_() for k, v in s["par"].items()}
    y = s["Y"].double().requires_grad_()
    r = s["R"].double().requires_grad_()

    def rms(v, w):
        return v / torch.sqrt(torch.mean(v * v, dim=1, keepdim=True) + NORM["eps"]) * (off + w)

    branch = NORM["branch_scale"] * (rms(y, par["w_post"]) if case["post"] else y)
    if par["gate"] is not None:
        branch = branch * par["gate"]
    if case["op"] == "norm_fwd":
        new = NORM["res_scale"] * r + branch
        return new.detach(), rms(new, par["w_pre"]).detach() if case["pre"] else None
    # R is the new residual: its gradient is dR and that of its norm, and goes on to the branch
    top = s["dR"].double()
    grads = {}
    if case["pre"]:
        got = torch.autograd.grad(rms(r, par["w_pre"]), [r, par["w_pre"]], s["dX"].double())
        top, grads["w_pre"] = top + got[0], got[1]
    names = [k for k in ("gate", "w_post") if par[k] is not None]
    got = torch.autograd.grad(branch, [y] + [par[k] for k in names], top)
    grads.update(zip(names, got[1:]))
    return NORM["res_scale"] * top, got[0], grads


def _exact_orth(u):
    """By singular values: the steps map each, s -> a s + b s^3 + c s^5, and keep its vectors."""
    v = u.double()
    long = v if v.shape[1] >= v.shape[2] else v.transpose(1, 2)
    q, t = torch.linalg.qr(long.cpu())
    left, sv, right = torch.linalg.svd(t)
    sv = sv / (torch.linalg.vector_norm(sv, dim=1, keepdim=True) + EPS)
    for _ in range(STEPS):
        sv = COEFFS[0] * sv + COEFFS[1] * sv ** 3 + COEFFS[2] * sv ** 5
    res = torch.matmul(q, torch.matmul(left * sv[:, None, :], right)).to(u.device)
    return res if v.shape[1] >= v.shape[2] else res.transpose(1, 2).contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "multi":
        return _exact_multi(s)
    if case["op"] in ("norm_fwd", "norm_bwd"):
        return _exact_norm(s)
    if case["op"] == "orth":
        return [_exact_orth(G) for G in s["G"]]
    new_p, new_m = [], []
    for P, G, M, scale in zip(s["P"], s["G"], s["M"], s["scale"]):
        m = MUON["momentum"] * M.double() + G.double()
        u = G.double() + MUON["momentum"] * m if case["nesterov"] else m
        new_p.append((1 - MUON["lr"] * MUON["weight_decay"]) * P.double() - MUON["lr"] * scale * _exact_orth(u))
        new_m.append(m)
    return new_p, new_m
