"""The operators around the LoRA projections in the runs they are used in: a training step of one MLP
block (norm, LoRA MLP, norm + gate + residual, all of it backward, optimizer step of its adapters), and
a served block whose rows belong to different adapters, eager and as a captured graph.

References are float64 on the same bf16 inputs.  Tolerance: max|err| / max|ref| <= 2e-2 per tensor, the
bar of the library's other bf16 chains (a handful of bf16 roundings, each 2^-8)."""
import pytest
import torch

import adapter_mlp_amd as lm

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
TOL = 2e-2


def rnd(g, *shape, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g) * scale + shift).to(BF).cuda()


def close(name, got, ref):
    ref = ref.detach()
    err = float((got.double().cpu() - ref).abs().max() / ref.abs().max())
    assert got.isfinite().all() and err <= TOL, f"{name}: {err:.3g}"


def rms(v, w, eps=1e-6):
    return v / torch.sqrt(v.square().mean(1, keepdim=True) + eps) * (1 + w)


def test_training_step_of_a_block():
    T, H, I, r = 300, 512, 1088, 16
    g = torch.Generator().manual_seed(3)
    R, w_in, w_post, w_next, gate = rnd(g, T, H), *(rnd(g, H, scale=0.1) for _ in range(3)), rnd(g, H, scale=0.2, shift=0.7)

    def proj(n_in, n_out):
        return lm.Proj(A=rnd(g, n_in, r, scale=n_in ** -0.5), B=rnd(g, r, n_out, scale=0.3 * r ** -0.5), scale=2.0,
                       W=rnd(g, n_in, n_out, scale=n_in ** -0.5))

    p = dict(gate=proj(H, I), up=proj(H, I), down=proj(I, H))
    kw = dict(unit_offset=True)
    block = dict(w_pre=w_next, w_post=w_post, gate=gate, res_scale=0.9, **kw)
    d_res, d_next = rnd(g, T, H), rnd(g, T, H)

    _, X = lm.block_norm_fwd(R, w_pre=w_in, **kw)
    Y, saved = lm.mlp_fwd(X, *p.values(), "swiglu")
    R2, X2 = lm.block_norm_fwd(R, Y, **block)
    dR2, dY, block_grads = lm.block_norm_bwd(d_res, d_next, R2, Y, **block)
    dX, grads = lm.mlp_bwd(dY, X, saved, *p.values(), "swiglu")
    dR, _, in_grads = lm.block_norm_bwd(dR2, dX, R, w_pre=w_in, **kw)

    leaf = {}

    def ref(name, t):
        leaf[name] = t.double().cpu().requires_grad_()
        return leaf[name]

    def z(name, x):
        q = p[name]
        return x @ q.W.double().cpu() + q.scale * (x @ ref("dA_" + name, q.A)) @ ref("dB_" + name, q.B)

    r64 = ref("R", R)
    x = rms(r64, ref("w_in", w_in))
    y = z("down", torch.nn.functional.silu(z("gate", x)) * z("up", x))
    out = 0.9 * r64 + ref("gate", gate) * rms(y, ref("w_post", w_post))
    nxt = rms(out, ref("w_pre", w_next))
    (out * d_res.double().cpu()).sum().add((nxt * d_next.double().cpu()).sum()).backward()
    close("R2", R2, out)
    close("X2", X2, nxt)
    for name, got in {"R": dR, "w_in": in_grads["w_pre"], **block_grads, **grads}.items():
        close(name, got, leaf[name].grad)

    # the optimizer step: adapters of three projections in two shapes, in one call
    params = [t for q in p.values() for t in (q.A, q.B)]
    update = [grads[f"d{ab}_{name}"] for name in p for ab in "AB"]
    moms = [torch.zeros(t.shape, device="cuda") for t in params]
    before = [t.double().cpu() for t in params]
    lm.muon_step(params, update, moms, lr=0.05, momentum=0.9, weight_decay=0.1, scale=1.0)
    for was, t, d, m in zip(before, params, update, moms):
        assert torch.equal(m, d.float())
        u = (d.float() + torch.tensor(0.9) .cuda() * d.float()).double().cpu()
        left, s, right = torch.linalg.svd(u, full_matrices=False)
        s = s / (s.norm() + 1e-7)
        for _ in range(5):
            a, b, c = lm.NS_COEFFS
            s = a * s + b * s ** 3 + c * s ** 5
        close("param", t, 0.995 * was - 0.05 * (left * s) @ right)
        assert not torch.equal(t.double().cpu(), was)
    Y2, _ = lm.mlp_fwd(X, *p.values(), "swiglu")  # the projections see the new adapters
    assert not torch.equal(Y2, Y)


def served(T, seed=0):
    H, I, r, n = 512, 1088, 16, 6
    g = torch.Generator().manual_seed(seed)
    s = dict(R=rnd(g, T, H), w=[rnd(g, H, scale=0.1) for _ in range(3)],
             ids=torch.randint(-1, n, (T,), generator=g, dtype=torch.int32).cuda())
    for name, n_in, n_out in (("v", H, H), ("o", H, H), ("gate", H, I), ("up", H, I), ("down", I, H)):
        s[name] = (rnd(g, n_in, n_out, scale=n_in ** -0.5),
                   lm.AdapterPool(A=rnd(g, n, n_in, r, scale=n_in ** -0.5), B=rnd(g, n, r, n_out, scale=0.5 * r ** -0.5),
                                  scale=(torch.rand(n, generator=g) + 0.5).cuda()))
    return s


def run_served(s):
    """One block for one position of each row (attention over itself alone is its value)."""
    def z(name, x):
        return lm.multi_fwd(x, s[name][0], s[name][1], s["ids"])

    kw = dict(unit_offset=True)
    _, x = lm.block_norm_fwd(s["R"], w_pre=s["w"][0], **kw)
    r, x = lm.block_norm_fwd(s["R"], z("o", z("v", x)), w_pre=s["w"][1], **kw)
    h = torch.nn.functional.silu(z("gate", x)) * z("up", x)
    return lm.block_norm_fwd(r, z("down", h), w_pre=s["w"][2], **kw)


def ref_served(s):
    def z(name, x):
        W, p = s[name]
        y = x @ W.double().cpu()
        for i in range(p.A.shape[0]):
            m = (s["ids"] == i).cpu()
            y[m] += float(p.scale[i]) * (x[m] @ p.A[i].double().cpu()) @ p.B[i].double().cpu()
        return y

    w = [t.double().cpu() for t in s["w"]]
    r = s["R"].double().cpu()
    r = r + z("o", z("v", rms(r, w[0])))
    x = rms(r, w[1])
    r = r + z("down", torch.nn.functional.silu(z("gate", x)) * z("up", x))
    return r, rms(r, w[2])


@pytest.mark.parametrize("T", [1, 9, 150, 1300])
def test_served_block(T):
    s = served(T)
    got, want = run_served(s), ref_served(s)
    close("R", got[0], want[0])
    close("X", got[1], want[1])


@pytest.mark.parametrize("T", [3, 200])
def test_served_block_as_a_graph(T):
    s = served(T)
    run_served(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run_served(s)
    for seed in (4, 5, 6):
        q = served(T, seed)
        s["R"].copy_(q["R"])
        s["ids"].copy_(q["ids"])
        graph.replay()
        torch.cuda.synchronize()
        eager = run_served(s)
        assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])
    close("R", out[0], ref_served(s)[0])


def test_two_calls_at_once_on_two_streams():
    a, b = served(300, 1), served(40, 2)
    want = run_served(a) + run_served(b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        got = []
        for s, q in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got += run_served(q)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
