"""Orthogonalised updates (orthogonalize / muon_step) against singular values in float64, and the
calls they refuse.

The steps map each singular value s -> a s + b s^3 + c s^5 and keep the singular vectors, so the
reference works on an SVD.  The kernels work in float64: a result is off by half a step of its type
relative to the value, and by what float64 leaves of the steps (each grows a small direction by a;
a^steps 2^-53 stays far below the 1e-9 allowed here, entries being at most about 1.2).  muon_step rounds U to
fp32 first; the reference rounds the same way, from the momentum that the call wrote.  Its sum is formed in
float64 and rounded, the kernel's is one fma: they may differ by one rounding, 2^-23 of an element, which
the steps grow by at most a^5 = 485 over the norm."""
import ctypes

import pytest
import torch

import adapter_mlp_amd as lm
from adapter_mlp_amd import _lib as L

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rnd(shape, dtype=torch.float32, seed=0, scale=1e-2, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g, dtype=torch.float64)
    fall = torch.exp(-4.0 * torch.arange(shape[-1], dtype=torch.float64) / shape[-1])  # unequal singular values
    return (x * fall * scale).to(dtype).to(device)


def ns64(u, steps=5, coeffs=lm.NS_COEFFS, eps=1e-7):
    a, b, c = coeffs
    left, s, right = torch.linalg.svd(u.double().cpu(), full_matrices=False)
    s = s / (s.square().sum(-1, keepdim=True).sqrt() + eps)
    for _ in range(steps):
        s = a * s + b * s ** 3 + c * s ** 5
    return left @ (s.unsqueeze(-1) * right)


def check(name, got, ref, slack=0.0):
    assert got.shape == ref.shape, name
    err = (got.double().cpu() - ref).abs()
    bound = HALF[got.dtype] * ref.abs() * (1 + 2.0 ** -7) + 1e-9 + slack
    bad = err > bound
    assert not bad.any(), f"{name}: off by {err[bad].max():.3g} at {int(bad.sum())} of {err.numel()}, bound {bound[bad].min():.3g}"


SHAPES = [(1, 1), (7, 1), (1, 1030), (5, 3), (2, 9), (16, 16), (64, 64), (100, 8), (8, 515), (511, 16), (16, 513), (1024, 17),
          (23, 777), (600, 24), (32, 512), (2049, 33), (40, 1537), (48, 640), (1100, 63), (64, 1025), (4096, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_orthogonalize(rows, cols, dtype):
    G = rnd((3, rows, cols), DT[dtype], seed=rows + cols)
    check("stack", lm.orthogonalize(G), ns64(G))
    check("matrix", lm.orthogonalize(G[1]), ns64(G[1]))


@pytest.mark.gpu
@pytest.mark.parametrize("steps", [1, 2, 6])
def test_steps_coefficients_eps(steps):
    G = rnd((2, 300, 20))
    kw = dict(steps=steps, coeffs=(1.875, -1.25, 0.375), eps=0.5)
    check("out", lm.orthogonalize(G, **kw), ns64(G, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("rows,cols", [(700, 16), (16, 1025), (1, 40), (530, 40), (64, 1000), (33, 33)])
def test_muon_step(rows, cols, nesterov, dtype):
    kw = dict(lr=0.03, momentum=0.9, weight_decay=0.1, nesterov=nesterov)
    P, M = rnd((2, rows, cols), DT[dtype], 1, scale=0.5), rnd((2, rows, cols), seed=2)
    p, m = P.clone(), M.clone()
    for k in range(2):
        G = rnd((2, rows, cols), DT[dtype], 3 + k)
        was, before = p.double().cpu(), m.double().cpu()
        lm.muon_step(p, G, m, **kw)
        mu = float(torch.tensor(0.9, dtype=torch.float32))
        g = G.double().cpu()
        m64 = mu * before + g
        assert ((m.double().cpu() - m64).abs() <= 2.0 ** -24 * m64.abs() * (1 + 2.0 ** -20)).all()
        now = m.double().cpu()
        u = (mu * now + g).float() if nesterov else now.float()
        scale = max(1.0, cols / rows) ** 0.5
        scale = float(torch.tensor(scale, dtype=torch.float32))
        want = (1 - 0.03 * 0.1) * was - 0.03 * scale * ns64(u)
        slack = 0.03 * scale * 485 * 2.0 ** -23 * float((u.abs().amax((1, 2)) / u.square().sum((1, 2)).sqrt()).max())
        check("P", p, want, slack)


@pytest.mark.gpu
def test_a_list_of_many_shapes():
    mats = [rnd((1 + i % 3, *((40 + 31 * i, 1 + 2 * i) if i % 2 else (1 + 2 * i, 40 + 31 * i))), seed=i) for i in range(32)]
    mats += [rnd((50 + i, 8), seed=i) for i in range(30)]  # more of one class than a launch takes
    for got, G in zip(lm.orthogonalize(mats), mats):
        check(str(tuple(G.shape)), got, ns64(G))


@pytest.mark.gpu
def test_zero_deficient_extreme_and_bad_matrices():
    G = rnd((6, 500, 16))
    G[0] = 0
    G[1, :, 3] = G[1, :, 4]   # a singular value of zero
    G[2, :, 1:] = 0           # rank one
    G[3] *= 1e-30
    G[4] *= 1e30
    G[5, 17, 2] = float("nan")
    out = lm.orthogonalize(G, eps=1e-40)
    assert not out[0].any()
    check("rest", out[1:5], ns64(G[1:5], eps=1e-40))
    assert out[5].isnan().all()
    check("eps", lm.orthogonalize(G[:5]), torch.cat([torch.zeros(1, 500, 16).double(), ns64(G[1:5])]))


# The most steps that each set of coefficients is taken to: |a|^steps <= 2^22.
MOST = [(12, lm.NS_COEFFS), (22, (2.0, -1.5, 0.5)), (24, (1.875, -1.25, 0.375)), (32, (1.5, -0.5, 0.0))]


@pytest.mark.gpu
@pytest.mark.parametrize("r", [16, 20, 40, 64])
@pytest.mark.parametrize("steps,coeffs", MOST)
def test_deficient_matrices_at_the_most_steps(steps, coeffs, r):
    """Gradients of fewer tokens than the rank: no singular value where rounding leaves 2^-53 in the Gram
    matrix, which each step multiplies by a^2.  An entry may be off by that."""
    g = torch.Generator().manual_seed(r)
    G = rnd((4, 700, r), device="cpu")
    G[0, :, r // 2] = G[0, :, r // 2 - 1]
    G[1] = torch.randint(-8, 9, (700, 1), generator=g) * torch.arange(1, r + 1)  # rank 1, exact in fp32
    G[2] = (torch.randint(-8, 9, (700, 3), generator=g) @ torch.randint(-8, 9, (3, r), generator=g)).float()
    G = G.cuda()
    slack = 2.0 ** -53 * coeffs[0] ** (2 * steps)
    for mats in (G, G.transpose(1, 2).contiguous()):
        check("deficient", lm.orthogonalize(mats, steps=steps, coeffs=coeffs), ns64(mats, steps, coeffs), slack)


@pytest.mark.gpu
@pytest.mark.parametrize("r", [4, 20, 40, 64])
def test_zeros_without_eps(r):
    G = rnd((2, 300, r))
    G[0] = 0
    out = lm.orthogonalize(G, eps=0.0)
    assert not out[0].any()
    check("rest", out[1:], ns64(G[1:], eps=0.0))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(3, 900, 24), (3, 24, 900)])
def test_in_place_other_stream_same_answer(shape):
    G = rnd(shape, torch.bfloat16)
    want = lm.orthogonalize(G)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side_out = lm.orthogonalize(G, stream=side)
    side.synchronize()
    assert torch.equal(side_out, want) and torch.equal(lm.orthogonalize(G), want)
    assert lm.orthogonalize(G, out=G) is G and torch.equal(G, want)


@pytest.mark.gpu
def test_unaligned_views():
    flat = rnd((1 + 2 * 600 * 17,), torch.bfloat16)
    G = flat[1:].view(2, 600, 17)
    check("tall", lm.orthogonalize(G), ns64(G))
    G = flat[1:].view(2, 17, 600)
    check("wide", lm.orthogonalize(G), ns64(G))


@pytest.mark.gpu
def test_captured_graph_replays():
    shapes = [(2, 300, 16), (3, 32, 700)]
    P, M, G = ([rnd(s, seed=10 * k + i) for i, s in enumerate(shapes)] for k in range(3))
    kw = dict(lr=0.01, weight_decay=0.1)
    p, m = [x.clone() for x in P], [x.clone() for x in M]
    ws = torch.empty(lm.orth_workspace_size(G), dtype=torch.uint8, device="cuda")
    lm.muon_step(p, G, m, ws=ws, **kw)  # loads the kernels
    for x, y in zip(p + m, P + M):
        x.copy_(y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lm.muon_step(p, G, m, ws=ws, **kw)
    for k in range(3):
        for i, x in enumerate(G):
            x.copy_(rnd(shapes[i], seed=100 + 7 * k + i))
        lm.muon_step(P, G, M, **kw)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(p + m, P + M))
        torch.zeros(1 << 20, device="cuda").sum().item()


@pytest.mark.gpu
def test_past_32_bit_offsets():
    G = torch.zeros(2050, 16384, 64, dtype=torch.bfloat16, device="cuda")
    assert G.numel() > 1 << 31
    G[-1] = rnd((16384, 64), torch.bfloat16)
    lm.orthogonalize(G, out=G)
    check("last", G[-1], ns64(rnd((16384, 64), torch.bfloat16)))
    assert not G[:-1].any()


@pytest.mark.gpu
def test_many_small_matrices():
    """More matrices than one launch of the steps takes."""
    G = [rnd((1000, 20, 1), torch.bfloat16, seed=k).repeat(3000, 1, 1) for k in range(2)]
    for got, want in zip(lm.orthogonalize(G), [lm.orthogonalize(g[:1000]) for g in G]):
        assert torch.equal(got.view(3000, 1000, 20, 1), want.expand(3000, 1000, 20, 1))


@pytest.mark.gpu
def test_nothing_to_do():
    assert lm.orthogonalize([]) == []
    lm.muon_step([], [], [], lr=0.1)
    assert lm.orthogonalize(torch.zeros(0, 100, 8, device="cuda")).shape == (0, 100, 8)


# ---- refusals (no GPU) ----

def test_binding_refuses():
    G, M = rnd((2, 30, 8), device="cpu"), rnd((2, 30, 8), device="cpu")
    with pytest.raises(ValueError, match="GPU only"):
        lm.orthogonalize(G)
    with pytest.raises(ValueError, match="GPU only"):
        lm.muon_step(G.clone(), G, M, lr=0.1)

    def bad(fn, *args, **kw):
        with pytest.raises(ValueError) as e:
            fn(*args, **kw)
        assert "GPU only" not in str(e.value)

    bad(lm.orthogonalize, G.half())
    bad(lm.orthogonalize, G.transpose(1, 2))
    bad(lm.orthogonalize, G[0, 0])
    bad(lm.orthogonalize, [G, G.bfloat16()])
    bad(lm.orthogonalize, G, out=G[:1])
    bad(lm.orthogonalize, [G, G], out=[G])
    bad(lm.muon_step, G, G, M.bfloat16(), lr=0.1)
    bad(lm.muon_step, G, G.bfloat16(), M, lr=0.1)
    bad(lm.muon_step, [G, G], [G], [M], lr=0.1)
    bad(lm.muon_step, [G], [G], [M], lr=0.1, scale=[1.0, 2.0])


@pytest.mark.parametrize("steps,coeffs", [m for m in MOST if m[0] < 32] + [(1, (2.0 ** 22, 0.0, 0.0)), (2, (-2.0 ** 11, 0.0, 0.0))])
def test_refuses_steps_that_grow_rounding_errors(steps, coeffs):
    mat = L.lora_orth_mat(1 << 20, None, 2 << 20, 1, 100, 8, 1.0, 0)
    size = ctypes.c_size_t()
    for k, want in ((steps, L.LORA_OK), (steps + 1, L.LORA_EINVAL), (32, L.LORA_EINVAL)):
        d = L.lora_orth_desc(1, k, *coeffs, 1e-7, L.LORA_F32, 0)
        assert L.load().lora_orth_workspace_size(ctypes.byref(d), ctypes.byref(mat), ctypes.byref(size)) == want
    muon = L.lora_muon_desc(L.lora_orth_desc(1, steps + 1, *coeffs, 1e-7, L.LORA_F32, 0), 0.1, 0.9, 0.0, 1, 0)
    mat.M = 3 << 20
    assert L.load().lora_muon_step(ctypes.byref(muon), ctypes.byref(mat), 1 << 30, 1 << 40, None) == L.LORA_EINVAL
    assert L.load().lora_orthogonalize(ctypes.byref(muon.orth), ctypes.byref(mat), 1 << 30, 1 << 40, None) == L.LORA_EINVAL


def test_library_refuses():
    """Refused on the host; no address here is read."""
    def call(muon=False, mats=((1, 2, 0, 1, 100, 8, 1.0, 0),), steps=5, a=1.0, eps=1e-7, dtype=L.LORA_F32, n=None, lr=0.1,
             wd=0.0, nest=1, ws=1 << 30, nbytes=1 << 40):
        table = (L.lora_orth_mat * max(1, len(mats)))()
        for m, (G, P, M, count, rows, cols, scale, rsv) in zip(table, mats):
            m.G, m.P, m.M = (x << 20 if isinstance(x, int) and x else (x or None) for x in (G, P, M))
            m.count, m.rows, m.cols, m.scale, m.reserved = count, rows, cols, scale, rsv
        d = L.lora_orth_desc(len(mats) if n is None else n, steps, a, 1.0, 1.0, eps, dtype, 0)
        lib = L.load()
        if muon:
            d = L.lora_muon_desc(d, lr, 0.9, wd, nest, 0)
            return lib.lora_muon_step(ctypes.byref(d), table, ws, nbytes, None)
        return lib.lora_orthogonalize(ctypes.byref(d), table, ws, nbytes, None)

    nan = float("nan")
    mat = (1, 2, 0, 1, 100, 8, 1.0, 0)
    for kw, want in ((dict(steps=0), L.LORA_EINVAL), (dict(steps=33), L.LORA_EINVAL), (dict(a=nan), L.LORA_EINVAL),
                     (dict(eps=-1.0), L.LORA_EINVAL), (dict(dtype=L.LORA_BF16_F32LORA), L.LORA_EDTYPE), (dict(n=-1), L.LORA_EINVAL),
                     (dict(mats=((1, 2, 0, 1, 65, 65, 1.0, 0),)), L.LORA_ESHAPE), (dict(mats=((1, 2, 0, 1, 0, 8, 1.0, 0),)), L.LORA_ESHAPE),
                     (dict(mats=((1, 2, 0, -1, 100, 8, 1.0, 0),)), L.LORA_ESHAPE),
                     (dict(mats=((1, 2, 0, 1 << 40, 100, 8, 1.0, 0),)), L.LORA_ESHAPE),
                     (dict(mats=((1, 2, 0, 1, 1 << 40, 8, 1.0, 0),)), L.LORA_ESHAPE),
                     (dict(mats=((1, 2, 0, (1 << 22) - 1, 33, 33, 1.0, 0),)), L.LORA_ESHAPE),
                     (dict(mats=((1, 2, 0, 1 << 15, 1 << 15, 1, 1.0, 0),)), L.LORA_ESHAPE),
                     (dict(mats=((1, 2, 0, 1, 1, 1 << 30, 1.0, 0),)), L.LORA_ESHAPE),
                     (dict(mats=((1, 2, 0, 1, 100, 8, 1.0, 1),)), L.LORA_EINVAL), (dict(mats=((0, 2, 0, 1, 100, 8, 1.0, 0),)), L.LORA_EINVAL),
                     (dict(mats=((1, 0, 0, 1, 100, 8, 1.0, 0),)), L.LORA_EINVAL), (dict(mats=((1, 2, 3, 1, 100, 8, 1.0, 0),)), L.LORA_EINVAL),
                     (dict(ws=None), L.LORA_EWORKSPACE), (dict(nbytes=1024), L.LORA_EWORKSPACE), (dict(ws=(1 << 30) + 8), L.LORA_EALIGN),
                     (dict(mats=(mat, (3, 2, 0, 1, 100, 8, 1.0, 0))), L.LORA_EUNSUPPORTED),
                     (dict(mats=(mat, (2, 4, 0, 1, 100, 8, 1.0, 0))), L.LORA_EUNSUPPORTED),
                     (dict(mats=(mat, (1, 1, 0, 1, 100, 8, 1.0, 0))), L.LORA_EUNSUPPORTED),
                     (dict(ws=1 << 20), L.LORA_EUNSUPPORTED), (dict(ws=(1 << 20) - 1024), L.LORA_EUNSUPPORTED),
                     (dict(muon=True), L.LORA_EINVAL), (dict(muon=True, mats=((1, 1, 3, 1, 100, 8, 1.0, 0),)), L.LORA_EUNSUPPORTED),
                     (dict(muon=True, mats=((1, 2, 1, 1, 100, 8, 1.0, 0),)), L.LORA_EUNSUPPORTED),
                     (dict(muon=True, mats=((1, 2, 2, 1, 100, 8, 1.0, 0),)), L.LORA_EUNSUPPORTED),
                     (dict(muon=True, mats=((1, 2, 3, 1, 100, 8, nan, 0),)), L.LORA_EINVAL),
                     (dict(muon=True, mats=((1, 2, 3, 1, 100, 8, 1.0, 0),), lr=nan), L.LORA_EINVAL),
                     (dict(muon=True, mats=((1, 2, 3, 1, 100, 8, 1.0, 0),), nest=2), L.LORA_EINVAL)):
        assert call(**kw) == want, kw
    assert L.load().lora_orthogonalize(None, None, None, 0, None) == L.LORA_EINVAL
    assert L.load().lora_muon_step(None, None, None, 0, None) == L.LORA_EINVAL
