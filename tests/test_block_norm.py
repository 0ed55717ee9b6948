"""Norms around a block (block_norm_fwd / block_norm_bwd) against their formulas in float64,
against differences of the forward, and the calls they refuse.

Tolerances, per element: half a step of the output's type relative to the value, and
C * 2^-24 times the magnitude that the fp32 arithmetic handles (the same formula with
absolute values of its terms).  C = 64 covers the row sums (at most 16 products a thread,
6 + 16 additions across threads), the root and some ten products; the column sums of the
parameter gradients add their terms one by one in runs of at most T / blocks rows."""
import ctypes

import pytest
import torch

import adapter_mlp_amd as lm
from adapter_mlp_amd import _lib as L

C32 = 64 * 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(T, H, mode, gate, post, pre, seed=0, device="cuda"):
    """mode: bf16, f32 or bf16_f32 (fp32 parameters)."""
    g = torch.Generator().manual_seed(seed)
    at, pt = DT[mode.split("_")[0]], DT[mode.split("_")[-1]]

    def rnd(shape, dtype, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=g) * scale + shift).to(dtype).to(device)

    shape = {"none": None, "col": (H,), "row": (T, 1), "elem": (T, H)}[gate]
    s = dict(R=rnd((T, H), at, 2.0), Y=rnd((T, H), at, 0.7), dR=rnd((T, H), at), dX=rnd((T, H), at) if pre else None)
    s["par"] = dict(w_pre=rnd((H,), pt, 0.2, 0.1) if pre else None, w_post=rnd((H,), pt, 0.2, 0.3) if post else None,
                    gate=None if shape is None else rnd(shape, pt if gate == "col" else at, 0.5, 0.2))
    s["kw"] = dict(res_scale=0.9, branch_scale=1.3, eps=1e-5, unit_offset=True)
    return s


def d64(t):
    return None if t is None else t.double().cpu()


def ref_fwd(s):
    """(values, magnitudes) of R_out and X."""
    kw, par = s["kw"], {k: d64(v) for k, v in s["par"].items()}
    off = 1.0 if kw["unit_offset"] else 0.0
    p = d64(s["Y"])
    if par["w_post"] is not None:
        p = p * (p.square().mean(1, keepdim=True) + kw["eps"]).rsqrt() * (off + par["w_post"])
    if par["gate"] is not None:
        p = p * par["gate"]
    r = kw["res_scale"] * d64(s["R"])
    p = kw["branch_scale"] * p
    out, mag = r + p, r.abs() + p.abs()
    if par["w_pre"] is None:
        return [(out, mag)]
    f = (out.square().mean(1, keepdim=True) + kw["eps"]).rsqrt() * (off + par["w_pre"])
    return [(out, mag), (out * f, mag * f.abs())]


def ref_bwd(s):
    """{name: (value, magnitude)} of the gradients; s["R"] is the forward's R_out."""
    kw, par = s["kw"], {k: d64(v) for k, v in s["par"].items()}
    off = 1.0 if kw["unit_offset"] else 0.0
    H, res = s["R"].shape[1], {}
    d = d64(s["dR"])
    mag = d.abs()
    if par["w_pre"] is not None:
        o, dx = d64(s["R"]), d64(s["dX"])
        u = (o.square().mean(1, keepdim=True) + kw["eps"]).rsqrt()
        q, n = dx * (off + par["w_pre"]), o * u
        d = d + u * (q - n * (q * n).mean(1, keepdim=True))
        mag = mag + u * (q.abs() + n.abs() * (q * n).abs().mean(1, keepdim=True))
        res["w_pre"] = ((dx * n).sum(0), (dx * n).abs().sum(0))
    res["dR"] = (kw["res_scale"] * d, abs(kw["res_scale"]) * mag)
    y = d64(s["Y"])
    v = (y.square().mean(1, keepdim=True) + kw["eps"]).rsqrt() if par["w_post"] is not None else torch.ones(y.shape[0], 1).double()
    w = off + par["w_post"] if par["w_post"] is not None else torch.ones(H).double()
    yn = y * v
    b, g = kw["branch_scale"], par["gate"] if par["gate"] is not None else torch.ones(1).double()
    if par["gate"] is not None:
        dg, mg = b * d * yn * w, b * mag * (yn * w).abs()
        dims = 0 if g.dim() == 1 else 1
        one = g.shape == dg.shape
        res["gate"] = (dg, mg) if one else (dg.sum(dims, keepdim=g.dim() == 2), mg.sum(dims, keepdim=g.dim() == 2))
    e, me = b * g * d, (b * g).abs() * mag
    if par["w_post"] is not None:
        res["w_post"] = ((e * yn).sum(0), (me * yn.abs()).sum(0))
        z, mz = e * w, me * w.abs()
        res["dY"] = (v * (z - yn * (z * yn).mean(1, keepdim=True)), v * (mz + yn.abs() * (mz * yn.abs()).mean(1, keepdim=True)))
    else:
        res["dY"] = (e, me)
    return res


def check(name, got, ref, mag):
    assert tuple(got.shape) == tuple(ref.shape), name
    err = (got.double().cpu() - ref).abs()
    bound = HALF[got.dtype] * ref.abs() * (1 + 2.0 ** -7) + C32 * mag
    bad = err > bound
    assert not bad.any(), f"{name}: off by {err[bad].max():.3g} at {int(bad.sum())} of {err.numel()}, bound {bound[bad].min():.3g}"


def run_fwd(s, **kw):
    return lm.block_norm_fwd(s["R"], s["Y"], **s["par"], **s["kw"], **kw)


def run_bwd(s, **kw):
    return lm.block_norm_bwd(s["dR"], s["dX"], s["R"], s["Y"], **s["par"], **s["kw"], **kw)


def check_fwd(s, out):
    ref = ref_fwd(s)
    check("R_out", out[0], *ref[0])
    if len(ref) > 1:
        check("X", out[1], *ref[1])
    else:
        assert out[1] is None


def check_bwd(s, got):
    dR, dY, grads = got
    ref = ref_bwd(s)
    assert set(grads) == {k for k, v in s["par"].items() if v is not None}
    for k, v in {"dR": dR, "dY": dY, **grads}.items():
        check(k, v, *ref[k])


SHAPES = [("bf16", 1, 64), ("bf16", 5, 512), ("bf16", 303, 576), ("bf16", 67, 1088), ("bf16", 1030, 2048), ("bf16", 9, 2112),
          ("bf16", 600, 4096), ("bf16", 3, 8192), ("bf16", 4, 16384), ("bf16_f32", 130, 1024), ("bf16_f32", 7, 4160),
          ("f32", 1, 1), ("f32", 6, 3), ("f32", 1003, 65), ("f32", 33, 1001), ("f32", 530, 1028), ("f32", 5, 4100),
          ("f32", 3, 5001), ("f32", 2, 16384)]


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["none", "col", "row", "elem"])
@pytest.mark.parametrize("mode,T,H", SHAPES)
def test_forward_and_backward(mode, T, H, gate):
    for post, pre in ((True, True), (False, True), (True, False)):
        s = make(T, H, mode, gate, post, pre)
        check_fwd(s, run_fwd(s))
        check_bwd(s, run_bwd(s))


@pytest.mark.gpu
@pytest.mark.parametrize("mode,T,H", [("bf16", 17, 4096), ("f32", 17, 250)])
def test_first_norm_and_plain_add(mode, T, H):
    s = make(T, H, mode, "none", False, True)
    kw = dict(eps=1e-5, unit_offset=False)
    out, X = lm.block_norm_fwd(s["R"], w_pre=s["par"]["w_pre"], **kw)
    assert out is s["R"]
    r = dict(s, Y=torch.zeros_like(s["R"]), kw=dict(res_scale=1.0, branch_scale=1.0, **kw))
    check("X", X, *ref_fwd(r)[1])
    dR, dY, grads = lm.block_norm_bwd(None, s["dX"], s["R"], w_pre=s["par"]["w_pre"], **kw)
    ref = ref_bwd(dict(r, dR=torch.zeros_like(s["R"])))
    assert dY is None
    check("dR", dR, *ref["dR"])
    check("w_pre", grads["w_pre"], *ref["w_pre"])
    # no norm at all: a gated residual
    s = make(T, H, mode, "row", False, False)
    check_fwd(s, run_fwd(s))
    check_bwd(s, run_bwd(s))


@pytest.mark.gpu
def test_gradients_against_differences():
    """dX and dR_out weigh the outputs; the fp32 gradients meet central differences of the float64
    forward, whose own error is h^2 and 1e-16 / h: 1e-9 at h = 1e-5 against the sums' 1e-6."""
    s = make(6, 40, "f32", "col", True, True)
    out = lm.block_norm_fwd(s["R"], s["Y"], **s["par"], **s["kw"])[0]
    # the backward is given the rounded R_out: 2^-24 of it, inside the tolerance
    dR, dY, grads = lm.block_norm_bwd(s["dR"], s["dX"], out, s["Y"], **s["par"], **s["kw"])

    def loss(q):
        o, x = ref_fwd(q)
        return (o[0] * d64(s["dR"])).sum() + (x[0] * d64(s["dX"])).sum()

    base = dict(s, R=d64(s["R"]), Y=d64(s["Y"]), par={k: d64(v) for k, v in s["par"].items()})
    for name, grad in {"R": dR, "Y": dY, **grads}.items():
        g = torch.Generator().manual_seed(5)
        where = base if name in ("R", "Y") else base["par"]
        x = where[name]
        for _ in range(4):
            v = torch.randn(x.shape, generator=g, dtype=torch.float64)
            h, side = 1e-5, []
            for sign in (1, -1):
                q = dict(base, par=dict(base["par"]))
                (q if name in ("R", "Y") else q["par"])[name] = x + sign * h * v
                side.append(loss(q))
            diff = (side[0] - side[1]) / (2 * h)
            dot = (d64(grad) * v).sum()
            scale = (d64(grad) * v).abs().sum()
            assert abs(diff - dot) <= 1e-5 * scale, (name, float(diff), float(dot))


@pytest.mark.gpu
def test_zero_rows_zero_and_bad_rows_stay_alone():
    s = make(64, 576, "bf16", "none", True, True)
    s["R"][7] = 0
    s["Y"][7] = 0
    s["Y"][9, 3] = float("nan")
    s["R"][11, 5] = float("inf")
    out, X = run_fwd(s)
    assert not out[7].any() and not X[7].any()
    assert out[9].isnan().all() and X[9].isnan().all()
    assert out[11, 5] == float("inf") and X[11].isnan().any()
    keep = [i for i in range(64) if i not in (9, 11)]
    assert out[keep].isfinite().all() and X[keep].isfinite().all()
    cut = dict(s, R=s["R"][keep].contiguous(), Y=s["Y"][keep].contiguous())
    a, b = run_fwd(cut)
    assert torch.equal(a, out[keep]) and torch.equal(b, X[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["bf16", "f32", "bf16_f32"])
def test_no_rows(mode):
    s = make(0, 128, mode, "col", True, True)
    out, X = run_fwd(s)
    assert out.shape == X.shape == (0, 128)
    grads = {k: torch.full_like(v, 7.0) for k, v in s["par"].items()}
    run_bwd(s, grads=grads)
    for k, v in grads.items():
        assert not v.any(), k


@pytest.mark.gpu
@pytest.mark.parametrize("H", [576, 4096])
def test_in_place(H):
    s = make(40, H, "bf16", "elem", True, True)
    out, X = run_fwd(s)
    dR, dY, grads = run_bwd(s)
    q = {k: v.clone() if torch.is_tensor(v) else v for k, v in s.items()}
    got = lm.block_norm_fwd(q["R"], q["Y"], **s["par"], **s["kw"], R_out=q["R"], X=q["Y"])
    assert got[0] is q["R"] and torch.equal(got[0], out) and torch.equal(got[1], X)
    q = {k: v.clone() if torch.is_tensor(v) else v for k, v in s.items()}
    got = lm.block_norm_bwd(q["dR"], q["dX"], q["R"], q["Y"], **s["par"], **s["kw"], dR=q["dR"], dY=q["dX"])
    assert torch.equal(got[0], dR) and torch.equal(got[1], dY)
    assert all(torch.equal(got[2][k], grads[k]) for k in grads)


@pytest.mark.gpu
def test_other_stream_and_same_answer_each_time():
    s = make(700, 4096, "bf16", "col", True, True)
    want = run_fwd(s) + run_bwd(s)[:2]
    grads = run_bwd(s)[2]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a = run_fwd(s) + run_bwd(s)[:2]
    b = run_fwd(s, stream=side) + run_bwd(s, stream=side)[:2]
    side.synchronize()
    for x, y, z in zip(want, a, b):
        assert torch.equal(x, y) and torch.equal(x, z)
    again = run_bwd(s)[2]
    assert all(torch.equal(again[k], grads[k]) for k in grads)


@pytest.mark.gpu
def test_captured_graph_replays():
    s = make(300, 1088, "bf16", "row", True, True)
    bufs = dict(R_out=torch.empty_like(s["R"]), X=torch.empty_like(s["R"]))
    run_fwd(s, **bufs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run_fwd(s, **bufs)
        held = lm.block_norm_bwd(s["dR"], s["dX"], bufs["R_out"], s["Y"], **s["par"], **s["kw"])
    for seed in (1, 2, 3):
        n = make(300, 1088, "bf16", "row", True, True, seed=seed)
        for k in ("R", "Y", "dR", "dX"):
            s[k].copy_(n[k])
        for k in s["par"]:
            s["par"][k].copy_(n["par"][k])
        g.replay()
        torch.cuda.synchronize()
        check_fwd(s, (bufs["R_out"], bufs["X"]))
        check_bwd(dict(s, R=bufs["R_out"]), held)
        torch.zeros(1 << 20, device="cuda").sum().item()


@pytest.mark.gpu
def test_past_two_gib():
    T, H = 70001, 16384
    assert T * H * 2 > 1 << 31
    R = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    Y = torch.zeros_like(R)
    s = make(3, H, "bf16", "none", True, True)
    R[-3:], Y[-3:] = s["R"], s["Y"]
    out, X = lm.block_norm_fwd(R, Y, **s["par"], **s["kw"])
    check_fwd(s, (out[-3:], X[-3:]))
    assert not out[:-3].any()
    del out, X
    dR_out, dX = torch.zeros_like(R), torch.zeros_like(R)
    dR_out[-3:], dX[-3:] = s["dR"], s["dX"]
    dR, dY, grads = lm.block_norm_bwd(dR_out, dX, R, Y, **s["par"], **s["kw"])
    check_bwd(s, (dR[-3:], dY[-3:], grads))


# More rows than blocks at every number of threads a row, with values in all of them: the rows that a block
# takes one after the other meet in its registers and in LDS.
DEEP = [("bf16", 4500, 576), ("bf16", 2100, 4096), ("bf16", 1100, 5120), ("bf16", 1100, 5184), ("bf16", 1100, 6144),
        ("bf16", 1100, 8192), ("bf16", 1100, 12288), ("bf16_f32", 1100, 5184), ("bf16_f32", 1100, 8192), ("bf16_f32", 1100, 16384),
        ("f32", 4500, 700), ("f32", 4500, 701), ("f32", 1100, 1025), ("f32", 1100, 2049), ("f32", 1100, 4095),
        ("f32", 1100, 5001), ("f32", 1100, 9001), ("f32", 1100, 4100), ("f32", 1100, 8196), ("f32", 1100, 16384)]


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["col", "elem"])
@pytest.mark.parametrize("mode,T,H", DEEP)
def test_more_rows_than_blocks(mode, T, H, gate):
    s = make(T, H, mode, gate, True, True, seed=T + H)
    check_fwd(s, run_fwd(s))
    check_bwd(s, run_bwd(s))


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["none", "col", "row", "elem"])
@pytest.mark.parametrize("T,H", [(33, 64), (1100, 1028), (5, 8192)])
def test_f32_at_four_byte_addresses(T, H, gate):
    def shifted(t):
        return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t) if torch.is_tensor(t) else t

    s = make(T, H, "f32", gate, True, True)
    q = {k: shifted(v) for k, v in s.items()}
    q["par"] = {k: shifted(v) for k, v in s["par"].items()}
    assert q["R"].data_ptr() % 16 == 4
    check_fwd(q, run_fwd(q))
    check_bwd(q, run_bwd(q))
    one = dict(s, Y=q["Y"])  # one tensor of the call is enough
    check_fwd(one, run_fwd(one))
    check_bwd(one, run_bwd(one))


# ---- refusals (no GPU) ----

def test_binding_refuses():
    s = make(4, 64, "bf16", "col", True, True, device="cpu")
    with pytest.raises(ValueError, match="GPU only"):
        run_fwd(s)
    with pytest.raises(ValueError, match="GPU only"):
        run_bwd(s)

    def bad(fn=run_fwd, par=None, extra=None, **kw):
        q = dict(s, par=dict(s["par"], **(par or {})), **kw)
        with pytest.raises(ValueError) as e:
            fn(q, **(extra or {}))
        assert "GPU only" not in str(e.value)

    z = torch.zeros
    bad(Y=z(4, 128, dtype=torch.bfloat16))
    bad(Y=z(4, 64))
    bad(Y=z(64, 4, dtype=torch.bfloat16).t())
    bad(R=z(256, dtype=torch.bfloat16))
    bad(R=z(4, 64, dtype=torch.float16))
    bad(par=dict(w_pre=z(32, dtype=torch.bfloat16)))
    bad(par=dict(w_pre=z(64)))  # parameters of two types
    bad(par=dict(gate=z(3, 1, dtype=torch.bfloat16)))
    bad(par=dict(gate=z(4, 1)))
    bad(extra=dict(X=z(4, 64)))
    bad(par=dict(w_pre=None), extra=dict(X=z(4, 64, dtype=torch.bfloat16)))
    bad(Y=None, extra=dict(R_out=z(4, 64, dtype=torch.bfloat16)))
    bad(run_bwd, dX=None)
    bad(run_bwd, par=dict(w_pre=None))
    bad(run_bwd, dR=z(4, 128, dtype=torch.bfloat16))
    bad(run_bwd, extra=dict(grads={}))
    bad(run_bwd, Y=None, extra=dict(dY=z(4, 64, dtype=torch.bfloat16)))


def status(name, *args):
    return getattr(L.load(), name)(*args)


def test_library_refuses():
    """Host checks: every call here is refused before anything is enqueued (the addresses are not read)."""
    def p(i):
        return ctypes.c_void_p(i << 20)

    def desc(T=4, H=64, eps=1e-6, res=1.0, br=1.0, off=1, gate=0, dtype=L.LORA_BF16, rsv=0):
        return ctypes.byref(L.lora_norm_desc(T, H, eps, res, br, off, gate, dtype, rsv))

    def fwd(d, R=1, Y=2, gate=0, post=3, pre=4, out=5, X=6):
        return status("lora_block_norm_fwd", d, *(p(x) if x else None for x in (R, Y, gate, post, pre, out, X)), None)

    for d, want in ((desc(H=96), L.LORA_ESHAPE), (desc(H=0), L.LORA_ESHAPE), (desc(H=16448), L.LORA_ESHAPE),
                    (desc(T=-1), L.LORA_ESHAPE), (desc(T=1 << 60), L.LORA_ESHAPE), (desc(dtype=7), L.LORA_EDTYPE),
                    (desc(gate=4), L.LORA_EINVAL), (desc(off=2), L.LORA_EINVAL), (desc(rsv=1), L.LORA_EINVAL),
                    (desc(eps=-1.0), L.LORA_EINVAL), (desc(eps=float("nan")), L.LORA_EINVAL),
                    (desc(res=float("inf")), L.LORA_EINVAL), (None, L.LORA_EINVAL)):
        assert fwd(d) == want
        assert status("lora_block_norm_workspace_size", d, None) == want
    ok = desc()
    assert fwd(ok, R=0) == L.LORA_EINVAL
    assert fwd(ok, Y=0) == L.LORA_EINVAL
    assert fwd(ok, out=0) == L.LORA_EINVAL
    assert fwd(ok, X=0) == L.LORA_EINVAL
    assert fwd(ok, gate=7) == L.LORA_EINVAL
    assert fwd(desc(gate=1)) == L.LORA_EINVAL
    assert fwd(ok, Y=0, out=0, post=3) == L.LORA_EINVAL
    assert fwd(desc(res=0.5), Y=0, out=0, post=0) == L.LORA_EINVAL
    assert fwd(ok, Y=0, out=0, post=0, pre=0, X=0) == L.LORA_EINVAL
    assert fwd(ok, out=6) == L.LORA_EUNSUPPORTED
    assert fwd(ok, out=4) == L.LORA_EUNSUPPORTED
    f = status("lora_block_norm_fwd", ok, p(1), p(2), None, p(3), p(4), ctypes.c_void_p((1 << 20) + 128), p(6), None)
    assert f == L.LORA_EUNSUPPORTED
    f = status("lora_block_norm_fwd", ok, p(1), ctypes.c_void_p((2 << 20) + 8), None, p(3), p(4), p(5), p(6), None)
    assert f == L.LORA_EALIGN

    def bwd(d, dro=1, dX=2, R=3, Y=4, gate=0, post=5, pre=6, dR=7, dY=8, g=(0, 9, 10), ws=11, n=1 << 19):
        gr = L.lora_norm_grads(*(p(x) if x else None for x in g))
        return status("lora_block_norm_bwd", d, *(p(x) if x else None for x in (dro, dX, R, Y, gate, post, pre, dR, dY)),
                      ctypes.byref(gr), p(ws) if ws else None, n, None)

    for kw, want in ((dict(dR=0), L.LORA_EINVAL), (dict(dX=0), L.LORA_EINVAL), (dict(R=0), L.LORA_EINVAL),
                     (dict(dY=0), L.LORA_EINVAL), (dict(Y=0, dY=0), L.LORA_EINVAL), (dict(g=(0, 9, 0)), L.LORA_EINVAL),
                     (dict(g=(12, 9, 10)), L.LORA_EINVAL), (dict(dro=0, pre=0, dX=0, g=(0, 9, 0)), L.LORA_EINVAL),
                     (dict(ws=0), L.LORA_EWORKSPACE), (dict(n=16), L.LORA_EWORKSPACE), (dict(dR=8), L.LORA_EUNSUPPORTED),
                     (dict(g=(0, 9, 9)), L.LORA_EUNSUPPORTED), (dict(g=(0, 9, 6)), L.LORA_EUNSUPPORTED),
                     (dict(ws=3), L.LORA_EUNSUPPORTED), (dict(dR=6), L.LORA_EUNSUPPORTED)):
        assert bwd(ok, **kw) == want, kw
