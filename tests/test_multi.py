"""Adapters of many requests beside a shared projection (multi_fwd) against the formula in float64,
and the calls it refuses.

Tolerance per element: half a step of the output's type relative to the value; the fp32 sums, whose
roundings number K / 32 + 16 in bf16 (the matrix cores add 32 products at a time) and K in fp32,
each 2^-24 of the sum of absolute products; and in bf16 one rounding of U = X A to bf16, 2^-8 of
the adapter term's absolute products."""
import ctypes

import pytest
import torch

import adapter_mlp_amd as lm
from adapter_mlp_amd import _lib as L

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(T, K, N, r, n, dtype="bf16", ids="mixed", seed=0, device="cuda"):
    g = torch.Generator().manual_seed(seed)

    def rnd(*shape, scale=1.0):
        return (torch.randn(shape, generator=g) * scale).to(DT[dtype]).to(device)

    s = dict(X=rnd(T, K), W=rnd(K, N, scale=K ** -0.5))
    s["pool"] = lm.AdapterPool(A=rnd(n, K, r, scale=K ** -0.5), B=rnd(n, r, N, scale=r ** -0.5),
                               scale=(torch.rand(n, generator=g) + 0.5).to(device))
    t = torch.arange(T)
    pick = {"mixed": torch.randint(-1, max(n, 1), (T,), generator=g), "runs": t * max(n, 1) // max(T, 1), "each": t % max(n, 1),
            "one": torch.full((T,), n - 1), "none": torch.full((T,), -1),
            "odd": torch.tensor([-5, n, 2 ** 31 - 1, -2 ** 31, 0, n - 1])[t % 6]}[ids]
    s["ids"] = pick.to(torch.int32).to(device)
    return s


def reference(s, base=None):
    """(value, bound) in float64."""
    X, ids = s["X"].double().cpu(), s["ids"].cpu().long()
    p = s["pool"]
    n, K, r = p.A.shape
    low = s["X"].dtype == torch.bfloat16
    c = (K / 32 + 16 if low else K) * 2.0 ** -24
    if base is None:
        W = s["W"].double().cpu()
        y, mag = X @ W, c * (X.abs() @ W.abs())
    else:
        y = base.double().cpu().clone()
        mag = c * y.abs()
    for i in range(n):
        rows = torch.nonzero(ids == i).flatten()
        if len(rows) == 0:
            continue
        A, B, k = p.A[i].double().cpu(), p.B[i].double().cpu(), float(p.scale[i])
        U = X[rows] @ A
        y[rows] += k * (U @ B)
        mag[rows] += k * ((c * (X[rows].abs() @ A.abs()) + ((2.0 ** -8 if low else 0) + r * 2.0 ** -24) * U.abs()) @ B.abs())
    return y, HALF[s["X"].dtype] * y.abs() * (1 + 2.0 ** -7) + mag


def check(got, ref):
    y, bound = ref
    assert got.shape == y.shape
    err = (got.double().cpu() - y).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"off by {err[bad].max():.3g} at {int(bad.sum())} of {err.numel()}, bound {bound[bad].min():.3g}"


def run(s, **kw):
    return lm.multi_fwd(s["X"], s["W"], s["pool"], s["ids"], **kw)


CASES = [(1, 64, 64, 8, 1), (1, 4096, 1024, 16, 3), (2, 128, 192, 16, 5), (16, 320, 576, 24, 7), (17, 1024, 128, 32, 40),
         (33, 1088, 704, 40, 4), (64, 512, 1024, 48, 9), (65, 4096, 512, 64, 80), (129, 2112, 320, 56, 6), (300, 576, 1088, 8, 300),
         (777, 1024, 640, 16, 12), (1030, 256, 2048, 64, 3), (2500, 512, 512, 32, 20),
         (1300, 640, 320, 40, 300), (450, 4096, 4160, 16, 5), (1025, 64, 64, 8, 1), (1800, 192, 448, 56, 70),
         (2304, 640, 640, 24, 2), (4096, 1664, 192, 16, 1), (3000, 2112, 704, 64, 9), (4097, 64, 64, 8, 1), (4100, 128, 192, 40, 5),
         (4500, 192, 448, 56, 70), (4300, 640, 320, 32, 300), (800, 4096, 2112, 48, 6)]


@pytest.mark.gpu
@pytest.mark.parametrize("ids", ["mixed", "runs", "each", "one", "none", "odd"])
@pytest.mark.parametrize("T,K,N,r,n", CASES)
def test_bf16(T, K, N, r, n, ids):
    s = make(T, K, N, r, n, ids=ids)
    check(run(s), reference(s))


@pytest.mark.gpu
@pytest.mark.parametrize("ids", ["mixed", "runs", "each", "odd"])
@pytest.mark.parametrize("T,K,N,r,n", [(1, 1, 1, 1, 1), (3, 70, 33, 5, 4), (65, 256, 704, 8, 6), (130, 333, 129, 64, 30), (18, 1500, 77, 17, 2)])
def test_f32(T, K, N, r, n, ids):
    s = make(T, K, N, r, n, "f32", ids)
    check(run(s), reference(s))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20, 700, 4200])
def test_added_to_a_base(T):
    s = make(T, 1024, 512, 16, 6)
    base = run(make(T, 1024, 512, 16, 6, ids="none"))
    got = base.clone()
    assert lm.multi_fwd(s["X"], None, s["pool"], s["ids"], Y=got) is got
    check(got, reference(s, base))
    none = s["ids"] < 0
    assert torch.equal(got[none], base[none])
    s = make(T, 100, 50, 3, 6, "f32")
    base = torch.randn(T, 50, device="cuda")
    got = lm.multi_fwd(s["X"], None, s["pool"], s["ids"], Y=base.clone())
    check(got, reference(s, base))


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,r", [(300, 14336, 64, 64), (129, 2048, 64, 8), (128, 2048, 64, 8), (1100, 320, 64, 40), (4200, 320, 64, 40)])
def test_one_workspace_for_both_forms(T, K, N, r):
    """The size that is asked for covers the call without W too, whichever path the one with W takes."""
    s = make(T, K, N, r, 5)
    ws = torch.empty(lm.multi_workspace_size(T, K, N, r, 5), dtype=torch.uint8, device="cuda")
    check(run(s, ws=ws), reference(s))
    base = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    check(lm.multi_fwd(s["X"], None, s["pool"], s["ids"], Y=base.clone(), ws=ws), reference(s, base))


@pytest.mark.gpu
def test_beside_an_nf4_base():
    s = make(40, 512, 512, 16, 5)
    q = lm.nf4_quantize(s["W"])
    Y = lm.nf4_gemm(s["X"], q)
    base = Y.clone()
    lm.multi_fwd(s["X"], None, s["pool"], s["ids"], Y=Y)
    check(Y, reference(s, base))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40, 900, 1100, 4200])
def test_one_adapter_agrees_with_o_fwd(T):
    s = make(T, 512, 768, 16, 3, ids="one")
    p = s["pool"]
    Y, _ = lm.o_fwd(s["X"], lm.Proj(A=p.A[2], B=p.B[2], scale=float(p.scale[2]), W=s["W"]))
    check(Y, reference(s))
    check(run(s), reference(s))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [9, 80, 1000, 1200, 4200])
def test_a_bad_adapter_or_row_stays_alone(T):
    s = make(T, 512, 512, 24, 8)
    want = run(s)
    s["pool"].A[3] = float("nan")
    s["pool"].B[5] = float("inf")
    s["X"][4, 7] = float("inf")
    got = run(s)
    hit = (s["ids"] == 3) | (s["ids"] == 5)
    hit[4] = True
    assert hit.any() and not hit.all()
    assert not got[hit].isfinite().all(1).any()
    assert torch.equal(got[~hit], want[~hit])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_rows_and_no_adapters(dtype):
    assert run(make(0, 128, 64, 8, 2, dtype)).shape == (0, 64)
    s = make(30, 128, 64, 8, 0, dtype, ids="none")
    check(run(s), reference(s))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 100, 600, 1500, 4200])
def test_other_stream_and_same_answer(T):
    s = make(T, 1024, 1024, 16, 7)
    want = run(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = run(s, stream=side)
    with torch.cuda.stream(side):
        b = run(s)
    side.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want) and torch.equal(run(s), want)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 90, 500, 1300, 4200])
def test_captured_graph_replays(T):
    s = make(T, 512, 576, 16, 6)
    Y = run(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(s, Y=Y)
    for seed in (1, 2, 3):
        q = make(T, 512, 576, 16, 6, ids="mixed" if seed < 3 else "runs", seed=seed)
        s["X"].copy_(q["X"])
        s["ids"].copy_(q["ids"])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, run(s))
        torch.zeros(1 << 20, device="cuda").sum().item()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 700, 1100, 4200])
def test_stacks_past_two_gib(T):
    s = make(T, 64, 128, 64, 2, ids="each")
    n = 1 << 18
    p = s["pool"]
    big = lm.AdapterPool(A=torch.zeros(n, 64, 64, dtype=torch.bfloat16, device="cuda"),
                         B=torch.zeros(n, 64, 128, dtype=torch.bfloat16, device="cuda"), scale=torch.zeros(n, device="cuda"))
    assert big.A.numel() * 2 >= 1 << 31
    for x, y in ((big.A, p.A), (big.B, p.B), (big.scale, p.scale)):
        x[n - 2:] = y
    got = lm.multi_fwd(s["X"], s["W"], big, s["ids"] + (n - 2))
    assert torch.equal(got, run(s))


@pytest.mark.gpu
@pytest.mark.parametrize("K,N,r", [(8, 5, 33), (5, 8, 3)])
def test_more_rows_than_a_grid_row(K, N, r):
    T = (1 << 22) + 77 if r > 16 else (1 << 24) + 77
    s = make(1000, K, N, r, 3, "f32")
    reps = -(-T // 1000)
    X = s["X"].repeat(reps, 1)[:T].contiguous()
    ids = s["ids"].repeat(reps)[:T].contiguous()
    got = lm.multi_fwd(X, s["W"], s["pool"], ids)
    want = run(s)
    full = T // 1000 * 1000
    assert torch.equal(got[:full].view(-1, 1000, N), want.expand(full // 1000, 1000, N))
    assert torch.equal(got[full:], want[:T - full])


@pytest.mark.gpu
@pytest.mark.parametrize("r", [8, 24, 32, 40, 64])
@pytest.mark.parametrize("T", [70, 1000, 4200])
def test_adapter_term_alone_keeps_its_bits(T, r):
    """Without a base (W = 0) what is left is U B_i.  However many rows share the batch, U loses no more
    than two bf16 parts leave of it: each rounds by half a step, 2^-8 2^-8 = 2^-16 of U."""
    K, N = 512, 512
    s = make(T, K, N, r, 5)
    s["W"].zero_()
    X, ids, p, c = s["X"].double().cpu(), s["ids"].cpu().long(), s["pool"], (K / 32 + 16) * 2.0 ** -24
    y, mag = torch.zeros(T, N).double(), torch.zeros(T, N).double()
    for i in range(5):
        rows = torch.nonzero(ids == i).flatten()
        A, B, k = p.A[i].double().cpu(), p.B[i].double().cpu(), float(p.scale[i])
        U = X[rows] @ A
        y[rows] = k * (U @ B)
        mag[rows] = k * ((c * (X[rows].abs() @ A.abs()) + (2.0 ** -16 + (r + 2) * 2.0 ** -24) * U.abs()) @ B.abs())
    check(run(s), (y, HALF[torch.bfloat16] * y.abs() * (1 + 2.0 ** -7) + mag))


@pytest.mark.gpu
@pytest.mark.parametrize("r", [16, 64])
@pytest.mark.parametrize("T", [40, 1000, 4200])
def test_an_infinite_weight_gives_its_infinity(T, r):
    """One infinity in a column of B_3: the rows of that adapter are infinite there, with the sign of their U."""
    s = make(T, 512, 512, r, 5)
    s["X"][::2] = 0.0
    s["X"][::2, 0] = 1.0                                # U of these rows is A's first row, a bf16 value: no low part
    s["pool"].scale.fill_(1.0)
    want = run(s)
    s["pool"].B[3, 5, 100] = float("inf")
    got = run(s)
    rows = (s["ids"] == 3).nonzero().flatten()
    U = s["X"][rows].double().cpu() @ s["pool"].A[3, :, 5].double().cpu()
    assert len(rows) and (U.abs() > 1e-4).all()         # far from where the fp32 sums could change a sign
    assert torch.equal(got[rows, 100].double().cpu(), U.sign() * float("inf"))
    got[rows, 100] = want[rows, 100]
    assert torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("ids", ["mixed", "runs"])
@pytest.mark.parametrize("T,K,N,r,n", [(1500, 1030, 1500, 51, 6), (2053, 512, 1055, 16, 3), (1601, 77, 1344, 7, 9)])
def test_f32_of_whole_tiles(T, K, N, r, n, ids):
    """512 blocks of 64 x 64 and more: the form that does not split K, through its pipelined steps and its tail."""
    s = make(T, K, N, r, n, "f32", ids)
    check(run(s), reference(s))
    base = torch.randn(T, N, generator=torch.Generator().manual_seed(1)).cuda()
    check(lm.multi_fwd(s["X"], None, s["pool"], s["ids"], Y=base.clone()), reference(s, base))


def shifted(t):
    """The same values one element past a 16-byte boundary."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    out = flat[1:].view(t.shape)
    assert out.data_ptr() % 16 == 4
    return out.copy_(t)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,r", [(9, 256, 128, 8), (130, 333, 129, 20), (1500, 128, 1536, 16)])
def test_f32_at_four_byte_addresses(T, K, N, r):
    s = make(T, K, N, r, 4, "f32")
    want = run(s)
    p = s["pool"]
    q = dict(s, X=shifted(s["X"]), W=shifted(s["W"]), pool=lm.AdapterPool(A=shifted(p.A), B=shifted(p.B), scale=shifted(p.scale)),
             ids=shifted(s["ids"]))
    assert torch.equal(run(q, Y=shifted(torch.zeros(T, N, device="cuda"))), want)


def on_device(T, K, N, r, n, seed, dtype="bf16"):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(DT[dtype])

    return dict(X=rnd(T, K), W=rnd(K, N, scale=K ** -0.5), ids=torch.randint(-1, n, (T,), generator=g, device="cuda", dtype=torch.int32),
                pool=lm.AdapterPool(A=rnd(n, K, r, scale=K ** -0.5), B=rnd(n, r, N, scale=r ** -0.5),
                                    scale=torch.rand(n, generator=g, device="cuda") + 0.5))


def check_on_device(s):
    """The call against float64 on the GPU, for sizes that take the CPU long; U to two bf16 parts."""
    K, low, p = s["X"].shape[1], s["X"].dtype == torch.bfloat16, s["pool"]
    n, _, r = p.A.shape
    X, W, c = s["X"].double(), s["W"].double(), (K / 32 + 16 if low else K) * 2.0 ** -24
    y, mag = X @ W, c * (X.abs() @ W.abs())
    del W
    for i in range(n):
        rows = torch.nonzero(s["ids"] == i).flatten()
        A, B, k = p.A[i].double(), p.B[i].double(), float(p.scale[i])
        U = X[rows] @ A
        y[rows] += k * (U @ B)
        mag[rows] += k * ((c * (X[rows].abs() @ A.abs()) + ((2.0 ** -16 if low else 0) + (r + 2) * 2.0 ** -24) * U.abs()) @ B.abs())
    err = (run(s).double() - y).abs_()
    bad = ~(err <= HALF[s["X"].dtype] * y.abs() * (1 + 2.0 ** -7) + mag)
    assert not bad.any(), f"off by {err[bad].max():.3g} at {int(bad.sum())} of {err.numel()}"


@pytest.mark.gpu
@pytest.mark.parametrize("r", [16, 40])
def test_split_and_unsplit_tiles_in_one_launch(r):
    """272 tiles of 256 x 256 on 256 CUs: the last 16 are split over K, and take their adapters in the first part."""
    check_on_device(on_device(4349, 8192, 4096, r, 5, seed=r))


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,r,dtype", [(3, 1 << 22, 64, 8, "bf16"), (255, 1 << 22, 64, 16, "bf16"), (3, 64, 1 << 22, 64, "bf16"),
                                           (255, 64, 1 << 22, 24, "bf16"), (3, 1 << 22, 33, 9, "f32"), (5, 33, 1 << 22, 64, "f32")])
def test_widest_sides(T, K, N, r, dtype):
    check_on_device(on_device(T, K, N, r, 3, 7, dtype))


@pytest.mark.gpu
def test_current_stream_without_the_internal_accessor(monkeypatch):
    s = make(5, 256, 128, 8, 3)
    want = run(s)
    torch.cuda.synchronize()
    side, dev = torch.cuda.Stream(), s["X"].device
    for missing in (False, True):
        if missing:
            monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
        assert lm._current_stream(dev) == torch.cuda.current_stream(dev).cuda_stream
        with torch.cuda.stream(side):
            assert lm._current_stream(dev) == side.cuda_stream
            got = run(s)
        side.synchronize()
        assert torch.equal(got, want)


# ---- refusals (no GPU) ----

def test_binding_refuses():
    s = make(4, 64, 128, 8, 3, device="cpu")
    with pytest.raises(ValueError, match="GPU only"):
        run(s)
    z, h = torch.zeros, torch.bfloat16

    def bad(pool=None, extra=None, **kw):
        q = dict(s, **kw)
        if pool:
            q["pool"] = lm.AdapterPool(**{**vars(s["pool"]), **pool})
        with pytest.raises(ValueError) as e:
            run(q, **(extra or {}))
        assert "GPU only" not in str(e.value)

    bad(X=z(4, 64))
    bad(X=z(4, 64, dtype=torch.float16))
    bad(X=z(64, 4, dtype=h).t())
    bad(W=z(128, 64, dtype=h))
    bad(W=None)
    bad(ids=s["ids"].long())
    bad(ids=s["ids"][:3])
    bad(pool=dict(A=z(64, 8, dtype=h)))
    bad(pool=dict(A=z(2, 64, 8, dtype=h)))
    bad(pool=dict(B=z(3, 16, 128, dtype=h)))
    bad(pool=dict(A=s["pool"].A.float()))
    bad(pool=dict(scale=z(3, dtype=h)))
    bad(pool=dict(scale=z(2)))
    bad(extra=dict(Y=z(4, 64, dtype=h)))


def test_library_refuses():
    """Refused on the host; no address here is read."""
    def call(T=4, K=128, N=192, r=8, n=3, dtype=L.LORA_BF16, rsv=0, X=1, W=2, A=3, B=4, sc=5, ids=6, Y=7, ws=8, nbytes=1 << 40, off=0):
        d = L.lora_multi_desc(T, K, N, r, n, dtype, rsv)
        at = [x << 30 if x else None for x in (X, W, A, B, sc, ids, Y, ws)]
        at[0] = at[0] + off if at[0] else None
        return L.load().lora_multi_fwd(ctypes.byref(d), *at, nbytes, None)

    for kw, want in ((dict(T=-1), L.LORA_ESHAPE), (dict(K=96), L.LORA_ESHAPE), (dict(N=0), L.LORA_ESHAPE), (dict(r=12), L.LORA_ESHAPE),
                     (dict(r=72), L.LORA_ESHAPE), (dict(r=0), L.LORA_ESHAPE), (dict(n=-1), L.LORA_ESHAPE), (dict(K=1 << 40), L.LORA_ESHAPE), (dict(K=(1 << 22) + 64, N=64), L.LORA_ESHAPE),
                     (dict(T=1 << 40), L.LORA_ESHAPE), (dict(T=1 << 24), L.LORA_ESHAPE), (dict(dtype=L.LORA_BF16_F32LORA), L.LORA_EDTYPE),
                     (dict(rsv=3), L.LORA_EINVAL), (dict(X=0), L.LORA_EINVAL), (dict(A=0), L.LORA_EINVAL), (dict(B=0), L.LORA_EINVAL),
                     (dict(sc=0), L.LORA_EINVAL), (dict(ids=0), L.LORA_EINVAL), (dict(Y=0), L.LORA_EINVAL), (dict(off=8), L.LORA_EALIGN),
                     (dict(ws=0), L.LORA_EWORKSPACE), (dict(nbytes=64), L.LORA_EWORKSPACE), (dict(Y=1), L.LORA_EUNSUPPORTED),
                     (dict(Y=6), L.LORA_EUNSUPPORTED), (dict(ws=7), L.LORA_EUNSUPPORTED), (dict(ws=2), L.LORA_EUNSUPPORTED)):
        assert call(**kw) == want, kw
    assert L.load().lora_multi_fwd(None, *[None] * 8, 0, None) == L.LORA_EINVAL
    assert call(T=0, X=0, Y=0, ids=0, ws=0, nbytes=0) == L.LORA_OK
