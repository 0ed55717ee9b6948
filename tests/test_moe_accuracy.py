"""moe_fwd over its sizes against float64 by the norm of each row's error (_moe_ref.py), a bound that follows the error's size
at every width, and, on the CPU, what that bound does not let pass."""
import pytest
import torch

import adapter_mlp_amd as lm
from _moe_ref import check_rows, layer
from test_moe import SIZES, make, run

WIDE = [(65, 128, 4096, 4, 2), (129, 64, 4160, 4, 4), (160, 8256, 64, 3, 2), (256, 8192, 128, 4, 3), (130, 4096, 64, 20, 6),
        (256, 128, 1024, 16, 5), (64, 1088, 1088, 64, 8), (20, 1088, 1088, 64, 8), (8, 64, 1088, 4, 4), (3, 4096, 4096, 2, 2)]
F32 = [(1, 5, 3, 2, 1), (4, 33, 17, 7, 3), (17, 250, 333, 10, 3), (9, 128, 64, 12, 4), (40, 36, 41, 4, 2), (64, 1090, 1092, 64, 8),
       (13, 127, 1301, 6, 2), (256, 15, 31, 30, 5)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,E,k", SIZES + WIDE)
def test_bf16(T, H, I, E, k):
    for seed, kw in enumerate((dict(), dict(mode="bf16_f32", shared=2, act="geglu_tanh", normalize=False, scale=1.5),
                               dict(shared=1, score="sigmoid", bias=True, scale=2.5), dict(score="sigmoid", normalize=False))):
        s = make(T, H, I, E, k, seed=seed, **kw)
        check_rows(s, run(s))


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,E,k", F32 + WIDE)
def test_f32(T, H, I, E, k):
    for seed, kw in enumerate((dict(), dict(shared=2, act="geglu_tanh", score="sigmoid", bias=True, normalize=False, scale=1.5))):
        s = make(T, H, I, E, k, "f32", seed=seed, **kw)
        check_rows(s, run(s))


@pytest.mark.gpu
def test_stacks_past_two_gib():
    H, I, E = 4096, 4096, 70
    assert E * H * I * 2 > 1 << 31
    small = make(3, H, I, 2, 2)
    big = {n: torch.zeros((E, H, I), dtype=torch.bfloat16, device="cuda") for n in ("gate", "up", "down")}
    for n in big:
        big[n][-2:] = getattr(small["ex"], n)
    router = torch.zeros(E, H, dtype=torch.bfloat16, device="cuda")
    router[-2:] = small["ex"].router
    router[:, 0], small["ex"].router[:, 0] = -30.0, 30.0
    router[-2:, 0] = 30.0
    small["X"][:, 0] = 1.0
    check_rows(small, run(dict(small, ex=lm.Experts(router=router, **big))))


# ---- what the bound refuses (no GPU) ----

@pytest.mark.parametrize("mode", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,I,E,k", SIZES + WIDE + F32)
def test_mistakes_are_seen(T, H, I, E, k, mode):
    """Of at most 20 rows and 8 experts, each as wide as on the GPU."""
    if mode == "bf16" and (H % 64 or I % 64):
        mode = "f32"
    E = min(E, 8)
    s = make(min(T, 20), H, I, E, min(k, E), mode, device="cpu")
    dt, step = s["X"].dtype, 64 if mode == "bf16" else 16
    right = layer(s)
    check_rows(s, right[0].to(dt), right)

    def planted(change):
        return layer(s, change)[0].to(dt)

    def last_step(name, t):  # of the inputs of gate and up, or of down
        if name != cut:
            return t
        t = t.clone()
        t[:, (t.shape[1] - 1) // step * step:] = 0
        return t

    wrong = [right[0].mul(0.98).to(dt), right[0].mul(1.02).to(dt), planted(lambda n, t: t.bfloat16().double() if n == "h" else t)]
    for cut in ("x", "h"):
        wrong.append(planted(last_step))
    for got in wrong:
        with pytest.raises(AssertionError, match="off by"):
            check_rows(s, got, right)
