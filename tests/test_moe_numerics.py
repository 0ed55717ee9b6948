"""moe_fwd where its numbers go to their ends.  References and bounds: _moe_ref.py."""
import pytest
import torch

import adapter_mlp_amd as lm
from _moe_ref import check_rows, routing
from test_moe import make, run


def choices(T, H, E, mode, *, shifted=False, seed=0, device="cuda"):
    """A layer of top-1 experts that differ, and X, router whose best two logits of every token lie 1e-11 to 1e-8 apart:
    experts 2 i and 2 i + 1 have the same row but for one element, moved by a step of its type."""
    s = make(T, H, 64, E, 1, mode, seed=seed, device=device)
    r = s["ex"].router
    r[1::2] = r[0:E // 2 * 2:2]
    j = torch.arange(E // 2, device=device) * 7 % H
    i = torch.arange(E // 2, device=device)
    step = 2.0 ** -7 if r.dtype == torch.bfloat16 else 2.0 ** -23
    old = r[2 * i, j].float()
    old = torch.where(old.abs() < 0.02, torch.full_like(old, 0.02), old).to(r.dtype)
    r[2 * i, j] = old
    r[2 * i + 1, j] = (old.double() * (1 + step)).to(r.dtype)
    x = s["X"][:, j].double()
    x = torch.where(x < 0, x - 0.5, x + 0.5)  # no gap of nothing
    s["X"][:, j] = (x * (2.0 ** -20 if r.dtype == torch.bfloat16 else 2.0 ** -6)).to(s["X"].dtype)
    if shifted:
        for name in ("X", "router"):
            t = s["X"] if name == "X" else r
            u = torch.empty(t.numel() + 1, dtype=t.dtype, device=device)[1:].view(t.shape).copy_(t)
            if name == "X":
                s["X"] = u
            else:
                s["ex"].router = u
    return s


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,E", [(1, 192, 16), (2, 512, 200), (4, 2048, 64), (30, 256, 16), (30, 256, 100), (200, 320, 400)])
@pytest.mark.parametrize("mode", ["bf16", "bf16_f32", "f32", "f32 shifted"])
def test_choice_between_near_logits(T, H, E, mode):
    """Products of two bf16 or fp32 numbers are exact in fp64, so a logit is off by a few 2^-53 of its terms, and by nothing
    of a sum's order or an address's alignment that could turn the choice."""
    s = choices(T, H, E, mode.split()[0], shifted=mode.endswith("shifted"), seed=T)
    l = (s["X"].double().cpu() @ s["ex"].router.double().cpu().t())
    top = l.topk(2, dim=1).values
    gap = top[:, 0] - top[:, 1]
    assert (gap > 1e-11).all() and (gap < 1e-8).all()
    assert torch.equal(routing(s)[0][:, 0].cpu(), l.argmax(1))
    check_rows(s, run(s))


@pytest.mark.gpu
@pytest.mark.parametrize("E", [4, 200])
@pytest.mark.parametrize("T", [1, 3, 50])
@pytest.mark.parametrize("mode", ["bf16", "bf16_f32", "f32"])
def test_choice_after_cancellation(T, E, mode):
    """Logits of 1 and 1/2 that are left of terms of 2^24."""
    s = make(T, 64, 64, E, 1, mode)
    s["X"][:, :3] = torch.tensor([4096.0, 1.0, 4096.0])
    s["ex"].router.zero_()
    s["ex"].router[1, :3] = torch.tensor([0.0, 0.5, 0.0])
    s["ex"].router[2, :3] = torch.tensor([4096.0, 1.0, -4096.0])
    assert (routing(s)[0] == 2).all()
    check_rows(s, run(s))


# T, E: one token whose choice is made beside gate and up; a small router; the choice as a launch of its own; many tokens
ROUTES = [(1, 16), (1, 300), (5, 16), (6, 400), (40, 16), (70, 500)]


@pytest.mark.gpu
@pytest.mark.parametrize("level", [-20.0, -87.0, -95.0, -103.0, -110.0, -700.0, -744.0, -1000.0, -30000.0])
@pytest.mark.parametrize("mode", ["bf16", "f32"])
@pytest.mark.parametrize("T,E", ROUTES)
def test_sigmoid_weights_of_far_logits(T, E, mode, level):
    """Normalised, they are those of the quotient, finite however small the scores are."""
    for k, bias in ((3, False), (1, False), (3, True)):
        s = make(T, 192, 64, E, k, mode, score="sigmoid", bias=bias, scale=1.5, shared=1, seed=T + E)
        s["X"][:, 0] = 1.0
        s["ex"].router[:, 0] = level
        ids, w = routing(s)
        assert w.isfinite().all() and torch.allclose(w.sum(1), torch.full_like(w[:, 0], 1.5))
        check_rows(s, run(s))
    # one chosen logit far above the others: no score is lost either way
    s = make(T, 192, 64, E, 3, mode, score="sigmoid", seed=1)
    s["X"][:, 0] = 1.0
    s["ex"].router[:, 0] = level
    s["ex"].router[E // 2, 0] = 5.0
    check_rows(s, run(s))
    # without the quotient the scores themselves, which may be nothing in Y's type
    s = make(T, 192, 64, E, 3, mode, score="sigmoid", normalize=False, shared=1, seed=2)
    s["X"][:, 0] = 1.0
    s["ex"].router[:, 0] = level
    check_rows(s, run(s))


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 3, 30])
@pytest.mark.parametrize("m", [1.0, 1.0078125])
def test_small_hidden_values(T, mode, m):
    """h of 2^-125 and more keeps its value, and an infinity in down stays one of its sign.  h is m^2 2^-p for ever larger p,
    an expert a p: its parts, where it is kept in two, end below the normal numbers."""
    ps = [0, 60, 95, 100, 103, 104, 108, 109, 110, 111, 112, 115, 116, 117, 118, 119, 120, 122, 123, 124, 125]
    for p in ps:
        for sign in (1.0, -1.0):
            s = make(T, 128, 64, 4, 2, mode, shared=1)
            for name in ("gate", "up", "down"):
                getattr(s["ex"], name).zero_()
            s["X"][:, 0] = 1.0
            # phi(x) of a small x is x / 2, of a large one x
            big = p == 0
            s["ex"].gate[4, 7, 0] = 64.0 * m if big else m * 2.0 ** -(p // 2)
            s["ex"].up[4, 7, 0] = sign * m * 2.0 ** -(p - p // 2 - (0 if big else 1))
            s["ex"].down[4, 3, 7] = float("inf")
            s["ex"].down[4, 5, 7] = float("-inf")
            s["ex"].down[4, 9, 7] = 1.5 * 2.0 ** (p // 2)
            y = run(s).double()
            assert (y[:, 3] == sign * float("inf")).all() and (y[:, 5] == -sign * float("inf")).all(), p
            x = m * 2.0 ** -(p // 2)
            h = (64.0 * m if big else x / (1 + torch.tensor(-x, dtype=torch.float64).exp())) * m * 2.0 ** -(p - p // 2 - (0 if big else 1))
            want = sign * h * 1.5 * 2.0 ** (p // 2)
            # half a step of Y's type, 2^-16 of h (two steps of 2^-133 at its smallest), phi's 16 * 2^-24 and two more roundings
            tol = (2.0 ** -8 + max(2.0 ** -16, 2.0 ** (p - 134)) if mode == "bf16" else 2.0 ** -24) + 18 * 2.0 ** -24
            assert ((y[:, 9] - want).abs() <= tol * abs(want)).all(), (p, float(y[0, 9]), float(want))
            keep = [n for n in range(128) if n not in (3, 5, 9)]
            assert not y[:, keep].any()


@pytest.mark.gpu
@pytest.mark.parametrize("E,H,mode,one", [(64, 512, "bf16", True), (64, 64, "f32", True), (65, 64, "f32", False), (512, 64, "bf16", False),
                                          (8, 4096, "bf16", True), (8, 4160, "bf16", False)])
def test_launches_of_the_choice(E, H, mode, one):
    """Logits and choice in one launch only where every token's block is quick to read the whole router."""
    s = make(20, H, 64, E, 2, mode)
    lm.trace_begin("moe")
    got = run(s)
    torch.cuda.synchronize()
    names = set(lm.trace_end())
    assert names & {"moe_route", "moe_logits", "moe_select"} == ({"moe_route"} if one else {"moe_logits", "moe_select"})
    check_rows(s, got)


@pytest.mark.gpu
@pytest.mark.parametrize("mode,T,H,I,E,k", [("bf16", 2, 192, 64, 6, 2), ("bf16", 8, 256, 192, 4, 2), ("bf16", 8, 256, 192, 200, 2),
                                            ("bf16", 40, 256, 192, 4, 2), ("bf16", 200, 4096, 192, 6, 3), ("bf16", 256, 192, 1088, 40, 3),
                                            ("f32", 9, 100, 70, 5, 2), ("f32", 16, 130, 200, 3, 3)])
def test_a_token_does_not_hang_on_the_others(mode, T, H, I, E, k):
    """In bf16, and in fp32 of up to 16 tokens, a token's bits are the same whatever the others choose."""
    s = make(T, H, I, E, k, mode, shared=1)
    want = run(s)
    other = make(T, H, I, E, k, mode, shared=1, seed=1)["X"]
    for t in (0, T - 1):
        alike = dict(s, X=s["X"][t].expand(T, -1).contiguous())  # all on the same experts
        assert torch.equal(run(alike), want[t].expand(T, -1))
        mixed = other.clone()
        mixed[t] = s["X"][t]
        assert torch.equal(run(dict(s, X=mixed))[t], want[t])
