"""qk_norm_rope in place in buffers that hold q, k and v head by head, [T, heads, 3, d] and [heads, T, 3, d]: their rows lie
between each other's along both the tokens and the heads, and share nothing."""
import ctypes

import pytest
import torch

from adapter_mlp_amd import _lib as L
from test_qk_norm_rope import make, run_bwd, run_fwd, status


def views(T, h, d, parts, heads_first, dtype, device):
    shape = (h, T, parts, d) if heads_first else (T, h, parts, d)
    buf = torch.full(shape, 5.0, dtype=dtype, device=device)
    return [buf[:, :, i].transpose(0, 1) if heads_first else buf[:, :, i] for i in range(parts)]


@pytest.mark.gpu
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("mode,T,h,d", [("bf16", 4, 4, 64), ("bf16", 77, 8, 128), ("bf16", 1, 3, 80), ("f32", 33, 5, 66), ("f32", 9, 1, 64),
                                        ("bf16", 2, 130, 16)])
def test_in_place(mode, T, h, d, heads_first):
    s = make(T, h, h, d, mode)
    want, wantb = run_fwd(s), run_bwd(s)
    q, k, v = views(T, h, d, 3, heads_first, s["Q"].dtype, "cuda")
    q.copy_(s["Q"])
    k.copy_(s["K"])
    got = run_fwd(dict(s, Q=q, K=k), Q_out=q, K_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1]) and bool((v == 5.0).all())
    # outputs to other parts of the same buffer, and gradients over theirs
    a, b, x, y, v = views(T, h, d, 5, heads_first, s["Q"].dtype, "cuda")
    a.copy_(s["Q"])
    b.copy_(s["K"])
    run_fwd(dict(s, Q=a, K=b), Q_out=x, K_out=y)
    assert torch.equal(x, want[0]) and torch.equal(y, want[1]) and torch.equal(a, s["Q"]) and bool((v == 5.0).all())
    x.copy_(s["dQ"])
    y.copy_(s["dK"])
    grads = run_bwd(dict(s, Q=a, K=b, dQ=x, dK=y), dQ=x, dK=y)[2]
    assert torch.equal(x, wantb[0]) and torch.equal(y, wantb[1]) and bool((v == 5.0).all())
    assert torch.equal(a, s["Q"]) and torch.equal(b, s["K"]) and all(torch.equal(grads[n], wantb[2][n]) for n in grads)
    # keys of fewer heads than the buffer has
    if h > 1:
        s = make(T, h, 1, d, mode)
        want = run_fwd(s)
        q, k, v = views(T, h, d, 3, heads_first, s["Q"].dtype, "cuda")
        q.copy_(s["Q"])
        k[:, 1:2].copy_(s["K"])
        run_fwd(dict(s, Q=q, K=k[:, 1:2]), Q_out=q, K_out=k[:, 1:2])
        assert torch.equal(q, want[0]) and torch.equal(k[:, 1:2], want[1]) and bool((k[:, :1] == 5.0).all()) and bool((v == 5.0).all())


def accepted(T, hq, hk, q, k, at, d=64):
    """Whether lora_qk_norm_rope_fwd takes q and k in place, k at `at` elements from q.  Where it does it ends at the next check,
    of the workspace of a backward: nothing is enqueued."""
    desc = L.lora_rope_desc(T, hq, hk, d, d, 1, 0, 1, 0, 1.0, 1e-6, 0, L.LORA_F32, 0)
    base, far = 1 << 40, 1 << 44
    p = ctypes.c_void_p
    Q, K = L.lora_heads(base, *q), L.lora_heads(base + 4 * at, *k)
    Q2, K2 = L.lora_heads(far, hq * d, d), L.lora_heads(2 * far, hk * d, d)
    w = [p((4 + i) * far) for i in range(6)]
    # the last output overlaps the workspace, so that every call is refused: by its name where nothing else is
    got = status("lora_qk_norm_rope_bwd", desc, Q2, K2, Q2, K2, w[0], w[1], None, w[2], w[3], Q, K, w[4], w[5], w[5], 1 << 24, None)
    assert got == L.LORA_EUNSUPPORTED
    text = L.load().lora_last_error().decode()
    assert text in ("ws overlaps dw_k", "dK overlaps dQ"), text
    return text == "ws overlaps dw_k"


def brute(T, hq, hk, q, k, at, d=64):
    rows = {t * q[0] + i * q[1] for t in range(T) for i in range(hq)}
    return all(abs(at + t * k[0] + i * k[1] - r) >= d for t in range(T) for i in range(hk) for r in rows)


def test_rows_between_rows_on_the_host():
    """Against every pair of rows, over offsets and strides."""
    d, seen = 64, set()
    for T, hq, hk in ((4, 4, 4), (3, 5, 2), (1, 4, 4), (4, 1, 1), (5, 4, 1), (1, 1, 3), (2, 2, 2)):
        for st, sh in ((3 * d * 4, 3 * d), (3 * d * 5 + 7, 3 * d), (3 * d, 3 * d * 6), (2 * d, 2 * d * 5 + 1), (d * 6, d), (d, d * 6), (4 * d * 5, 130)):
            st = st if T > 1 else 9999
            if T > 1 and max(hq, hk) > 1 and not (st >= (max(hq, hk) - 1) * sh + d or sh >= (T - 1) * st + d):
                continue  # rows of one tensor overlap
            for at in [n * d // 4 for n in range(-30, 31)] + [d - 1, d + 1, -d + 1, 2 * d - 1, 2 * d + 1, st, sh, st + d, sh + d, 4 * st]:
                fits = accepted(T, hq, hk, (st, sh), (st, sh), at)
                assert fits == brute(T, hq, hk, (st, sh), (st, sh), at), (T, hq, hk, st, sh, at)
                seen.add(fits)
    assert seen == {False, True}
    # other strides: refused unless one of the simple forms holds, never taken where rows meet
    for q, k in (((768, 192), (768, 64)), ((768, 192), (800, 192)), ((1024, 64), (1024, 192)), ((192, 1024), (64, 1024))):
        for at in range(-800, 900, 32):
            assert not accepted(4, 4, 4, q, k, at) or brute(4, 4, 4, q, k, at), (q, k, at)
    # far more tokens than heads, at once
    assert accepted(1 << 24, 512, 512, (512 * 3 * 64, 3 * 64), (512 * 3 * 64, 3 * 64), 64)
    assert not accepted(1 << 24, 512, 512, (512 * 3 * 64, 3 * 64), (512 * 3 * 64, 3 * 64), 63)
