"""The MLP of routed experts in float64, and how far a row of moe_fwd's output may be from it.

The bound is one of sizes, not of worst cases.  A sum of K products in fp32, whatever its order, makes K roundings of
partial sums, each at most 2^-24 of a partial sum; these roundings do not know of each other, so that the sum's error is
of the size sqrt(K) * 2^-24 * sqrt(sum of the squared products).  That is carried through the layer as squares: e and g
into h = phi(e) g (|phi'| <= 1.13; phi itself by 16 * 2^-24 of |e|), bf16 keeps h to 2^-16, down adds its own sum's size,
and a weight is off by at most 96 * 2^-24 (softmax: an exponential of a difference of at most 80, a sum and a quotient) or
4 * 2^-24 (sigmoid: formed in fp64, rounded once, multiplied).  With d the result, elementwise, |Y - y| <= |round(y) - y|
+ 2 |d|, where d is the error before the rounding: what rounding moves is within |d| of the distance that it moves y itself.
A row passes where the norm of Y - y is at most the norm of round(y) - y plus 2 * 4 times the norm of d's sizes."""
import torch

U = 2.0 ** -24


def score_logs(l, score):
    """The logarithms of the scores: finite however far down the logits lie."""
    return torch.log_softmax(l, 1) if score == "softmax" else torch.nn.functional.logsigmoid(l)


def routing(s):
    """Chosen experts (ties to the lower index, NaN last) and weights."""
    ex, kw = s["ex"], s["kw"]
    l = s["X"].double() @ ex.router.double().t()
    log = score_logs(l, kw["score"])
    key = l if ex.bias is None else log.exp() + ex.bias.double()
    key = torch.where(key.isnan(), torch.full_like(key, -torch.inf), key)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :s["k"]]
    w = log.gather(1, ids)
    w = torch.softmax(w, 1) if kw["normalize"] else w.exp()
    return ids, w * kw["scale"]


def phi(e, act):
    return e * torch.sigmoid(e) if act == "swiglu" else torch.nn.functional.gelu(e, approximate="tanh")


def layer(s, change=lambda name, t: t):
    """y and the size of its error before the last rounding.  change(name, t) may replace the inputs x and their weights'
    of gate and up ("x", "gate", "up") and h ("h"), for tests that plant a mistake."""
    ex, x, act = s["ex"], s["X"].double(), s["kw"]["act"]
    E, n, (T, H), I = ex.router.shape[0], ex.gate.shape[0], x.shape, ex.gate.shape[1]
    ids, w = routing(s)
    y, var, part = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    keep = 2.0 ** -16 if s["X"].dtype == torch.bfloat16 else 0.0
    rel = (96 if s["kw"]["score"] == "softmax" else 4) * U
    for e in range(n):
        hit = (ids == e).any(1) if e < E else torch.ones(T, dtype=torch.bool, device=x.device)
        rows = torch.nonzero(hit).flatten()
        if len(rows) == 0:
            continue
        we = (w * (ids == e)).sum(1)[rows, None] if e < E else torch.ones(len(rows), 1, dtype=torch.float64, device=x.device)
        xe, G, P, D = change("x", x[rows]), ex.gate[e].double().t().contiguous(), ex.up[e].double().t().contiguous(), ex.down[e].double().t().contiguous()
        G, P = change("gate", G), change("up", P)
        a, b = xe @ G, xe @ P
        da, db = H ** 0.5 * U * (xe.square() @ G.square()).sqrt(), H ** 0.5 * U * (xe.square() @ P.square()).sqrt()
        f = phi(a, act)
        h = change("h", f * b)
        dh = (1.13 * da * b).square() + (16 * U * a * b).square() + (f * db).square() + ((keep + 4 * U) * h).square()
        terms, D2 = h @ D, D.square()
        y[rows] += we * terms
        var[rows] += we.square() * (dh @ D2 + (I + n) * U * U * (h.square() @ D2))
        part[rows] += rel * (we * terms).abs()
    return y, var.sqrt() + part


def check_rows(s, got, of=None):
    """of: (y, sizes) where the caller has them."""
    y, size = layer(s) if of is None else of
    assert got.shape == y.shape and got.dtype == s["X"].dtype
    off = (got.double() - y).norm(dim=1)
    most = (y.to(got.dtype).double() - y).norm(dim=1) + 2 * 4 * size.norm(dim=1)
    bad = ~(off <= most)
    assert not bad.any(), f"row {int(bad.nonzero()[0])} of {len(bad)} ({int(bad.sum())} bad): off by {off[bad][0]:.3g}, at most " \
                          f"{most[bad][0]:.3g}, of norm {y.norm(dim=1)[bad][0]:.3g}"
