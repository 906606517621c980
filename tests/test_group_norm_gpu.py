"""Group norm with an activation on the GPU against its fp64 form, element by element, and its
gradients against reverse mode in fp64."""
import pytest
import torch

import operators_ref as R

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def kda(cuda_ok):
    from gated_delta_rule_75_b200 import build
    build.build()
    import gated_delta_rule_75_b200 as kda
    return kda


def inputs(M, G, d, io, per_group, seed, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)
    shape = (G, d) if per_group else (d,)
    t = lambda v: v.to(R.IO[io]).cuda()
    return (t(n(M, G, d) + offset), t(n(M, G, d) * 2), (1 + 0.2 * n(*shape)).cuda(), (0.2 * n(*shape)).cuda(),
            t(n(M, G, d)))


SIZES = [(1, 1, 1), (3, 2, 5), (2, 3, 8), (7, 5, 32), (65, 1, 64), (33, 4, 128), (300, 16, 128), (10, 33, 100),
         (9, 2, 250), (5, 3, 255), (4, 7, 512), (6, 1, 509), (2000, 3, 64), (1, 300, 128), (3, 700, 20)]
FORMS = [("sigmoid", False, False, True, True, False), ("silu", True, True, True, True, True),
         ("silu", False, True, False, True, False), ("none", True, False, False, False, True),
         ("none", False, True, True, False, False)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("name,center,per_group,gated,weighted,biased", FORMS)
@pytest.mark.parametrize("M,G,d", SIZES)
def test_values_and_gradients(kda, M, G, d, name, center, per_group, gated, weighted, biased, io):
    x, z, w, b, dy = inputs(M, G, d, io, per_group, M + 31 * G + d, offset=0.5 if center else 0.0)
    z, w, b = z if gated else None, w if weighted else None, b if biased else None
    kw = dict(eps=EPS, activation=name, center=center)
    out = kda.group_norm_fwd(x, w, bias=b, gate=z, **kw)
    form = lambda x, w, b, z: R.group_norm(x, w, b, z, EPS, name, center)
    bound = R.group_norm_bound(R.d(x), R.d(w), R.d(b), R.d(z), EPS, name, center)
    R.within(out, form(R.d(x), R.d(w), R.d(b), R.d(z)), bound, "out")
    dx, dz, dw, db = kda.group_norm_bwd(x, w, dy, bias=b, gate=z, **kw)
    want = R.grads(form, [R.d(t) for t in (x, w, b, z)], R.d(dy))
    assert (dz is None) == (z is None) and (dw is None) == (w is None) and (db is None) == (b is None)
    # magnitudes that the gradients sum, each off by a few ROW (its own rounding, the statistics', the
    # activation's): 8 ROW of them bounds the error; sums over tokens add at most (tokens a slot, the slots,
    # the rows) half steps, under 2^-12 of the magnitudes for these sizes even one after another
    X = R.d(x)
    mu = X.mean(-1, keepdim=True) if center else torch.zeros_like(X[..., :1])
    r = 1 / torch.sqrt(((X - mu) ** 2).mean(-1, keepdim=True) + EPS)
    xh = (X - mu) * r
    big = (X.abs() + (X.abs().mean(-1, keepdim=True) if center else 0)) * r        # what xh is made of
    big = big + big.mean(-1, keepdim=True) * xh.abs()
    W = torch.ones(d).double() if w is None else R.d(w).abs()
    nb = big * W + (0 if b is None else R.d(b).abs())
    t = R.d(z) if gated else form(X, R.d(w), R.d(b), None) if name == "none" else \
        R.group_norm(X, R.d(w), R.d(b), None, EPS, "none", center)
    f, slope = R.act(name, t).abs(), 1.1
    dn = R.d(dy).abs() * ((f + (0 if gated else slope)) if gated else slope * (1 + nb * (name != "none")))
    c = dn * W
    dx_big = r * (c + xh.abs() * (c * big).mean(-1, keepdim=True) + c.mean(-1, keepdim=True)) * (1 + big)
    R.within(dx, want[0], 8 * R.ROW * dx_big, "dx")
    if gated:
        R.within(dz, want[3], 8 * R.ROW * R.d(dy).abs() * nb * slope, "dgate")
    rows = 0 if per_group else (0, 1)
    steps = (M * (1 if per_group else G) + 64) * 2.0 ** -24
    if weighted:
        R.within(dw, want[1], (8 * R.ROW + steps) * (dn * big).sum(rows), "dweight")
    if biased:
        R.within(db, want[2], (8 * R.ROW + steps) * dn.sum(rows), "dbias")
    again = kda.group_norm_bwd(x, w, dy, bias=b, gate=z, **kw)
    assert all(p is None or torch.equal(p, q) for p, q in zip((dx, dz, dw, db), again))


def test_leading_axes_and_constant_rows(kda):
    x, z, w, _, _ = inputs(12, 2, 64, "f32", False, 3)
    a = kda.group_norm_fwd(x.view(3, 4, 2, 64), w, gate=z.view(3, 4, 2, 64))
    assert torch.equal(a.view(12, 2, 64), kda.group_norm_fwd(x, w, gate=z))
    x[:] = 5.0                                            # no variance: the centred norm is exactly zero
    assert float(kda.group_norm_fwd(x, w, activation="none", center=True).abs().max()) == 0
    x[:] = 0.0
    assert float(kda.group_norm_fwd(x, w, activation="none").abs().max()) == 0


def test_large_offset_loses_nothing_more(kda):
    """A mean 1000 times the deviation: the error stays that of the inputs' own magnitude."""
    x, _, w, b, _ = inputs(40, 3, 128, "f32", False, 5, offset=1000.0)
    out = kda.group_norm_fwd(x, w, bias=b, activation="none", center=True)
    want = R.group_norm(R.d(x), R.d(w), R.d(b), None, EPS, "none", True)
    R.within(out, want, R.group_norm_bound(R.d(x), R.d(w), R.d(b), None, EPS, "none", True), "out")


def test_extreme_gates_and_bad_rows(kda):
    x, z, w, _, _ = inputs(6, 2, 32, "f32", False, 7)
    z[0, 0] = float("inf")
    z[1, 0] = -1e30
    x[2, 1, 3] = float("nan")
    out = kda.group_norm_fwd(x, w, gate=z, activation="sigmoid")
    n = kda.group_norm_fwd(x, w, activation="none")
    assert torch.equal(out[0, 0], n[0, 0]) and float(out[1, 0].abs().max()) == 0
    bad = ~torch.isfinite(out)
    assert bool(bad[2, 1].all()) and int(bad.sum()) == 32


def test_no_rows(kda):
    w = torch.ones(64, device="cuda")
    x = torch.zeros(0, 4, 64, device="cuda")
    assert kda.group_norm_fwd(x, w).shape == (0, 4, 64)
    dx, _, dw, db = kda.group_norm_bwd(x, w, x, bias=w)
    assert dx.shape == (0, 4, 64) and float(dw.abs().sum()) == 0 and float(db.abs().sum()) == 0
    x = torch.zeros(3, 0, 64, device="cuda")
    assert kda.group_norm_fwd(x, w).shape == (3, 0, 64)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["sigmoid", "silu"])
@pytest.mark.parametrize("low,high", [(8.0, 20.0), (-20.0, -8.0), (-1.0, 1.0)])
@pytest.mark.parametrize("gated", [True, False])
def test_slopes_of_open_and_shut_gates(kda, gated, low, high, name, io):
    """Gradients through the flat parts of the activation, relative to the slope there.  An error of the slope: the
    exponential's (with its argument's, for bf16 I/O, |t| + 4 half steps; 4 for fp32), 1 + e, the
    reciprocal's, three products: under 40 half steps for |t| <= 21, which ROW, 64, covers.  n, where it
    is the argument, is off by ROW of what it is made of, and the slope by that share more."""
    M, G, d = 50, 3, 64
    x, _, w, b, dy = inputs(M, G, d, io, False, 77)
    g = torch.Generator().manual_seed(5)
    z = (low + (high - low) * torch.rand((M, G, d), generator=g)).to(R.IO[io]).cuda() if gated else None
    if not gated:                        # n in [low, high] but for a few outliers
        w, b = w * (high - low) / 8, b * 0 + (low + high) / 2
    kw = dict(eps=EPS, activation=name)
    got = kda.group_norm_bwd(x, w, dy, bias=b, gate=z, **kw)
    want = R.grads(lambda x, w, b, z: R.group_norm(x, w, b, z, EPS, name, False), [R.d(t) for t in (x, w, b, z)], R.d(dy))
    X, W, Y = R.d(x), R.d(w), R.d(dy)
    r = 1 / torch.sqrt((X ** 2).mean(-1, keepdim=True) + EPS)
    big = X.abs() * r * (1 + (X.abs() * r).mean(-1, keepdim=True))
    n, nb = X * r * W + R.d(b), big * W.abs() + R.d(b).abs()
    t = R.d(z) if gated else n
    s = torch.sigmoid(t)
    rest = torch.sigmoid(-t)
    slope = s * rest if name == "sigmoid" else s * (1 + t.abs() * rest)      # the magnitudes that SiLU's sums
    f = R.act(name, t).abs()
    dn = Y.abs() * (f if gated else slope * (1 + 2 * nb))                    # (its own slope is below 2 of it)
    if gated:
        R.within(got[1], want[3], 2 * R.ROW * Y.abs() * nb * slope, "dgate")
    c = dn * W.abs()
    R.within(got[0], want[0], 4 * R.ROW * r * (c + big * (c * big).mean(-1, keepdim=True)) * (1 + big), "dx")
    steps = 8 * R.ROW + (M * G + 64) * 2.0 ** -24
    R.within(got[2], want[1], steps * (dn * big).sum((0, 1)), "dweight")
    R.within(got[3], want[2], steps * dn.sum((0, 1)), "dbias")


def test_no_heads(kda):
    """Without heads the gradients of weights that they share are zero, not what the memory held."""
    for k in range(4):
        torch.full((64,), float("nan"), device="cuda")                # what a fresh tensor is made of next
        w = torch.ones(64, device="cuda")
        torch.full((64,), float("nan"), device="cuda")
        x = torch.zeros(3, 0, 64, device="cuda")
        dx, dz, dw, db = kda.group_norm_bwd(x, w, x, bias=w, gate=x)
        assert dx.shape == dz.shape == (3, 0, 64) and bool((dw == 0).all()) and bool((db == 0).all())
        w = torch.ones(0, 64, device="cuda")
        assert kda.group_norm_bwd(x, w, x)[2].shape == (0, 64)
