"""Refusals of the gated linear recurrence, the drafted token trees and the group norm, on the
host (no GPU), and the fp64 gradient formulas their GPU tests use, against differences."""
import ctypes
import random

import pytest
import torch

import operators_ref as R

FAKE = 0x7f0000000000   # never dereferenced: the checks run before anything is launched
GAP = 1 << 32           # distance between fake tensors


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_75_b200 import build
    build.build()
    import gated_delta_rule_75_b200 as kda
    return kda._load()


def at(i, off=0):
    return FAKE + i * GAP + off


def test_header_constants_match_the_binding():
    import re
    import os
    import gated_delta_rule_75_b200 as kda
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kda.h")).read()
    value = lambda n: int(re.search(r"#define %s (\d+)" % n, src).group(1))
    assert value("KDA_GLR_TILE") == kda.GLR_TILE and value("KDA_TREE_MAX_NODES") == kda.TREE_MAX_NODES


def scan(lib, x=at(0), g=at(1), h0=None, out=at(2), hT=None, starts=None, cu=None, B=2, T=100, D=64, io=1):
    return lib.kda_glr_scan_fwd(x, g, h0, out, hT, starts, cu, B, T, D, io, None)


def scan_bwd(lib, x=at(0), g=at(1), h0=None, starts=at(2), dout=at(3), dhT=None, dx=at(4), dg=at(5), dh0=None,
             cu=None, B=2, T=100, D=64, io=1):
    return lib.kda_glr_scan_bwd(x, g, h0, starts, dout, dhT, dx, dg, dh0, cu, B, T, D, io, None)


def test_scan_argument_errors(lib):
    BAD, UNS, OK = 1, 2, 0
    assert scan(lib, B=-1) == BAD and scan(lib, T=-1) == BAD and scan(lib, D=-1) == BAD
    assert scan(lib, io=2) == UNS and scan(lib, D=(1 << 20) + 1) == UNS
    assert scan(lib, B=1 << 30, T=1 << 30) == UNS and scan(lib, T=1 << 62) == UNS
    assert scan(lib, x=None) == BAD and scan(lib, g=None) == BAD and scan(lib, out=None) == BAD
    assert scan(lib, x=at(0, 2)) == BAD and scan(lib, g=at(1, 4)) == BAD and scan(lib, hT=at(3, 8)) == BAD
    assert scan(lib, starts=at(3, 4)) == BAD and scan(lib, cu=at(3, 2)) == BAD
    assert scan(lib, cu=at(3), B=0) == BAD
    assert scan(lib, out=at(0)) == BAD and scan(lib, out=at(1, 1024)) == BAD          # over x, inside log_a
    assert scan(lib, hT=at(2, 64)) == BAD and scan(lib, starts=at(2)) == BAD
    assert scan(lib, h0=at(3), hT=at(3, 256)) == BAD                                   # half over h0
    assert scan(lib, T=0, h0=at(3), hT=at(3, 256)) == BAD                              # without tokens too
    assert scan(lib, B=0) == OK and scan(lib, D=0) == OK
    assert lib.kda_glr_scan_fwd_slots(at(0), at(1), at(2), None, at(3), None, None, 2, 100, 4, 64, 1, None) == BAD
    assert lib.kda_glr_scan_fwd_slots(at(0), at(1), None, at(4), at(3), None, None, 2, 100, 4, 64, 1, None) == BAD
    assert lib.kda_glr_scan_fwd_slots(at(0), at(1), at(2), at(4), at(3), None, None, 2, 100, -1, 64, 1, None) == BAD


def test_scan_backward_argument_errors(lib):
    BAD, UNS, OK = 1, 2, 0
    assert scan_bwd(lib, B=-1) == BAD and scan_bwd(lib, io=5) == UNS and scan_bwd(lib, D=1 << 21) == UNS
    for name in ("x", "g", "dout", "dx", "dg"):
        assert scan_bwd(lib, **{name: None}) == BAD, name
        assert scan_bwd(lib, **{name: at(9, 4)}) == BAD, name
    assert scan_bwd(lib, dx=at(3)) == BAD and scan_bwd(lib, dg=at(1)) == BAD and scan_bwd(lib, dx=at(5)) == BAD
    assert scan_bwd(lib, dh0=at(6, 4)) == BAD and scan_bwd(lib, dh0=at(4)) == BAD
    assert scan_bwd(lib, dhT=at(6), dh0=at(6, 128)) == BAD and scan_bwd(lib, dhT=at(6), dh0=at(6)) == BAD
    assert scan_bwd(lib, T=0, dhT=at(6), dh0=at(6, 128)) == BAD
    assert scan_bwd(lib, cu=at(6), B=0) == BAD and scan_bwd(lib, B=0) == OK


def test_step_argument_errors(lib):
    step = lambda x=at(0), g=at(1), s=at(2), out=at(3), N=4, D=64, io=1: lib.kda_glr_step(x, g, s, out, N, D, io, None)
    assert step(N=-1) == 1 and step(io=9) == 2 and step(D=1 << 21) == 2
    assert step(s=None) == 1 and step(out=at(2)) == 1 and step(x=at(0, 8)) == 1 and step(out=at(0)) == 1
    assert step(N=0) == 0 and step(D=0) == 0
    assert lib.kda_glr_step_slots(at(0), at(1), at(2), None, at(3), 4, 8, 64, 1, None) == 1
    assert lib.kda_glr_step_slots(at(0), at(1), at(2), at(4, 2), at(3), 4, 8, 64, 1, None) == 1


def tree(lib, q=at(0), k=at(1), v=at(2), g=at(3), b=at(4), s=at(5), slots=None, par=at(6), nodes=None, out=at(7),
         N=2, P=4, K=8, H=2, dk=128, dv=64, io=1):
    return lib.kda_tree_fwd(q, k, v, g, b, s, slots, par, nodes, out, N, P, K, H, dk, dv, ctypes.c_float(1), io, None)


def commit(lib, k=at(1), v=at(2), g=at(3), b=at(4), s=at(5), slots=None, par=at(6), acc=at(7),
           N=2, P=4, K=8, H=2, dk=128, dv=64, io=1):
    return lib.kda_tree_commit(k, v, g, b, s, slots, par, acc, N, P, K, H, dk, dv, io, None)


def test_tree_argument_errors(lib):
    for call in (tree, commit):
        assert call(lib, K=65) == 2 and call(lib, dk=96) == 2 and call(lib, dv=32) == 2 and call(lib, io=3) == 2
        assert call(lib, N=-1) == 1 and call(lib, K=-1) == 1 and call(lib, H=-1) == 1
        assert call(lib, N=1 << 20, H=1 << 20) == 2
        for name in ("k", "v", "g", "s"):
            assert call(lib, **{name: None}) == 1 and call(lib, **{name: at(9, 8)}) == 1, name
        for name in ("b", "par"):
            assert call(lib, **{name: None}) == 1 and call(lib, **{name: at(9, 2)}) == 1, name
        assert call(lib, slots=at(9, 1)) == 1 and call(lib, slots=at(9), P=-1) == 1
        assert call(lib, N=0) == 0 and call(lib, H=0) == 0 and call(lib, K=0) == 0
    assert tree(lib, q=None) == 1 and tree(lib, out=at(2)) == 1 and tree(lib, out=at(5, 4096)) == 1
    assert tree(lib, nodes=at(9, 2)) == 1
    assert commit(lib, acc=None) == 1 and commit(lib, s=at(2)) == 1 and commit(lib, acc=at(9, 3)) == 1


def test_group_norm_argument_errors(lib):
    def fwd(x=at(0), z=at(1), w=at(2), b=None, out=at(3), M=4, G=2, dd=64, eps=1e-5, act=1, io=1):
        return lib.kda_group_norm_fwd(x, z, w, b, out, M, G, dd, 0, 0, ctypes.c_float(eps), act, io, None)

    def bwd(x=at(0), z=at(1), w=at(2), b=None, dy=at(3), dx=at(4), dz=at(5), dw=at(6), db=None, M=4, G=2, dd=64,
            eps=1e-5, act=1, io=1):
        return lib.kda_group_norm_bwd(x, z, w, b, dy, dx, dz, dw, db, M, G, dd, 0, 0, ctypes.c_float(eps), act, io, None)

    for call in (fwd, bwd):
        assert call(M=-1) == 1 and call(G=-1) == 1 and call(dd=0) == 1 and call(act=3) == 1 and call(act=-1) == 1
        assert call(eps=0.0) == 1 and call(eps=-1.0) == 1 and call(eps=float("nan")) == 1 and call(eps=float("inf")) == 1
        assert call(dd=513) == 2 and call(io=2) == 2 and call(G=65536) == 2
        assert call(x=None) == 1 and call(x=at(0, 8)) == 1 and call(w=at(2, 4)) == 1 and call(z=at(1, 2)) == 1
        assert call(G=0) == 0
    assert fwd(out=at(0)) == 1 and fwd(out=at(1)) == 1 and fwd(out=None) == 1 and fwd(M=0) == 0
    assert bwd(dz=None) == 1 and bwd(z=None) == 1 and bwd(dx=at(3)) == 1 and bwd(dx=at(5)) == 1 and bwd(dw=at(2)) == 1


def test_python_binding_checks_on_host():
    import gated_delta_rule_75_b200 as kda
    x = torch.zeros(2, 8, 16)
    for bad in (lambda: kda.glr_scan_fwd(x, x[:, :4]), lambda: kda.glr_scan_fwd(x[0], x[0]),
                lambda: kda.glr_scan_fwd(x, x, h0=torch.zeros(3, 16)),
                lambda: kda.glr_scan_fwd(x, x, cu_seqlens=torch.tensor([0, 8], dtype=torch.int32)),
                lambda: kda.glr_scan_fwd(x[:1], x[:1], cu_seqlens=torch.tensor([0, 8])),
                lambda: kda.glr_scan_fwd(x.transpose(1, 2), x.transpose(1, 2)),
                lambda: kda.glr_scan_fwd(x, x, slots=torch.zeros(2, dtype=torch.int32)),
                lambda: kda.glr_scan_fwd(x, x, state_pool=torch.zeros(2, 16)),
                lambda: kda.glr_scan_bwd(x, x, x, starts=torch.zeros(2, 2, 16)),
                lambda: kda.glr_scan_fwd(x, x),                       # not on a CUDA device
                lambda: kda.glr_step(x[0], x[0], torch.zeros(7, 16)),
                lambda: kda.group_norm_fwd(x, torch.ones(8)), lambda: kda.group_norm_fwd(x, activation="tanh"),
                lambda: kda.group_norm_fwd(x, torch.ones(8, 16), bias=torch.ones(16)),
                lambda: kda.group_norm_bwd(x, None, x[:1]), lambda: kda.group_norm_fwd(x, torch.ones(16))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        kda.glr_scan_fwd(x.double(), x)
    with pytest.raises(TypeError):
        kda.glr_scan_fwd(x, x.double())
    with pytest.raises(TypeError):
        kda.group_norm_fwd(x.half())
    k, g, b = torch.zeros(2, 4, 1, 64), torch.zeros(2, 4, 1, 64), torch.zeros(2, 4, 1)
    S, par = torch.zeros(2, 1, 64, 64), torch.zeros(2, 4, dtype=torch.int32)
    for bad in (lambda: kda.tree_fwd(k, k, k, g, b, S, par[:1], 1.0), lambda: kda.tree_fwd(k[:1], k, k, g, b, S, par, 1.0),
                lambda: kda.tree_fwd(k, k, k, g, b, S[:1], par, 1.0), lambda: kda.tree_fwd(k, k, k, g, b, S, par, 1.0),
                lambda: kda.tree_fwd(k, k, k, g, b, S, par, 1.0, num_nodes=par[0]),
                lambda: kda.tree_commit(k, k, g, b, S, par, par)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        kda.tree_fwd(k, k, k, g, b, S, par.long(), 1.0)


def test_gradient_formulas_against_differences():
    """The fp64 gradients that the GPU tests compare with: the reverse recurrence of the scan and
    reverse mode through the norm, along random directions, against central differences (step e: the
    truncation is e^2 of third derivatives of order 1, the rounding 2^-52 / e)."""
    torch.manual_seed(5)
    D, cu, e = 3, [0, 4, 4, 9], 1e-5
    x, la, h0 = torch.randn(1, 9, D).double(), -torch.rand(1, 9, D).double(), torch.randn(3, D).double()
    dout, dhT = torch.randn(1, 9, D).double(), torch.randn(3, D).double()

    def loss(x, la, h0):
        H, hT, _, _ = R.glr(x, la, h0, cu)
        return float((H * dout).sum() + (hT * dhT).sum())

    g = R.glr_grads(x, la, h0, dout, dhT, cu)[:3]
    for i in range(3):
        v = [torch.randn_like(t) * (j == i) for j, t in enumerate((x, la, h0))]
        up = loss(*(t + e * w for t, w in zip((x, la, h0), v)))
        down = loss(*(t - e * w for t, w in zip((x, la, h0), v)))
        want = float((g[i] * v[i]).sum())
        assert abs((up - down) / (2 * e) - want) <= 1e-7 * (1 + abs(want)), i
    for name, center, gated in (("silu", True, True), ("sigmoid", False, True), ("silu", False, False)):
        t = [torch.randn(5, 2, 7).double(), torch.randn(7).double(), torch.randn(7).double(),
             torch.randn(5, 2, 7).double() if gated else None]
        dy = torch.randn(5, 2, 7).double()
        f = lambda x, w, b, z: R.group_norm(x, w, b, z, 1e-5, name, center)
        g = R.grads(f, t, dy)
        for i in range(4):
            if t[i] is None:
                continue
            v = torch.randn_like(t[i])
            move = lambda s: [y + s * v if j == i else y for j, y in enumerate(t)]
            diff = float(((f(*move(e)) - f(*move(-e))) * dy).sum()) / (2 * e)
            want = float((g[i] * v).sum())
            assert abs(diff - want) <= 1e-6 * (1 + abs(want)), (name, i)


def test_tree_formula_against_one_path():
    """The reference tree on a chain equals the token recurrence, and on a fork each branch does."""
    rng = random.Random(3)
    x, scale = R.tree_inputs(1, 6, 2, 64, 64, "f32", 4, device="cpu")
    x = {m: t.double() for m, t in x.items()}
    parents = R.make_tree(rng, 6, 4)
    out = R.tree(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["state"], [parents], scale)
    for i in range(6):
        path, j = [], i
        while j >= 0:
            path, j = [j] + path, parents[j]
        S = x["state"][0]
        for j in path:
            S = torch.exp(x["log_alpha"][0, j])[:, :, None] * S
            err = x["beta"][0, j][:, None] * (x["v"][0, j] - (x["k"][0, j][:, :, None] * S).sum(1))
            S = S + x["k"][0, j][:, :, None] * err[:, None]
        torch.testing.assert_close(out[0, i], scale * (x["q"][0, i][:, :, None] * S).sum(1))


def test_import_without_cuda_in_torch():
    """The package and its modules import where torch was built without CUDA (names of its CUDA bindings are
    missing there); only calls raise."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import sys; sys.path.insert(0, %r)\n"
            "import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda_')]:\n"
            "    delattr(torch._C, name)\n"
            "import gated_delta_rule_75_b200 as kda\n"
            "import gated_delta_rule_75_b200.context_parallel\n"
            "x = torch.zeros(1, 4, 8)\n"
            "try:\n    kda.glr_scan_fwd(x, x)\n"
            "except ValueError as e:\n    assert 'CUDA device' in str(e)\n    print('raised')\n" % root)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "raised" in r.stdout, r.stderr[-1500:]
