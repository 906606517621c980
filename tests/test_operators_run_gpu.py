"""The operators together, as a model uses them: a speculative decoding round on a state pool, a
recurrent layer's training step, the calls captured in CUDA graphs, on another stream."""
import os
import random
import subprocess
import sys

import pytest
import torch

import operators_ref as R
import workloads as W
from kda_testutil import TOL

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def kda(cuda_ok):
    from gated_delta_rule_75_b200 import build
    build.build()
    import gated_delta_rule_75_b200 as kda
    return kda


def test_speculative_decoding_round(kda):
    """Prompts prefilled into pool slots, a tree of drafts read over them and normed, one path of each
    committed, then a decode step: the step's output is that of the token sequence taken in order."""
    rng = random.Random(2)
    N, K, H, dd, P, lens = 3, 12, 2, 128, 5, [70, 64, 9]
    cfg = W.small_prefill(H=H, dk=dd, dv=dd, io_dtype="f32", seed=61, gate_shift=-2.0, lengths=lens)
    inp = W.make_prefill(cfg, "cuda")
    x, scale = R.tree_inputs(N, K, H, dd, dd, "f32", 62, P=P)
    pool = torch.zeros_like(x["state"])
    slots = torch.tensor([3, 0, 4], dtype=torch.int32, device="cuda")
    kda.chunk_fwd(inp["q"], inp["k"], inp["v"], inp["log_alpha"], inp["beta"], scale,
                  cu_seqlens=inp["cu_seqlens"], state_pool=pool, slots=slots)
    parents = [R.make_tree(rng, K, 5) for _ in range(N)]
    par = torch.tensor(parents, dtype=torch.int32, device="cuda")
    drafts = [x[m] for m in ("q", "k", "v", "log_alpha", "beta")]
    o = kda.tree_fwd(*drafts, pool, par, scale, slots=slots)
    weight, z = torch.rand(dd, device="cuda") + 0.5, torch.randn_like(o)
    y = kda.group_norm_fwd(o, weight, gate=z, activation="sigmoid")
    # fp64: the prompt's state by the token recurrence, then the trees
    S = torch.zeros(P, H, dd, dd, dtype=torch.float64)
    t0 = 0
    for n, L in enumerate(lens):
        tok = [R.d(inp[m][0, t0:t0 + L]) for m in ("k", "v", "log_alpha", "beta")]
        S[[3, 0, 4][n]] = R.tree_states(*tok, S[[3, 0, 4][n]], list(range(-1, L - 1)), L)[-1]
        t0 += L
    want = R.tree(*(R.d(t) for t in drafts), S, parents, scale, slots=[3, 0, 4])
    assert R.rel(o, want) <= 2 * TOL["f32"]
    assert R.rel(y, R.group_norm(want, R.d(weight), None, R.d(z), 1e-5, "sigmoid", False)) <= 4 * TOL["f32"]
    accepted = [rng.randrange(K) for _ in range(N)]
    kda.tree_commit(*drafts[1:], pool, par, torch.tensor(accepted, dtype=torch.int32, device="cuda"), slots=slots)
    S = R.tree_commit(*(R.d(t) for t in drafts[1:]), S, parents, accepted, slots=[3, 0, 4])
    assert R.rel(pool, S) <= 2 * TOL["f32"]
    nxt, _ = R.tree_inputs(N, 1, H, dd, dd, "f32", 63)
    c = [nxt[m][:, 0].contiguous() for m in ("q", "k", "v", "log_alpha", "beta")]
    got = kda.recurrent_step(*c, pool, scale, slots=slots)
    want = R.tree(*(R.d(nxt[m]) for m in ("q", "k", "v", "log_alpha", "beta")), S, [[-1]] * N, scale, slots=[3, 0, 4])
    assert R.rel(got, want[:, 0]) <= 2 * TOL["f32"]


def test_recurrent_layer_training_step(kda):
    """scan -> centred group norm with a gate, forward and backward, on packed sequences; the gradients
    of every input against reverse mode in fp64."""
    g = torch.Generator().manual_seed(9)
    cu, G, dd = [0, 90, 90, 231], 3, 32
    T, D = cu[-1], G * dd
    n = lambda *s: torch.randn(s, generator=g)
    x, la, h0 = n(1, T, D).cuda(), (-torch.rand((1, T, D), generator=g) * 0.3).cuda(), n(3, D).cuda()
    z, w, dy = n(1, T, G, dd).cuda(), (1 + 0.1 * n(G, dd)).cuda(), n(1, T, G, dd).cuda()
    dcu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    h, hT, starts = kda.glr_scan_fwd(x, la, h0=h0, cu_seqlens=dcu, output_starts=True)
    h4 = h.view(1, T, G, dd)
    y = kda.group_norm_fwd(h4, w, gate=z, activation="silu", center=True)
    dh, dz, dw, _ = kda.group_norm_bwd(h4, w, dy, gate=z, activation="silu", center=True)
    dx, dla, dh0 = kda.glr_scan_bwd(x, la, dh.view(1, T, D), starts=starts, h0=h0, cu_seqlens=dcu)

    def layer(x, la, h0, w, z):
        rows = []
        for s in range(3):
            c = h0[s]
            for t in range(cu[s], cu[s + 1]):
                c = torch.exp(la[0, t]) * c + x[0, t]
                rows.append(c)
        return R.group_norm(torch.stack(rows).view(1, T, G, dd), w, None, z, 1e-5, "silu", True)

    leaves = [R.d(t) for t in (x, la, h0, w, z)]
    want = R.grads(layer, leaves, R.d(dy))
    # a chain of two operators, each within a few ROW: relative norm, with the scan's sums of up to 100 terms
    for got, ref, what in zip((y, dx, dla, dh0, dw, dz), [layer(*leaves), *want], ("y", "dx", "dlog_a", "dh0", "dw", "dz")):
        assert R.rel(got, ref) <= 2e-5, what


CHILD = r"""
import sys, torch, random
sys.path[:0] = [ROOT, ROOT + "/tests"]
import operators_ref as R
import gated_delta_rule_75_b200 as kda

def i32(v): return torch.tensor(v, dtype=torch.int32, device="cuda")
torch.manual_seed(0)
N, K, H, d = 3, 10, 2, 128
x, scale = R.tree_inputs(N, K, H, d, d, "bf16", 1)
par = i32([R.make_tree(random.Random(n), K, 4) for n in range(N)])
acc = i32([3, 9, -1])
sx = torch.randn(2, 700, 72, device="cuda")
sl = -torch.rand(2, 700, 72, device="cuda")
w = torch.rand(36, device="cuda")

def round_(out):
    st = x["state"].clone()
    o = kda.tree_fwd(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], st, par, scale)
    kda.tree_commit(x["k"], x["v"], x["log_alpha"], x["beta"], st, par, acc)
    h, hT, starts = kda.glr_scan_fwd(sx, sl, output_starts=True)
    y = kda.group_norm_fwd(h.view(2, 700, 2, 36), w, gate=sx.view(2, 700, 2, 36))
    dh, dz, dw, _ = kda.group_norm_bwd(h.view(2, 700, 2, 36), w, y, gate=sx.view(2, 700, 2, 36))
    dx, dl, dh0 = kda.glr_scan_bwd(sx, sl, dh.view(2, 700, 72), starts=starts)
    dx2, _, _ = kda.glr_scan_bwd(sx, sl, dh.view(2, 700, 72))
    kda.glr_step(sx[:, 0].contiguous(), sl[:, 0].contiguous(), hT)
    for a, b in zip(out, (o, st, h, hT, y, dh, dz, dw, dx, dl, dh0, dx2)):
        a.copy_(b)

def fresh():
    return [torch.full(s, float("nan"), dtype=t, device="cuda") for s, t in shapes]

shapes = [((N, K, H, d), torch.bfloat16), (tuple(x["state"].shape), torch.float32), ((2, 700, 72), torch.float32),
          ((2, 72), torch.float32), ((2, 700, 2, 36), torch.float32), ((2, 700, 2, 36), torch.float32),
          ((2, 700, 2, 36), torch.float32), ((36,), torch.float32), ((2, 700, 72), torch.float32),
          ((2, 700, 72), torch.float32), ((2, 72), torch.float32), ((2, 700, 72), torch.float32)]
want = fresh()
round_(want)
torch.cuda.synchronize()
assert all(bool(torch.isfinite(t.float()).all()) for t in want)
side = torch.cuda.Stream()
side.wait_stream(torch.cuda.current_stream())
got = fresh()
with torch.cuda.stream(side):                       # another stream
    round_(got)
side.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want)), "another stream"
bufs = [fresh(), fresh()]
graphs = []
for b in bufs:                                       # two graphs, replayed in turn and at the same time
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        round_(b)
    graphs.append(g)
for rep in range(3):
    for b in bufs:
        for t in b:
            t.fill_(float("nan"))
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    graphs[0].replay()
    with torch.cuda.stream(side):
        graphs[1].replay()
    torch.cuda.synchronize()
    for b in bufs:
        assert all(torch.equal(p, q) for p, q in zip(b, want)), "replay %d" % rep
assert kda.get_error() == 0
print("operators ok")
"""


def test_other_stream_and_graphs(cuda_ok):
    from gated_delta_rule_75_b200 import build
    build.build()
    env = dict(os.environ)
    env.pop("KDA_DEBUG", None)
    r = subprocess.run([sys.executable, "-c", "ROOT = %r\n" % ROOT + CHILD], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "operators ok" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


CONCURRENT = r"""
import sys, torch
sys.path[:0] = [ROOT, ROOT + "/tests"]
import gated_delta_rule_75_b200 as kda
torch.manual_seed(3)
sets = []
for D, T in ((256, 20000), (200, 24000), (65, 9000)):
    x, la = torch.randn(1, T, D, device="cuda"), -torch.rand(1, T, D, device="cuda") * 0.2
    sets.append((x, la, torch.randn(1, T, D, device="cuda")))
def one(x, la, dout):
    h, hT, starts = kda.glr_scan_fwd(x, la, output_starts=True)
    return h, hT, *kda.glr_scan_bwd(x, la, dout, starts=starts)
want = [one(*s) for s in sets]
torch.cuda.synchronize()
streams = [torch.cuda.Stream() for _ in range(3)]
for rep in range(4):
    got = []
    for k in range(6):
        with torch.cuda.stream(streams[(k + rep) % 3]):
            got.append((k % 3, one(*sets[k % 3])))
    torch.cuda.synchronize()
    for i, g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want[i])), (rep, i)
assert kda.get_error() == 0
print("streams ok")
"""


def test_scans_on_several_streams_at_once(cuda_ok):
    """Scans whose tiles wait on one another, each wanting every SM, issued on three streams together:
    all end, with the results of running them one after another."""
    from gated_delta_rule_75_b200 import build
    build.build()
    env = dict(os.environ)
    env.pop("KDA_DEBUG", None)
    r = subprocess.run([sys.executable, "-c", "ROOT = %r\n" % ROOT + CONCURRENT], env=env, capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0 and "streams ok" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


def test_strong_decays_and_repeated_offsets(cuda_ok, kda):
    """Decays from none to e^-100 in one tensor, sequences of one token, many empty ones in a row."""
    lens = [1] * 5 + [0] * 200 + [64, 0, 63, 1, 129] + [0] * 40 + [700]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    g = torch.Generator().manual_seed(17)
    T, D = cu[-1], 72
    x = torch.randn((1, T, D), generator=g).cuda()
    la = (-100 * torch.rand((1, T, D), generator=g) ** 4).cuda()
    h0 = torch.randn((len(lens), D), generator=g).cuda()
    dcu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out, hT, starts = kda.glr_scan_fwd(x, la, h0=h0, cu_seqlens=dcu, output_starts=True)
    H, want, E, eT = R.glr(R.d(x), R.d(la), R.d(h0), cu)
    R.within(out, H, E, "out")
    R.within(hT, want, eT, "hT")
    dx, dla, dh0 = kda.glr_scan_bwd(x, la, x, starts=starts, h0=h0, dhT=h0, cu_seqlens=dcu)
    want = R.glr_grads(R.d(x), R.d(la), R.d(h0), R.d(x), R.d(h0), cu)
    R.within(dx, want[0], want[3], "dx")
    R.within(dla, want[1], want[4], "dlog_a")
    R.within(dh0, want[2], want[5], "dh0")
