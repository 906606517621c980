"""Plain fp64 forms of the gated linear recurrence, the drafted token tree and the group
norm, token by token, with bounds on what fp32 arithmetic may add.  Test helpers."""
import math

import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}    # rounding to nearest
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def d(t):
    return None if t is None else t.detach().cpu().double()


def spans(B, T, cu):
    """(row, first token, past the last, sequence) of every sequence."""
    if cu is None:
        return [(b, 0, T, b) for b in range(B)]
    return [(0, cu[n], cu[n + 1], n) for n in range(len(cu) - 1)]


# One step of the recurrence in fp32: the exponential is within an ulp (2 half steps), the running
# product, the local sum, the fold over tiles and the final fma round once each: 6 half steps, here 8.
STEP = 8 * 2.0 ** -24


def glr(x, log_a, h0, cu=None):
    """h, hT, and bounds on the fp32 error of both: an error already there decays with the state, and
    every step adds at most STEP of the magnitudes it sums."""
    B, T, D = x.shape
    N = B if cu is None else len(cu) - 1
    h0 = torch.zeros(N, D, dtype=torch.float64) if h0 is None else h0
    a = torch.exp(log_a)
    H, E = torch.zeros_like(x), torch.zeros_like(x)
    hT, eT = h0.clone(), torch.zeros_like(h0)
    for b, t0, t1, n in spans(B, T, cu):
        h, m, e = h0[n].clone(), h0[n].abs(), torch.zeros(D, dtype=torch.float64)
        for t in range(t0, t1):
            h = a[b, t] * h + x[b, t]
            m = a[b, t] * m + x[b, t].abs()
            e = a[b, t] * e + STEP * m
            H[b, t], E[b, t] = h, e
        hT[n], eT[n] = h, e
    return H, hT, E, eT


def glr_grads(x, log_a, h0, dout, dhT, cu=None):
    """dx, dlog_a, dh0 and bounds on their fp32 errors."""
    B, T, D = x.shape
    H, hT, E, _ = glr(x, log_a, h0, cu)
    N = hT.shape[0]
    h0 = torch.zeros(N, D, dtype=torch.float64) if h0 is None else h0
    a = torch.exp(log_a)
    dx, dla, eg, el = (torch.zeros_like(x) for _ in range(4))
    dh0 = torch.zeros_like(h0) if dhT is None else dhT.clone()
    e0 = torch.zeros_like(h0)
    for b, t0, t1, n in spans(B, T, cu):
        g, m, e = dh0[n].clone(), dh0[n].abs(), torch.zeros(D, dtype=torch.float64)
        for t in range(t1 - 1, t0 - 1, -1):
            g, m = g + dout[b, t], m + dout[b, t].abs()
            e = e + STEP * m
            dx[b, t], eg[b, t] = g, e
            before, eb = (H[b, t - 1], E[b, t - 1]) if t > t0 else (h0[n], torch.zeros_like(e))
            dla[b, t] = g * a[b, t] * before
            el[b, t] = a[b, t] * (e * before.abs() + g.abs() * eb + e * eb) + STEP * dla[b, t].abs()
            g, m, e = a[b, t] * g, a[b, t] * m, a[b, t] * e
        dh0[n], e0[n] = g, e
    return dx, dla, dh0, eg, el, e0 + STEP * dh0.abs()


def within(got, want, bound, what):
    """|got - want| <= bound plus half a step of got's type, element by element; tiny values of a type
    with few bits may fall below its normal range."""
    step = HALF_STEP[got.dtype]
    g = d(got)
    off = (g - want).abs() - (bound + step * (want.abs() + bound) + 1e-37)
    assert torch.isfinite(g).equal(torch.isfinite(want)), what
    assert float(off.max() if off.numel() else -1) <= 0, (what, float(off.max()), int(off.argmax()))


# ---------------------------------------------------------------- trees

def tree_states(k, v, log_alpha, beta, S0, parents, live):
    """States of every live node of one sequence, [H, dk, dv] each, fp64."""
    S = []
    a = torch.exp(log_alpha)
    for i in range(live):
        p = int(parents[i])
        X = a[i][:, :, None] * (S0 if p < 0 else S[p])
        err = beta[i][:, None] * (v[i] - torch.einsum("hc,hcd->hd", k[i], X))
        S.append(X + k[i][:, :, None] * err[:, None, :])
    return S


def tree(q, k, v, log_alpha, beta, state, parents, scale, num_nodes=None, slots=None):
    """Outputs [N, K, H, dv] of all nodes, zero past num_nodes."""
    N, K, H, dk = k.shape
    out = torch.zeros_like(v)
    for n in range(N):
        row = n if slots is None else slots[n]
        S0 = state[row] if 0 <= row < state.shape[0] else torch.zeros_like(state[0])
        S = tree_states(k[n], v[n], log_alpha[n], beta[n], S0, parents[n], K if num_nodes is None else num_nodes[n])
        for i, s in enumerate(S):
            out[n, i] = scale * torch.einsum("hc,hcd->hd", q[n, i], s)
    return out


def tree_commit(k, v, log_alpha, beta, state, parents, accepted, slots=None):
    state = state.clone()
    for n in range(k.shape[0]):
        row = n if slots is None else slots[n]
        if not 0 <= row < state.shape[0] or not 0 <= accepted[n] < k.shape[1]:
            continue
        S = tree_states(k[n], v[n], log_alpha[n], beta[n], state[row], parents[n], accepted[n] + 1)
        state[row] = S[accepted[n]]
    return state


# ---------------------------------------------------------------- group norm

def act(name, z):
    s = torch.sigmoid(z)
    return {"none": z, "sigmoid": s, "silu": z * s}[name]


def group_norm(x, w, b, gate, eps, name, center):
    mu = x.mean(-1, keepdim=True) if center else torch.zeros_like(x[..., :1])
    r = 1 / torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + eps)
    n = (x - mu) * r
    n = n if w is None else n * w
    n = n if b is None else n + b
    return act(name, n) if gate is None else n * act(name, gate)


# Sums over a row: at most 16 elements in a lane, then five rounds over lanes: 21 half steps of the
# magnitudes; with the mean's own error, the square root and the products, under 64 half steps.
ROW = 64 * 2.0 ** -24


def group_norm_bound(x, w, b, gate, eps, name, center):
    """Bound on the fp32 error of group_norm: ROW of the magnitudes that make up n, through an
    activation whose slope is at most 1.1 (1 + |n| for the product with a gate's activation)."""
    mu = x.mean(-1, keepdim=True) if center else torch.zeros_like(x[..., :1])
    r = 1 / torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + eps)
    big = (x.abs() + (x.abs().mean(-1, keepdim=True) if center else 0)) * r
    # an error of the mean also shifts the variance, by no more than the same share
    big = big + big.mean(-1, keepdim=True) * (x - mu).abs() * r
    big = big * (1 if w is None else w.abs()) + (0 if b is None else b.abs())
    if gate is None:
        return 1.1 * ROW * big + ROW * act(name, big).abs()
    return 2 * ROW * big * act(name, gate).abs()


def grads(f, inputs, dout):
    """Gradients of sum(dout * f(inputs)) in fp64 by reverse mode; None stays None."""
    leaves = [None if t is None else t.clone().requires_grad_(True) for t in inputs]
    (f(*leaves) * dout).sum().backward()
    return [None if t is None else t.grad for t in leaves]


def rel(got, want):
    return float((d(got) - want).norm() / max(float(want.norm()), 1e-300))


def make_tree(rng, K, deep):
    """Parents of K nodes with paths of at most `deep` nodes."""
    parents, depth = [], []
    for i in range(K):
        open_ = [j for j in range(i) if depth[j] < deep]
        p = rng.choice(open_) if open_ and rng.random() < 0.85 else -1
        parents.append(p)
        depth.append(1 if p < 0 else depth[p] + 1)
    return parents


def tree_inputs(N, K, H, dk, dv, io, seed, P=None, shift=-2.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)
    q, k = n(N, K, H, dk), n(N, K, H, dk)
    x = {"q": (q / q.norm(dim=-1, keepdim=True)).to(IO[io]), "k": (k / k.norm(dim=-1, keepdim=True)).to(IO[io]),
         "v": n(N, K, H, dv).to(IO[io]),
         "log_alpha": -torch.nn.functional.softplus(n(N, K, H, dk) + shift), "beta": torch.sigmoid(n(N, K, H)),
         "state": n(P or N, H, dk, dv) * 0.1}
    return {m: t.to(device) for m, t in x.items()}, 1 / math.sqrt(dk)
