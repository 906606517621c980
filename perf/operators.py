"""Cases for the operators around the delta rule: the gated linear recurrence (scan, its
gradients, its decode step), drafted token trees over cached states, and the gated group norm.

run() takes a prepared state through one pass, in plain torch operations, or through the
library's own entry points where `own` is true; exact() gives the same outputs in 64 bits."""
import math
import random

import torch

own = False

_T = {"f32": torch.float32, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "bf16": 2}

# Widths are H * d of the library's own workloads (32 heads of 128, 16 of 128, 2 of 64) or
# generic ones; lengths are those of its prefill and packed workloads, or odd ones.
_LISTED = [
    # the batched prefill's shape through a recurrent layer: 8 sequences of 8192 tokens
    {"name": "scan_batched_bf16", "op": "scan", "B": 8, "T": 8192, "D": 4096, "N": 0, "io": "bf16"},
    # one long document, fp32, few channels: the whole length has to be cut to fill the GPU
    {"name": "scan_long_f32", "op": "scan", "B": 1, "T": 131071, "D": 1024, "N": 0, "io": "f32"},
    # packed prompts of odd lengths, some empty, a width that no power of two divides
    {"name": "scan_packed_bf16", "op": "scan", "B": 1, "T": 30011, "D": 1000, "N": 37, "io": "bf16"},
    # a training step of the recurrence: forward, then the gradients of every input
    {"name": "scan_train_bf16", "op": "scan_train", "B": 4, "T": 8192, "D": 4096, "N": 0, "io": "bf16"},
    # one decoded token for each of 256 running requests, states in a pool
    {"name": "scan_step_pool", "op": "scan_step", "N": 256, "D": 4096, "io": "bf16"},
    # one request whose drafter proposed 8 tokens: latency
    {"name": "tree_one_request", "op": "tree", "N": 1, "K": 8, "H": 32, "dk": 128, "dv": 128, "deep": 8, "io": "bf16"},
    # a served batch, 16 drafted tokens each
    {"name": "tree_batch", "op": "tree", "N": 64, "K": 16, "H": 32, "dk": 128, "dv": 128, "deep": 6, "io": "bf16"},
    # wide trees, nearly the most nodes, deep paths
    {"name": "tree_wide", "op": "tree", "N": 40, "K": 61, "H": 32, "dk": 128, "dv": 128, "deep": 12, "io": "bf16"},
    # the accepted paths of the served batch go into the pool
    {"name": "tree_commit_batch", "op": "tree_commit", "N": 64, "K": 16, "H": 32, "dk": 128, "dv": 128, "deep": 6, "io": "bf16"},
    # the output norm and gate of the batched prefill
    {"name": "norm_batched_bf16", "op": "norm", "M": 65536, "G": 32, "d": 128, "act": "sigmoid", "center": False,
     "per_group": False, "gate": True, "io": "bf16"},
    # the same at one decoded token for each of 64 requests: latency
    {"name": "norm_decode", "op": "norm", "M": 64, "G": 32, "d": 128, "act": "silu", "center": False,
     "per_group": False, "gate": True, "io": "bf16"},
    # gradients of a centred norm with weights of every head, odd row count, fp32
    {"name": "norm_grad_f32", "op": "norm_grad", "M": 20011, "G": 16, "d": 128, "act": "silu", "center": True,
     "per_group": True, "gate": True, "io": "f32"},
]


def listed():
    return [dict(c) for c in _LISTED]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_train", "scan_step", "tree", "tree", "tree_commit", "norm", "norm_grad"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op in ("scan", "scan_train"):
        most = (1 << 27) if op == "scan" else (1 << 26)
        D = _log(rng, 32, 4096)
        T = _log(rng, 1, max(1, min(131072, most // D)))
        B = _log(rng, 1, max(1, min(16, most // (D * T))))
        N = 0
        if rng.random() < 0.5:
            T, B, N = min(B * T, 131072), 1, rng.randint(1, 64)
        return {"op": op, "B": B, "T": T, "D": D, "N": N, "io": io}
    if op == "scan_step":
        return {"op": op, "N": _log(rng, 1, 2048), "D": _log(rng, 64, 8192), "io": io}
    if op in ("tree", "tree_commit"):
        K, H = _log(rng, 1, 64), rng.choice([1, 3, 8, 16, 32])
        N = _log(rng, 1, max(1, min(128, 75000 // (K * H))))
        return {"op": op, "N": N, "K": K, "H": H, "dk": rng.choice([64, 128]), "dv": rng.choice([64, 128]),
                "deep": rng.randint(1, 16), "io": io}
    d = rng.choice([32, 64, 80, 100, 128, 192, 256, 512])
    G = _log(rng, 1, 64)
    most = (1 << 28) if op == "norm" else (1 << 25)
    return {"op": op, "M": _log(rng, 1, min(65536, most // (G * d))), "G": G, "d": d,
            "act": rng.choice(["none", "sigmoid", "silu"]), "center": rng.random() < 0.5,
            "per_group": rng.random() < 0.5, "gate": rng.random() < 0.8, "io": io}


# ---------------------------------------------------------------- inputs

def _lengths(rng, total, n):
    """n lengths of very different sizes that sum to `total`; some may be empty."""
    w = [rng.expovariate(1.0) ** 2 * (rng.random() > 0.1) + 1e-9 for _ in range(n)]
    lens = [int(total * x / sum(w)) for x in w]
    lens[max(range(n), key=lambda i: w[i])] += total - sum(lens)
    return lens


def _tree(rng, K, deep):
    """Parents of K drafted nodes (-1: the cached state), no path longer than `deep` nodes where K allows."""
    parents, depth = [], []
    for i in range(K):
        open_ = [j for j in range(max(0, i - 12), i) if depth[j] < deep]
        p = rng.choice(open_) if open_ and rng.random() < 0.9 else -1
        parents.append(p)
        depth.append(1 if p < 0 else depth[p] + 1)
    return parents


def prepare(case, seed):
    rng = random.Random(seed)
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, io = case["op"], _T[case["io"]]
    s = dict(case)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    if op in ("scan", "scan_train", "scan_step"):
        D = case["D"]
        shape = (case["N"], D) if op == "scan_step" else (case["B"], case["T"], D)
        # decays from near 1 (long memory) to about 0.7; the input keeps the state near unit variance
        s["log_a"] = normal(*shape).sub_(4).exp_().log1p_().neg_()
        s["x"] = (normal(*shape) * (1 - torch.exp(2 * s["log_a"])).sqrt_()).to(io)
        if op == "scan_step":
            P = case["N"] + 3
            s["pool"] = normal(P, D)
            s["slots"] = ints(rng.sample(range(P), case["N"]))
            return s
        n = case["N"] or case["B"]
        s["h0"] = normal(n, D)
        s["cu"] = None
        if case["N"]:
            cu = [0]
            for x in _lengths(rng, case["T"], case["N"]):
                cu.append(cu[-1] + x)
            s["cu"] = ints(cu)
        if op == "scan_train":
            s["dout"] = normal(*shape).to(io)
            s["dhT"] = normal(n, D)
        return s
    if op in ("tree", "tree_commit"):
        N, K, H, dk, dv = (case[k] for k in ("N", "K", "H", "dk", "dv"))
        q, k = normal(N, K, H, dk), normal(N, K, H, dk)
        s["q"] = (q / q.norm(dim=-1, keepdim=True)).to(io)
        s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(io)
        s["v"] = normal(N, K, H, dv).to(io)
        s["log_alpha"] = -torch.nn.functional.softplus(normal(N, K, H, dk) - 2)
        s["beta"] = torch.sigmoid(normal(N, K, H))
        P = N + 2
        s["pool"] = normal(P, H, dk, dv) * 0.1
        s["slots"] = ints(rng.sample(range(P), N))
        s["parents"] = ints([_tree(rng, K, case["deep"]) for _ in range(N)])
        nodes = [rng.randint(max(1, (3 * K) // 4), K) for _ in range(N)]   # drafts end early here and there
        s["nodes"] = ints(nodes)
        s["accepted"] = ints([rng.randrange(n) for n in nodes])
        s["out"] = torch.zeros((N, K, H, dv), dtype=io, device=dev)
        s["scale"] = 1 / math.sqrt(dk)
        return s
    M, G, d = case["M"], case["G"], case["d"]
    s["x"] = (normal(M, G, d) * 0.5 + (0.3 * normal(1, G, d) if case["center"] else 0)).to(io)
    s["z"] = normal(M, G, d).to(io) if case["gate"] else None
    shape = (G, d) if case["per_group"] else (d,)
    s["weight"] = 1 + 0.1 * normal(*shape)
    s["bias"] = 0.1 * normal(*shape) if case["center"] else None
    s["dout"] = normal(M, G, d).to(io) if op == "norm_grad" else None
    return s


# ---------------------------------------------------------------- plain forms

def _starts(s):
    """First token of every sequence that has one, and which sequence that is, on the packed axis."""
    n = s["h0"].shape[0]
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(n + 1, device=s["x"].device) * s["T"]
    full = (cu[1:] > cu[:-1]).nonzero()[:, 0]
    return cu, full


def _doubling(a, h):
    """h_t <- a_t h_{t-1} + h_t over the first axis, by doubling the span that each row covers."""
    span = 1
    while span < h.shape[0]:
        h = torch.cat([h[:span], h[span:] + a[span:] * h[:-span]])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return h


def _scan_plain(s):
    D = s["D"]
    x, a = s["x"].to(torch.float32, copy=True).reshape(-1, D), torch.exp(s["log_a"]).reshape(-1, D)
    cu, full = _starts(s)
    first, last = cu[:-1][full], cu[1:][full] - 1
    cut = a.clone()
    cut[first] = 0                              # nothing crosses into a sequence
    x[first] = x[first] + a[first] * s["h0"][full]
    h = _doubling(cut, x)
    hT = s["h0"].clone()
    hT[full] = h[last]
    return a, cut, h, hT, first, last, full


def _plain_scan(s):
    a, cut, h, hT, first, last, full = _scan_plain(s)
    out = h.to(s["x"].dtype).view_as(s["x"])
    if s["op"] == "scan":
        return [out, hT]
    D = s["D"]
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = s["h0"][full]
    del h
    g = s["dout"].float().reshape(-1, D).clone()
    g[last] = g[last] + s["dhT"][full]
    back = torch.cat([cut[1:], torch.zeros_like(cut[:1])]).flip(0)   # the decay from t + 1 to t, last token first
    g = _doubling(back, g.flip(0)).flip(0)
    dlog_a = (g * a * before).view_as(s["log_a"])
    dh0 = s["dhT"].clone()
    dh0[full] = a[first] * g[first]
    return [out, hT, g.to(s["x"].dtype).view_as(s["x"]), dlog_a, dh0]


def _plain_step(s):
    at = s["slots"].long()
    h = torch.exp(s["log_a"]) * s["pool"][at] + s["x"].float()
    s["pool"][at] = h
    return [h.to(s["x"].dtype), s["pool"]]


def _ancestors(parents):
    """[N, K, K] truth values: j is i itself or one of its ancestors."""
    N, K = parents.shape
    at = torch.arange(K, device=parents.device)
    up = (parents[:, :, None] == at).float() + torch.eye(K, device=parents.device)
    span = 1
    while span < K:
        up = ((up @ up) > 0).float()
        span *= 2
    return up > 0


def _tree_parts(s):
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    K = k.shape[1]
    up = _ancestors(s["parents"])
    G = torch.einsum("nij,njhc->nihc", up.double(), s["log_alpha"].double())
    gap = (G[:, :, None] - G[:, None]).float()                       # [N, i, j, H, c]: decay from j to i
    gap = torch.exp(gap.masked_fill_(~up[:, :, :, None, None], -math.inf))
    A = torch.einsum("nihc,nijhc,njhc->nhij", k, gap, k)
    A = A * ~torch.eye(K, dtype=torch.bool, device=A.device)
    E = torch.exp(G.float())
    S0 = s["pool"][s["slots"].long()]
    beta = s["beta"].permute(0, 2, 1)[..., None]                     # [N, H, K, 1]
    vhat = torch.einsum("nihc,nhcd->nhid", k * E, S0)
    u = beta * (v.permute(0, 2, 1, 3) - vhat)
    # u = (I + beta A)^-1 (..): A is nilpotent, so the inverse is a finite product
    X, span = -beta * A, 1
    while span < K:
        u = u + X @ u
        X, span = X @ X, span * 2
    return q, k, up, G, gap, E, S0, u


def _plain_tree(s):
    q, k, up, G, gap, E, S0, u = _tree_parts(s)
    Aq = torch.einsum("nihc,nijhc,njhc->nhij", q, gap, k)
    o = torch.einsum("nihc,nhcd->nhid", q * E, S0) + Aq @ u
    o = (s["scale"] * o).permute(0, 2, 1, 3)
    live = torch.arange(o.shape[1], device=o.device) < s["nodes"].long()[:, None]
    s["out"][live] = o[live].to(s["out"].dtype)
    return s["out"]


def _plain_commit(s):
    _, k, up, G, gap, E, S0, u = _tree_parts(s)
    n = torch.arange(k.shape[0], device=k.device)
    at = s["accepted"].long()
    w = k * gap[n, at]                                               # zero off the accepted path
    S = E[n, at][..., None] * S0 + torch.einsum("njhc,nhjd->nhcd", w, u)
    s["pool"][s["slots"].long()] = S
    return s["pool"]


_EPS = 1e-5


def _act(name, z):
    if name == "none":
        return z, torch.ones_like(z)
    p = 1 / (1 + torch.exp(-z))
    return (p, p * (1 - p)) if name == "sigmoid" else (z * p, p * (1 + z * (1 - p)))


def _norm_parts(s, x, z, w, b):
    mean = x.mean(-1, keepdim=True) if s["center"] else 0
    x = x - mean
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS)
    xh = x * rstd
    n = xh * w if b is None else xh * w + b
    f, df = _act(s["act"], n if z is None else z)
    return rstd, xh, n, f, df


def _norm_all(s, x, z, w, b, dy):
    rstd, xh, n, f, df = _norm_parts(s, x, z, w, b)
    if dy is None:
        return [f if z is None else n * f]
    dn = dy * df if z is None else dy * f
    dz = None if z is None else dy * n * df
    rows = (0,) if w.dim() == 2 else (0, 1)
    dw = (dn * xh).sum(rows)
    db = None if b is None else dn.sum(rows)
    dxh = dn * w
    back = dxh - xh * (dxh * xh).mean(-1, keepdim=True)
    if s["center"]:
        back = back - dxh.mean(-1, keepdim=True)
    return [back * rstd, dz, dw, db]


def _plain_norm(s):
    f = lambda t: None if t is None else t.float()
    r = _norm_all(s, f(s["x"]), f(s["z"]), s["weight"], s["bias"], f(s["dout"]))
    io = s["x"].dtype
    return [t if i >= 2 or t is None else t.to(io) for i, t in enumerate(r)]


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if not own:
        return {"scan": _plain_scan, "scan_train": _plain_scan, "scan_step": _plain_step, "tree": _plain_tree,
                "tree_commit": _plain_commit, "norm": _plain_norm, "norm_grad": _plain_norm}[op](s)
    import gated_delta_rule_75_b200 as kda
    if op == "scan":
        return list(kda.glr_scan_fwd(s["x"], s["log_a"], h0=s["h0"], cu_seqlens=s["cu"]))
    if op == "scan_train":
        out, hT, starts = kda.glr_scan_fwd(s["x"], s["log_a"], h0=s["h0"], cu_seqlens=s["cu"], output_starts=True)
        grads = kda.glr_scan_bwd(s["x"], s["log_a"], s["dout"], starts=starts, h0=s["h0"], dhT=s["dhT"],
                                 cu_seqlens=s["cu"])
        return [out, hT, *grads]
    if op == "scan_step":
        return [kda.glr_step(s["x"], s["log_a"], s["pool"], slots=s["slots"]), s["pool"]]
    if op == "tree":
        return kda.tree_fwd(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["pool"], s["parents"], s["scale"],
                            num_nodes=s["nodes"], slots=s["slots"], out=s["out"])
    if op == "tree_commit":
        return kda.tree_commit(s["k"], s["v"], s["log_alpha"], s["beta"], s["pool"], s["parents"], s["accepted"],
                               slots=s["slots"])
    if op == "norm":
        return [kda.group_norm_fwd(s["x"], s["weight"], bias=s["bias"], gate=s["z"], eps=_EPS, activation=s["act"],
                                   center=s["center"])]
    dx, dgate, dweight, dbias = kda.group_norm_bwd(s["x"], s["weight"], s["dout"], bias=s["bias"], gate=s["z"],
                                                   eps=_EPS, activation=s["act"], center=s["center"])
    return [dx, dgate, dweight, dbias]


def work(case):
    """Bytes and operations of one pass: every input read once, every output written once."""
    op, e = case["op"], _BYTES[case["io"]]
    if op == "scan_step":
        n = case["N"] * case["D"]
        return {"bytes": n * (2 * e + 4 + 8), "flops": 3 * n}
    if op in ("scan", "scan_train"):
        n, rows = case["B"] * case["T"] * case["D"], (case["N"] or case["B"]) * case["D"]
        if op == "scan":
            return {"bytes": n * (2 * e + 4) + 8 * rows, "flops": 3 * n}
        return {"bytes": n * (4 * e + 8) + 16 * rows, "flops": 8 * n}
    if op in ("tree", "tree_commit"):
        N, K, H, dk, dv = (case[k] for k in ("N", "K", "H", "dk", "dv"))
        if op == "tree":
            token = e * (2 * dk + 2 * dv) + 4 * dk + 4
            return {"bytes": N * H * (4 * dk * dv + K * token), "flops": N * H * K * 4 * dk * dv}
        token = e * (dk + dv) + 4 * dk + 4
        return {"bytes": N * H * (8 * dk * dv + token), "flops": N * H * 7 * dk * dv}
    n = case["M"] * case["G"] * case["d"]
    if op == "norm":
        return {"bytes": n * e * (3 if case["gate"] else 2), "flops": 12 * n}
    return {"bytes": n * e * (5 if case["gate"] else 3), "flops": 30 * n}


# ---------------------------------------------------------------- 64 bits, from the definitions

def _exact_scan(s):
    x, la = s["x"].double(), s["log_a"].double()
    B, T, D = x.shape
    a = torch.exp(la)
    del la
    if s["cu"] is None:
        spans = [(slice(None), 0, T, slice(None))]
    else:
        cu = s["cu"].tolist()
        spans = [(slice(0, 1), cu[n], cu[n + 1], slice(n, n + 1)) for n in range(len(cu) - 1)]
    hT = s["h0"].double()
    grads = s["op"] == "scan_train"
    H = torch.empty_like(x)
    for b, t0, t1, n in spans:
        h = hT[n].clone()
        for t in range(t0, t1):
            h = torch.addcmul(x[b, t], a[b, t], h)
            H[b, t] = h
        hT[n] = h
    if not grads:
        return [H, hT]
    dx, dla, dh0 = s["dout"].double(), torch.empty_like(x), s["dhT"].double()
    for b, t0, t1, n in spans:
        g = dh0[n].clone()
        for t in range(t1 - 1, t0 - 1, -1):
            g = g + dx[b, t]
            dx[b, t] = g
            g = a[b, t] * g
            dla[b, t] = g * (H[b, t - 1] if t > t0 else s["h0"][n].double())
        dh0[n] = g
    return [H, hT, dx, dla, dh0]


def _exact_tree(s):
    """Token by token along every path, with the state of every node kept."""
    N, K, H, dk = s["k"].shape
    dv = s["v"].shape[-1]
    parents, nodes, acc, slots = (s[n].tolist() for n in ("parents", "nodes", "accepted", "slots"))
    commit = s["op"] == "tree_commit"
    out = torch.zeros((N, K, H, dv), dtype=torch.float64, device="cuda")
    pool = s["pool"].double()
    for n in range(N):
        S = [None] * K
        q, k, v, al, be = (s[m][n].double() for m in ("q", "k", "v", "log_alpha", "beta"))
        al = torch.exp(al)
        for i in range(nodes[n]):
            p = parents[n][i]
            X = al[i][:, :, None] * (pool[slots[n]] if p < 0 else S[p])
            err = be[i][:, None] * (v[i] - (k[i][:, :, None] * X).sum(1))
            S[i] = X + k[i][:, :, None] * err[:, None, :]
            if not commit:
                out[n, i] = s["scale"] * (q[i][:, :, None] * S[i]).sum(1)
        if commit:
            pool[slots[n]] = S[acc[n]]
    return pool if commit else out


def _exact_norm(s):
    """Values by the definition; gradients by the chain rule through the statistics, row by row."""
    D = lambda t: None if t is None else t.double()
    x, z, w, b, dy = (D(s[n]) for n in ("x", "z", "weight", "bias", "dout"))
    d = x.shape[-1]
    mu = x.sum(-1, keepdim=True) / d if s["center"] else torch.zeros_like(x[..., :1])
    var = ((x - mu) ** 2).sum(-1, keepdim=True) / d
    r = (var + _EPS) ** -0.5
    n = (x - mu) * r * w + (0 if b is None else b)
    t = n if z is None else z
    sg = torch.sigmoid(t)
    f = {"none": t, "sigmoid": sg, "silu": t * sg}[s["act"]]
    if dy is None:
        return [f if z is None else n * f]
    df = {"none": torch.ones_like(t), "sigmoid": sg - sg * sg, "silu": sg + t * (sg - sg * sg)}[s["act"]]
    dn = dy * (df if z is None else f)
    dz = None if z is None else dy * n * df
    c = dn * w
    dvar = (c * (x - mu)).sum(-1, keepdim=True) * -0.5 * r ** 3
    dx = c * r + dvar * 2 * (x - mu) / d
    if s["center"]:
        dx = dx - (c * r).sum(-1, keepdim=True) / d
    per = w.dim() == 2
    dw = dn * (x - mu) * r
    return [dx, dz, dw.sum(0) if per else dw.sum((0, 1)), None if b is None else dn.sum(0) if per else dn.sum((0, 1))]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("scan", "scan_train"):
        return _exact_scan(s)
    if case["op"] == "scan_step":
        at = s["slots"].long()
        pool = s["pool"].double()
        h = torch.exp(s["log_a"].double()) * pool[at] + s["x"].double()
        pool[at] = h
        return [h, pool]
    if case["op"] in ("tree", "tree_commit"):
        return _exact_tree(s)
    return _exact_norm(s)
