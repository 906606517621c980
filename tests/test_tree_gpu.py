"""Drafted token trees on the GPU against the fp64 token recurrence along every path."""
import random

import pytest
import torch

import operators_ref as R

pytestmark = pytest.mark.gpu

# relative 2-norm.  fp32: sums of 128 terms, at most 128 half steps of 2^-24 on the magnitudes, 7.6e-6,
# which the norm over a whole output averages down.  bf16: at most half a step, 2^-8, on every value
# besides.
TOL = {"f32": 1e-5, "bf16": 2.0 ** -8 + 1e-5}


@pytest.fixture(scope="module")
def kda(cuda_ok):
    from gated_delta_rule_75_b200 import build
    build.build()
    import gated_delta_rule_75_b200 as kda
    return kda


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def ref(x):
    return [R.d(x[m]) for m in ("q", "k", "v", "log_alpha", "beta", "state")]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N,K,H,dk,dv,deep,shift", [
    (1, 1, 1, 128, 128, 1, -2), (2, 5, 3, 128, 64, 5, -2), (3, 16, 2, 64, 128, 6, -2), (2, 17, 2, 128, 128, 4, 0),
    (1, 33, 1, 64, 64, 33, -2), (2, 64, 2, 128, 128, 64, -4), (2, 61, 1, 128, 128, 12, -2), (2, 40, 2, 64, 128, 1, -2),
    (1, 64, 1, 128, 128, 64, 6), (40, 8, 4, 128, 128, 8, -2)])
def test_tree_and_commit(kda, N, K, H, dk, dv, deep, shift, io):
    rng = random.Random(N * 1000 + K)
    x, scale = R.tree_inputs(N, K, H, dk, dv, io, K + dk, shift=float(shift))
    parents = [list(range(-1, K - 1)) if deep >= K else R.make_tree(rng, K, deep) for _ in range(N)]
    out = kda.tree_fwd(*(x[m] for m in ("q", "k", "v", "log_alpha", "beta", "state")), i32(parents), scale)
    want = R.tree(*ref(x), parents, scale)
    assert R.rel(out, want) <= TOL[io]
    for n in range(N):                                    # node by node, so that none hides among others
        for i in range(K):
            # a few 2^-9 random roundings of bf16 average to less than the bound over one row; fp32 the same
            assert R.rel(out[n, i], want[n, i]) <= 2 * TOL[io], (n, i)
    accepted = [rng.randrange(-1, K) for _ in range(N)]
    accepted[0] = K - 1
    before = x["state"].clone()
    want = R.tree_commit(*(R.d(x[m]) for m in ("k", "v", "log_alpha", "beta", "state")), parents, accepted)
    got = kda.tree_commit(*(x[m] for m in ("k", "v", "log_alpha", "beta", "state")), i32(parents), i32(accepted))
    assert got is x["state"] and R.rel(got, want) <= TOL["f32"]
    for n in range(N):
        if accepted[n] < 0:
            assert torch.equal(got[n], before[n])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_slots_and_node_counts(kda, io):
    """Pools in any order, a shared slot (read only), no slot, trees that end early: their rows stay."""
    rng = random.Random(8)
    N, K, H, P = 5, 20, 2, 4
    x, scale = R.tree_inputs(N, K, H, 128, 128, io, 31, P=P)
    x["state"] = x["state"][:P].contiguous()
    parents = [R.make_tree(rng, K, 5) for _ in range(N)]
    nodes, slots = [20, 0, 13, 1, 19], [3, 1, -1, 0, 3]
    pool = x["state"].clone()
    out = torch.full((N, K, H, 128), 7.0, dtype=R.IO[io], device="cuda")
    args = [x[m] for m in ("q", "k", "v", "log_alpha", "beta")]
    # what stands behind a tree's last node is never looked at
    for n in range(N):
        for t in args:
            t[n, nodes[n]:] = float("nan")
    par = i32(parents)
    for n in range(N):
        par[n, nodes[n]:] = 99
    got = kda.tree_fwd(*args, pool, par, scale, num_nodes=i32(nodes), slots=i32(slots), out=out)
    assert got is out and torch.equal(pool, x["state"])
    clean = [torch.nan_to_num(R.d(t)) for t in args]
    want = R.tree(*clean, R.d(pool), parents, scale, num_nodes=nodes, slots=slots)
    for n in range(N):
        if nodes[n]:
            assert R.rel(out[n, :nodes[n]], want[n, :nodes[n]]) <= TOL[io], n
        assert bool((out[n, nodes[n]:] == 7).all())
    fresh = kda.tree_fwd(*args, pool, par, scale, num_nodes=i32(nodes), slots=i32(slots))
    assert all(float(fresh[n, nodes[n]:].abs().sum()) == 0 for n in range(N))


def test_commit_equals_decode_steps(kda):
    """A chain committed at once gives the states, and the tree the outputs, of the decode step taken
    token by token on the same pool."""
    N, K, H = 3, 7, 2
    x, scale = R.tree_inputs(N, K, H, 128, 128, "f32", 77, P=6)
    slots = i32([5, 0, 2])
    par = i32([list(range(-1, K - 1))] * N)
    one = x["state"].clone()
    outs = kda.tree_fwd(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], one, par, scale, slots=slots)
    steps = one.clone()
    for i in range(K):
        c = lambda m: x[m][:, i].contiguous()
        o = kda.recurrent_step(c("q"), c("k"), c("v"), c("log_alpha"), c("beta"), steps, scale, slots=slots)
        assert R.rel(outs[:, i], R.d(o)) <= 2 * TOL["f32"]
    kda.tree_commit(x["k"], x["v"], x["log_alpha"], x["beta"], one, par, i32([K - 1] * N), slots=slots)
    assert R.rel(one, R.d(steps)) <= 2 * TOL["f32"]
    for p in (1, 3, 4):
        assert torch.equal(one[p], x["state"][p])


def test_bad_trees_are_reported(kda):
    x, scale = R.tree_inputs(2, 4, 1, 64, 64, "f32", 5, P=2)
    a = [x[m] for m in ("q", "k", "v", "log_alpha", "beta")]
    ok = [[-1, 0, 1, 2]] * 2
    before = x["state"].clone()
    for kw in ({"par": [[0, 0, 1, 2]] * 2}, {"par": [[-1, -2, 0, 0]] * 2}, {"par": [[-1, 0, 1, 1 << 30]] * 2},
               {"nodes": [5, 1]}, {"nodes": [-1, 4]}, {"slots": [0, 2]}):
        with pytest.raises(kda.KDAError) as e:
            kda.tree_fwd(*a, x["state"], i32(kw.get("par", ok)), scale,
                         num_nodes=i32(kw["nodes"]) if "nodes" in kw else None,
                         slots=i32(kw["slots"]) if "slots" in kw else None)
        assert e.value.status == kda.KDA_ERR_INVALID_ARG
    for acc, slots in (([4, -1], [0, 1]), ([-2, -1], [0, 1]), ([-1, 0], [0, 2])):
        with pytest.raises(kda.KDAError):
            kda.tree_commit(*a[1:], x["state"], i32(ok), i32(acc), slots=i32(slots))
        assert torch.equal(x["state"], before)
    with pytest.raises(kda.KDAError):                     # a bad parent on the accepted path counts as the root
        kda.tree_commit(*a[1:], x["state"], i32([[-1, 0, 7, 2], ok[0]]), i32([2, -1]))


def test_not_a_number_stays_on_its_branch(kda):
    x, scale = R.tree_inputs(1, 6, 1, 128, 128, "bf16", 6)
    par = [-1, 0, 0, 1, 2, -1]
    x["v"][0, 1, 0, 5] = float("nan")
    x["log_alpha"][0, 5] = float("-inf")                  # forgets the state: fine
    out = kda.tree_fwd(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["state"], i32([par]), scale)
    bad = (~torch.isfinite(out[0, :, 0])).any(-1).tolist()
    assert bad == [False, True, False, True, False, False]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("K,dk,dv", [(1, 128, 128), (16, 128, 64), (16, 64, 128), (17, 128, 128), (32, 64, 64), (61, 128, 128)])
def test_outputs_come_from_every_bit_of_the_state(kda, K, dk, dv, io):
    """Queries and keys that pick one row of the cached state, no decay: every product is exact, so the output
    is that row (or, behind a write of strength 1/2 of a zero value, half of it), rounded once and exactly.
    The state's values lie 2^-20 beside the middle between two bf16 values: what is lost of 24 bits shows."""
    g = torch.Generator().manual_seed(K + dk + dv)
    N, H = 3, 2
    coarse = torch.randint(128, 256, (N, H, dk, dv), generator=g) / 128.0                 # bf16 values in [1, 2)
    side = (torch.randint(0, 2, coarse.shape, generator=g) * 2 - 1) * 2.0 ** -20
    sign = torch.randint(0, 2, coarse.shape, generator=g) * 2.0 - 1
    state = (coarse + 2.0 ** -8 + side) * sign * 2.0 ** torch.randint(-9, 9, (N, H, dk, 1), generator=g)
    assert bool((state.to(torch.float32).double() == state.double()).all())
    pick = torch.randint(0, dk, (N, K, H), generator=g)
    q = torch.nn.functional.one_hot(pick, dk).to(R.IO[io])
    v, zero = torch.zeros(N, K, H, dv, dtype=R.IO[io]), torch.zeros(N, K, H, dk)
    rows = torch.stack([torch.stack([state[n, h][pick[n, :, h]] for h in range(H)], 1) for n in range(N)])
    for beta, share in ((0.0, 1.0), (0.5, 0.5)):
        out = kda.tree_fwd(q.cuda(), q.cuda(), v.cuda(), zero.cuda(), torch.full((N, K, H), beta).cuda(),
                           state.float().cuda(), i32([[-1] * K] * N), 1.0)
        assert torch.equal(out.cpu(), (share * rows).to(R.IO[io])), beta


@pytest.mark.parametrize("K", [3, 16, 30, 64])
def test_products_with_the_state_sum_up_closely(kda, K):
    """The products with the state alone (no decay, no writes), fp32.  Operands are three bf16 summands, and
    products of a weight have sums of their own, so the sums that reach the result's size take 8 additions of
    16 channels.  An addition loses at most a step, 2^-23, of what is there by then, which after j of the 8 is
    sqrt(j / 8) of the result's norm: 5.8 2^-23 in all, 16 2^-31 in the sums a weight below; a half step,
    2^-24, for joining the sums, for the scale and for the products that are left out: under 8.8e-7, in any
    rounding.  (All 48 additions at full size: up to 48 2^-23.)"""
    x, scale = R.tree_inputs(4, K, 3, 128, 128, "f32", 900 + K)
    x["log_alpha"].zero_()
    x["beta"].zero_()
    parents = [[-1] * K] * 4
    out = kda.tree_fwd(*(x[m] for m in ("q", "k", "v", "log_alpha", "beta", "state")), i32(parents), scale)
    err = R.rel(out, R.tree(*ref(x), parents, scale))
    print("relative error", err)
    assert err <= 8.8e-7
