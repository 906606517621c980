"""Gated linear recurrence on the GPU against the fp64 recurrence, element by element: lengths
from one token over tile borders to many tiles, packed sequences with empty ones, channel counts
that no vector divides, pools, strong and no decay, gradients, refusals of the device."""
import numpy as np
import pytest
import torch

import operators_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda(cuda_ok):
    from gated_delta_rule_75_b200 import build
    build.build()
    import gated_delta_rule_75_b200 as kda
    return kda


def inputs(B, T, D, io, seed, N=None, decay="usual"):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)
    la = -torch.log1p(torch.exp(n(B, T, D) - 3))
    if decay == "none":
        la = torch.zeros(B, T, D)
    elif decay == "strong":
        la = -40 * torch.rand((B, T, D), generator=g)
    elif decay == "forget":                                  # exp(-inf) = 0 here and there
        la = torch.where(torch.rand((B, T, D), generator=g) < 0.1, torch.tensor(float("-inf")), la)
    x = n(B, T, D).to(R.IO[io])
    return x.cuda(), la.cuda(), n(N or B, D).cuda()


def offsets(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return cu, torch.tensor(cu, dtype=torch.int32, device="cuda")


def starts_of(H, h0, B, T, cu, tile):
    """States before the first token of every tile."""
    h0 = torch.zeros(B if cu is None else len(cu) - 1, H.shape[-1], dtype=torch.float64) if h0 is None else h0
    out = torch.zeros(B, -(-T // tile), H.shape[-1], dtype=torch.float64)
    for b, t0, t1, n in R.spans(B, T, cu):
        for t in range(t0, t1):
            if t % tile == 0:
                out[b, t // tile] = h0[n] if t == t0 else H[b, t - 1]
    return out


FIXED = [(1, 1, 1), (2, 1, 7), (3, 63, 130), (2, 64, 64), (1, 65, 4), (2, 129, 33), (1, 500, 6), (5, 200, 260),
         (1, 2500, 12), (1, 9001, 3)]
PACKED = [([1], 5), ([3, 0, 1, 0, 60, 64, 65], 36), ([0, 0, 130], 7), ([200, 0, 0], 8), ([1] * 70, 4),
          ([700, 1, 64, 128, 333], 132), ([5000, 0, 2111], 5)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", FIXED)
def test_forward_and_backward_rows(kda, B, T, D, io):
    x, la, h0 = inputs(B, T, D, io, 100 * T + D)
    check(kda, x, la, h0, None, None)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens,D", PACKED)
def test_forward_and_backward_packed(kda, lens, D, io):
    cu, dcu = offsets(lens)
    x, la, h0 = inputs(1, cu[-1], D, io, 7 * cu[-1] + D, N=len(lens))
    check(kda, x, la, h0, cu, dcu)


@pytest.mark.parametrize("decay", ["none", "strong", "forget"])
def test_decay_extremes(kda, decay):
    x, la, h0 = inputs(2, 300, 40, "f32", 3, decay=decay)
    check(kda, x, la, h0, None, None)
    cu, dcu = offsets([129, 0, 400])
    x, la, h0 = inputs(1, cu[-1], 24, "bf16", 4, N=3, decay=decay)
    check(kda, x, la, h0, cu, dcu)


def check(kda, x, la, h0, cu, dcu):
    B, T, D = x.shape
    H, hT, E, eT = R.glr(R.d(x), R.d(la), R.d(h0), cu)
    out, last, starts = kda.glr_scan_fwd(x, la, h0=h0, cu_seqlens=dcu, output_starts=True)
    R.within(out, H, E, "out")
    R.within(last, hT, eT, "hT")
    R.within(starts, starts_of(H, R.d(h0), B, T, cu, kda.GLR_TILE), starts_of(E, h0.cpu().double() * 0, B, T, cu, kda.GLR_TILE),
             "starts")
    again, _ = kda.glr_scan_fwd(x, la, h0=h0, cu_seqlens=dcu)
    assert torch.equal(out, again)
    g = torch.Generator().manual_seed(T + D)
    dout = torch.randn((B, T, D), generator=g).to(x.dtype).cuda()
    dhT = torch.randn(h0.shape, generator=g).cuda()
    for first, seed in ((h0, dhT), (None, None)):
        if first is None:
            starts = None
        dx, dla, dh0 = kda.glr_scan_bwd(x, la, dout, starts=starts, h0=first, dhT=seed, cu_seqlens=dcu)
        want = R.glr_grads(R.d(x), R.d(la), R.d(first), R.d(dout), R.d(seed), cu)
        R.within(dx, want[0], want[3], "dx")
        R.within(dla, want[1], want[4], "dlog_a")
        R.within(dh0, want[2], want[5], "dh0")
    assert kda.glr_scan_bwd(x, la, dout, cu_seqlens=dcu, need_dh0=False)[2] is None


def test_pool_chunked_scan_then_steps(kda):
    """Prompts scanned in two pieces and then token by token, all through pool slots, one of them
    without a state: every output equals the whole recurrence's."""
    lens, D, P, cut, steps = [150, 64, 3], 20, 5, 70, 3
    full = [n + steps for n in lens]
    cu, _ = offsets(full)
    x, la, h0 = inputs(1, cu[-1], D, "f32", 9, N=3)
    slots = torch.tensor([4, -1, 0], dtype=torch.int32, device="cuda")
    pool = torch.randn(P, D, device="cuda")
    before = pool.clone()
    pool[4], pool[0] = h0[0], h0[2]
    first = R.d(h0)
    first[1] = 0
    H, hT, E, eT = R.glr(R.d(x), R.d(la), first, cu)

    def part(pieces):
        at = torch.cat([torch.arange(cu[n] + a, cu[n] + b) for n, (a, b) in enumerate(pieces)]).cuda()
        _, seg = offsets([b - a for a, b in pieces])
        return x[:, at].contiguous(), la[:, at].contiguous(), seg, at

    a, b, seg, at = part([(0, min(cut, n)) for n in lens])
    out, got = kda.glr_scan_fwd(a, b, cu_seqlens=seg, state_pool=pool, slots=slots)
    assert got is pool
    R.within(out[0], H[0, at.cpu()], E[0, at.cpu()], "first piece")
    a, b, seg, at = part([(min(cut, n), n) for n in lens])
    out, _ = kda.glr_scan_fwd(a, b, cu_seqlens=seg, state_pool=pool, slots=slots)
    # the sequence without a slot has at most `cut` tokens: its second piece is empty
    R.within(out[0], H[0, at.cpu()], E[0, at.cpu()], "second piece")
    for s in range(steps):
        at = torch.tensor([cu[n] + lens[n] + s for n in range(3)])
        o = kda.glr_step(x[0, at].contiguous(), la[0, at].contiguous(), pool, slots=slots)
        for n in (0, 2):
            R.within(o[n], H[0, at[n]], E[0, at[n]], "step")
        assert float(o[1].abs().max()) == 0
    R.within(pool[4], hT[0], eT[0], "state 4")
    R.within(pool[0], hT[2], eT[2], "state 0")
    assert torch.equal(pool[1:4], before[1:4])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N,D", [(1, 1), (3, 5), (7, 256), (130, 1030), (2, 4099)])
def test_step(kda, N, D, io):
    x, la, h = inputs(1, N, D, io, N + D, N=N)
    state = h.clone()
    out = kda.glr_step(x[0], la[0], state)
    want, _, E, _ = R.glr(R.d(x).transpose(0, 1), R.d(la).transpose(0, 1), R.d(h))
    R.within(out, want[:, 0], E[:, 0], "out")
    R.within(state, want[:, 0], E[:, 0], "state")


def test_state_in_place_and_no_states(kda):
    x, la, h0 = inputs(2, 100, 12, "f32", 21)
    _, want = kda.glr_scan_fwd(x, la, h0=h0)
    buf = h0.clone()
    _, got = kda.glr_scan_fwd(x, la, h0=buf, hT=buf)
    assert got is buf and torch.equal(buf, want)
    out, none = kda.glr_scan_fwd(x, la, output_final_state=False)
    assert none is None
    H, _, E, _ = R.glr(R.d(x), R.d(la), None)
    R.within(out, H, E, "out")


def test_no_tokens(kda):
    x, la, h0 = inputs(2, 1, 8, "f32", 22)
    out, hT, starts = kda.glr_scan_fwd(x[:, :0], la[:, :0], h0=h0, output_starts=True)
    assert out.shape == (2, 0, 8) and starts.shape == (2, 0, 8) and torch.equal(hT, h0)
    dx, dla, dh0 = kda.glr_scan_bwd(x[:, :0], la[:, :0], x[:, :0], h0=h0, dhT=h0)
    assert dx.numel() == 0 and torch.equal(dh0, h0)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, hT = kda.glr_scan_fwd(x[:1, :0], la[:1, :0], h0=h0, cu_seqlens=cu)
    assert torch.equal(hT, h0)
    pool = h0.clone()
    kda.glr_scan_fwd(x[:1, :0], la[:1, :0], cu_seqlens=cu, state_pool=pool,
                     slots=torch.tensor([1, -1], dtype=torch.int32, device="cuda"))
    assert torch.equal(pool, h0)
    assert kda.glr_step(x[0, :0].reshape(0, 8), la[0, :0].reshape(0, 8), h0[:0]).shape == (0, 8)


def test_bad_slots_and_offsets_are_reported(kda):
    x, la, _ = inputs(1, 100, 8, "f32", 23)
    pool = torch.ones(2, 8, device="cuda")
    _, cu = offsets([40, 60])
    slots = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    with pytest.raises(kda.KDAError) as e:
        kda.glr_scan_fwd(x, la, cu_seqlens=cu, state_pool=pool, slots=slots)
    assert e.value.status == kda.KDA_ERR_INVALID_ARG and float(pool[1].min()) == 1
    with pytest.raises(kda.KDAError):
        kda.glr_step(x[0, :2], la[0, :2], pool, slots=slots)
    for bad in ([0, 60, 40, 100], [1, 50, 100], [0, 50, 90], [0, -5, 100], [0, 120, 100]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        with pytest.raises(kda.KDAError) as e:
            kda.glr_scan_fwd(x, la, cu_seqlens=cu)
        assert e.value.status == kda.KDA_ERR_INVALID_ARG
        with pytest.raises(kda.KDAError):
            kda.glr_scan_bwd(x, la, x, cu_seqlens=cu)


def test_not_a_number_stays_in_its_sequence_and_channel(kda):
    cu, dcu = offsets([100, 200, 150])
    x, la, h0 = inputs(1, 450, 8, "f32", 24, N=3)
    x[0, 150, 3] = float("nan")
    x[0, 20, 1] = float("inf")
    out, hT = kda.glr_scan_fwd(x, la, h0=h0, cu_seqlens=dcu)
    bad = ~torch.isfinite(out[0])
    want = torch.zeros_like(bad)
    want[150:300, 3] = True
    want[20:100, 1] = True
    assert torch.equal(bad, want) and int((~torch.isfinite(hT)).sum()) == 2


@pytest.mark.parametrize("io,D", [("f32", 40), ("bf16", 7)])
@pytest.mark.parametrize("end", [0, 1, 64, 90, 150])
def test_rows_behind_the_last_sequence_stay(kda, io, D, end):
    """Offsets that end before the tokens do (padding behind the last sequence) are reported; what lies in
    a sequence is computed, what lies behind is not written."""
    T = 200
    lens = [end - end // 3, 0, end // 3]
    cu, dcu = offsets(lens)
    x, la, h0 = inputs(1, T, D, io, 31 + end, N=3)
    x[:, end:] = float("nan")
    out = torch.full_like(x, 5.0)
    hT = torch.empty_like(h0)
    with pytest.raises(kda.KDAError) as e:
        kda.glr_scan_fwd(x, la, h0=h0, cu_seqlens=dcu, out=out, hT=hT)
    assert e.value.status == kda.KDA_ERR_INVALID_ARG
    H, want, E, eT = R.glr(R.d(x), R.d(la), R.d(h0), cu)
    R.within(out[:, :end], H[:, :end], E[:, :end], "out")
    R.within(hT, want, eT, "hT")
    assert bool((out[:, end:] == 5).all())


HALF = 2.0 ** -24


def long_sums(a, x, first):
    """h_t = a_t h_{t-1} + x_t of one sequence in fp64, and a bound on its fp32 error that lets no error
    through that grows with the number of tiles on top of what fp32 decays must cost: every decay is rounded
    once (its exponential within 1.5 half steps) and meets what stands before it.  Sums and products are
    folded as a tree: a run's 16 tokens, 4 runs, 8 tiles, 8 blocks, then the carried state through the same and 16
    tokens, under 120 roundings of partial sums, of which none is above twice the largest |h| so far; the
    products of decays under 34 in a group of 4096 tokens, which are exact where nothing decays."""
    h, e = first, np.zeros_like(first)
    H, E = np.empty_like(x), np.empty_like(x)
    for t in range(len(x)):
        e = a[t] * (e + (a[t] != 1) * 1.5 * HALF * np.abs(h))
        h = a[t] * h + x[t]
        H[t], E[t] = h, e
    most = 2 * np.maximum.accumulate(np.maximum(np.abs(H), np.abs(first)), 0)
    groups = 1 + np.arange(len(x))[:, None] // 4096
    return H, E + HALF * most * (120 + groups * (1 + 34 * (a != 1).any()))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("least", [0.0, -2e-4])
@pytest.mark.parametrize("lens,D,packed", [([9001], 8, False), ([70000], 3, False), ([4097, 0, 12288, 600, 33000], 6, True)])
def test_long_memories(kda, lens, D, packed, least, io):
    """Decays of 1, or next to it, over many blocks of tiles: forward and backward."""
    T, N = sum(lens), len(lens)
    cu, dcu = offsets(lens)
    g = torch.Generator().manual_seed(T + D)
    x, dout = (torch.randn((1, T, D), generator=g).to(R.IO[io]) for _ in range(2))
    la = least * torch.rand((1, T, D), generator=g)
    h0, dhT = (100 * torch.randn((N, D), generator=g) for _ in range(2))
    kw = {"cu_seqlens": dcu if packed else None}
    out, hT, starts = kda.glr_scan_fwd(x.cuda(), la.cuda(), h0=h0.cuda(), output_starts=True, **kw)
    dx, dla, dh0 = kda.glr_scan_bwd(x.cuda(), la.cuda(), dout.cuda(), starts=starts, h0=h0.cuda(), dhT=dhT.cuda(), **kw)
    t64 = lambda v: torch.from_numpy(np.ascontiguousarray(v))
    for n in range(N):
        s = slice(cu[n], cu[n + 1])
        if lens[n] == 0:
            assert torch.equal(hT[n].cpu(), h0[n]) and torch.equal(dh0[n].cpu(), dhT[n])
            continue
        a, X, Y = torch.exp(la[0, s].double()).numpy(), R.d(x[0, s]).numpy(), R.d(dout[0, s]).numpy()
        first, last = h0[n].double().numpy(), dhT[n].double().numpy()
        H, E = long_sums(a, X, first)
        R.within(out[0, s], t64(H), t64(E), "out")
        R.within(hT[n], t64(H[-1]), t64(E[-1]), "hT")
        # g_t = dout_t + a_{t+1} g_{t+1}: the same sums from the end, with each decay a token later
        G, EG = long_sums(np.concatenate([np.ones((1, D)), a[:0:-1]]), Y[::-1], last)
        G, EG = G[::-1], EG[::-1]
        R.within(dx[0, s], t64(G), t64(EG), "dx")
        before, eb = np.concatenate([first[None], H[:-1]]), np.concatenate([np.zeros((1, D)), E[:-1]])
        # the decay of dlog_a = g a h and the two products once more
        bound = a * (np.abs(before) * EG + np.abs(G) * eb + EG * eb) + 4 * HALF * np.abs(G * a * before)
        R.within(dla[0, s], t64(G * a * before), t64(bound), "dlog_a")
        R.within(dh0[n], t64(a[0] * G[0]), t64(a[0] * EG[0] + 4 * HALF * np.abs(G[0])), "dh0")


@pytest.mark.parametrize("T,D", [(700, 8), (20000, 5), (131072, 4)])
def test_a_state_without_decay_stays_as_it_is(kda, T, D):
    """No decay and no input (padding, a kept state): every product is by 1 and every sum with 0, so the state
    passes any number of tiles bit for bit, and so do the gradients."""
    g = torch.Generator().manual_seed(T)
    zero = torch.zeros(2, T, D, device="cuda")
    h0, dhT = (torch.randn((2, D), generator=g).cuda() for _ in range(2))
    out, hT, starts = kda.glr_scan_fwd(zero, zero, h0=h0, output_starts=True)
    assert torch.equal(hT, h0) and torch.equal(out, h0[:, None].expand_as(out))
    assert torch.equal(starts, h0[:, None].expand_as(starts))
    dx, dla, dh0 = kda.glr_scan_bwd(zero, zero, zero, starts=starts, h0=h0, dhT=dhT)
    assert torch.equal(dh0, dhT) and torch.equal(dx, dhT[:, None].expand_as(dx))
    assert torch.equal(dla, (dhT * h0)[:, None].expand_as(dla))


@pytest.mark.parametrize("B,T,D,packed", [(64, 128, 4096, False), (64, 100, 1000, False), (1, 2000, 4096, True),
                                          (16, 512, 2048, False), (16, 513, 2048, False), (2, 64 * 71, 2048, False)])
def test_workspace_is_what_the_header_says(kda, B, T, D, packed):
    x, la = torch.zeros(B, T, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, T, D, device="cuda")
    _, dcu = offsets([T // 2, T - T // 2])
    h0 = torch.randn(2 if packed else B, D, device="cuda")
    kda.workspace_high_water(reset=True)
    out, hT = kda.glr_scan_fwd(x, la, h0=h0, cu_seqlens=dcu if packed else None)
    used = kda.workspace_high_water()
    tiles, channels = -(-T // 64), B * (-(-D // 64) * 64)
    blocks = -(-tiles // 8)
    says = 8 * tiles * channels + (8 * blocks * channels if blocks > 1 else 0) + (8 * (tiles + 1) if packed else 0)
    assert used <= says + 4096                            # the pool's own rounding
    assert torch.equal(hT, h0)


@pytest.mark.parametrize("io,B,T,D", [("bf16", 1024, 65, 4096), ("bf16", 700, 66, 4094), ("bf16", 300, 129, 4093),
                                      ("f32", 512, 65, 4096), ("f32", 400, 67, 2046)])
def test_many_short_rows(kda, io, B, T, D):
    """Tiles that take a worker next to no time, so that workers run as far ahead of the copies as the ring
    lets them: every one of many calls ends well, with the same result, which is the recurrence's."""
    g = torch.Generator(device="cuda").manual_seed(T + D)
    x = torch.randn((B, T, D), generator=g, device="cuda").to(R.IO[io])
    la = torch.rand((B, T, D), generator=g, device="cuda").mul_(-0.2)
    h0 = torch.randn((B, D), generator=g, device="cuda")
    out, hT, starts = kda.glr_scan_fwd(x, la, h0=h0, output_starts=True)
    h, m, e = h0.double(), h0.double().abs(), torch.zeros_like(h0, dtype=torch.float64)
    for t in range(T):                                    # the bound of operators_ref.glr
        a, y = torch.exp(la[:, t].double()), x[:, t].double()
        h, m = a * h + y, a * m + y.abs()
        e = a * e + R.STEP * m
        assert bool(((out[:, t].double() - h).abs() <= e + R.HALF_STEP[x.dtype] * (h.abs() + e)).all()), t
    assert bool(((hT.double() - h).abs() <= e + R.HALF_STEP[torch.float32] * (h.abs() + e)).all())
    again = torch.empty_like(out)
    grads = kda.glr_scan_bwd(x, la, x, starts=starts, h0=h0, dhT=h0)
    for _ in range(25):
        kda.glr_scan_fwd(x, la, h0=h0, out=again, hT=hT)
        assert torch.equal(out, again)
    for _ in range(10):
        assert all(torch.equal(p, q) for p, q in zip(grads, kda.glr_scan_bwd(x, la, x, starts=starts, h0=h0, dhT=h0)))
