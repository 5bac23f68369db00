"""GPU parity of the router's balance and its gradient against oracle.block (float64).

Tolerances are worst-case bounds, element by element, with U = 2^-24 half a step of fp32: an
exponential's argument l - max is off by half a step of it, d U for a distance d, the
exponential by a few steps; a sum of n by n U of its terms' magnitudes in any order, a product or
quotient by a step; a logarithm's argument off by r relative moves it by r. Whole numbers are exact.
"""

import numpy as np
import pytest
import torch

import bit_quantized_mixture_nf4_amd as e4b
from oracle import block
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV)


def host(t):
    return t.detach().cpu().double().numpy()


def within(got, ref, err, name):
    g = host(got)
    assert got.dtype == torch.float32 and g.shape == ref.shape, (name, g.shape, ref.shape)
    same = (g == ref) | (np.isnan(g) & np.isnan(ref))  # infinities and NaN
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(g - ref) <= (err + U * np.abs(ref)) * (1 + 2.0 ** -6) + 1e-37))
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{g[bad][0]} against {ref[bad][0]}")


def inputs(T, E, k, masked, seed=0):
    rng = np.random.default_rng(1000 * seed + T + E)
    lg = (rng.standard_normal((T, E)) * 2 + rng.standard_normal(E)).astype(np.float32)
    mask = None
    if masked:
        lg[rng.random((T, E)) < 0.2] = -np.inf
        lg[rng.random(T) < 0.1] = -np.inf
        mask = rng.random(T) > 0.2
    idx = np.argsort(-lg.astype(np.float64), axis=1, kind="stable")[:, :k].astype(np.int32)
    if masked:
        idx[rng.random((T, k)) < 0.1] = rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31])
        # what a token that is not counted holds is not looked at
        lg[~mask] = rng.choice([np.nan, np.inf, 3e38], ((~mask).sum(), E))
    return lg, idx, mask


def bounds(T, S, rng):
    cuts = np.sort(rng.integers(0, T + 1, S + 1)).astype(np.int32)
    if S > 2:
        cuts[1] = cuts[0]  # an empty one
    return cuts


def check(lg, idx, mask, cu, top_k=None):
    """Both directions against the oracle; the results."""
    T, E = lg.shape
    k = idx.shape[1]
    rng = np.random.default_rng(T)
    lg_d, idx_d = dev(lg), torch.from_numpy(idx).to(DEV)
    cu_d = None if cu is None else torch.from_numpy(np.asarray(cu, np.int32)).to(DEV)
    mask_d = None if mask is None else torch.from_numpy(mask).to(DEV)
    f = e4b.moe_balance(lg_d, idx_d, cu_tokens=cu_d, token_mask=mask_d)
    ref = block.balance(lg, idx, cu, mask)
    S = len(ref["loss"])
    assert f.counts.dtype == f.tokens.dtype == torch.int32 and f.top_k == k
    assert np.array_equal(f.counts.cpu().numpy(), ref["counts"]) and np.array_equal(f.tokens.cpu().numpy(), ref["tokens"])

    counted = ref["lse"] != -np.inf
    lg64 = np.where(counted[:, None], lg, 0.0).astype(np.float64)
    fin = np.isfinite(lg64)
    top = np.where(fin, lg64, -np.inf).max(axis=1, keepdims=True, initial=-np.inf)
    top = np.where(np.isfinite(top), top, 0.0)
    d = np.where(fin, top - np.where(fin, lg64, top), 0.0)
    z = np.where(fin, np.exp(-d), 0.0)
    tot = np.maximum(z.sum(axis=1, keepdims=True), 1e-300)
    p = z / tot * counted[:, None]
    # each exponential, and the sum of them relative to itself
    r_term = (d + 4) * U
    r_sum = (z * r_term).sum(axis=1, keepdims=True) / tot + (E + 2) * U
    r_p = r_term + r_sum + 4 * U
    lse_err = np.where(counted, r_sum[:, 0] + 2 * U * (np.abs(np.log(tot[:, 0])) + 1) + U * np.abs(top[:, 0]), 0.0)
    within(f.lse, ref["lse"], lse_err, "lse")
    lse0 = np.where(counted, ref["lse"], 0.0)
    seg = np.zeros(T, np.int64)
    ends = [0, T] if cu is None else [min(max(int(c), 0), T) for c in cu]
    prob_err, loss_err, z_err = np.zeros((S, E)), np.zeros(S), np.zeros(S)
    for s in range(S):
        sl = slice(ends[s], max(ends[s], ends[s + 1]))
        seg[sl] = s
        n = float(ref["tokens"][s])
        if not n:
            continue
        prob_err[s] = (p[sl] * r_p[sl]).sum(axis=0) + (n + 8) * U * p[sl].sum(axis=0)
        loss_err[s] = E / (k * n * n) * (ref["counts"][s] * prob_err[s]).sum() + 4 * U * ref["loss"][s]
        z_err[s] = (2 * np.abs(lse0[sl]) * lse_err[sl]).sum() / n + (n + 8) * U * ref["z"][s]
    within(f.prob, ref["prob"], prob_err, "prob")
    within(f.loss, ref["loss"], loss_err, "loss")
    within(f.z_loss, ref["z"], z_err, "z_loss")

    gl, gz = rng.standard_normal(S).astype(np.float32), rng.standard_normal(S).astype(np.float32)
    add = rng.standard_normal((T, E)).astype(np.float32)
    n = np.maximum(ref["tokens"], 1).astype(np.float64)
    a_l, a_z = (np.abs(gl) * E / (k * n * n))[seg][:, None], (np.abs(gz) * 2 / n)[seg][:, None]
    c = ref["counts"][seg].astype(np.float64)
    dot = (c * p).sum(axis=1, keepdims=True)
    dot_err = (c * p * r_p).sum(axis=1, keepdims=True) + (E + 4) * U * dot
    term = p * (a_l * (c + dot) + a_z * np.abs(lse0)[:, None])
    err = p * (a_l * dot_err + a_z * lse_err[:, None]) + term * (r_p + 8 * U) + 2 * U * term
    for name, kw in (("both", dict(grad_loss=gl, grad_z=gz)), ("loss", dict(grad_loss=gl)), ("z", dict(grad_z=gz)),
                     ("neither", {})):
        want = block.balance_backward(ref, np.where(counted[:, None], lg, 0.0), k, cu=cu, add=add, **kw)
        got = e4b.moe_balance_backward(f, lg_d, cu_tokens=cu_d, add=dev(add), **{m: dev(v) for m, v in kw.items()})
        within(got, want, err + 2 * U * (np.abs(add) + term), "grad_logits " + name)
        assert torch.equal(got[torch.from_numpy(~counted).to(DEV)].cpu(), torch.from_numpy(add[~counted]))
    alone = e4b.moe_balance_backward(f, lg_d, dev(gl), dev(gz), cu_tokens=cu_d)
    within(alone, block.balance_backward(ref, np.where(counted[:, None], lg, 0.0), k, gl, gz, cu), err, "grad_logits alone")
    place = dev(add)
    inside = e4b.moe_balance_backward(f, lg_d, dev(gl), dev(gz), cu_tokens=cu_d, add=place, out=place)
    fresh = e4b.moe_balance_backward(f, lg_d, dev(gl), dev(gz), cu_tokens=cu_d, add=dev(add))
    assert inside.data_ptr() == place.data_ptr() and torch.equal(inside.view(torch.int32), fresh.view(torch.int32))
    return f


@pytest.mark.parametrize("T,E,k,S,masked", [
    (1, 1, 1, 1, False), (8, 128, 8, 1, False), (3, 5, 5, 1, True), (64, 60, 4, 1, True), (65, 64, 8, 1, False),
    (200, 128, 8, 1, True), (1000, 7, 2, 1, False), (300, 256, 16, 1, True), (130, 255, 3, 1, True), (77, 257, 9, 1, False),
    (90, 300, 32, 1, True), (70, 512, 8, 1, False), (33, 1000, 4, 1, True), (40, 1024, 32, 1, True), (66, 1023, 1, 1, False),
    (8, 128, 8, 3, False), (1, 16, 2, 2, False), (500, 64, 8, 9, True), (257, 33, 3, 64, True), (700, 8, 2, 65, False),
    (300, 64, 4, 300, True), (50, 12, 2, 4097, False), (9000, 16, 2, 5, True), (0, 8, 2, 1, False), (0, 300, 3, 4, False),
])
def test_balance_and_its_gradient(T, E, k, S, masked):
    announce(f"balance T={T} E={E} k={k} S={S} masked={masked}")
    lg, idx, mask = inputs(T, E, k, masked)
    check(lg, idx, mask, bounds(T, S, np.random.default_rng(S)) if S > 1 else None)


@pytest.mark.parametrize("cu", [[0, 64, 64, 100], [5, 40], [-9, 50, 1000], [0, 0, 0, 100, 100], [100, 100], [30, 31, 32, 33]])
def test_sequences_at_their_edges(cu):
    announce(f"balance sequences {cu}")
    lg, idx, mask = inputs(100, 24, 3, True, seed=1)
    check(lg, idx, mask, cu)


def test_one_sequence_by_bounds_is_the_whole_batch():
    lg, idx, _ = inputs(4000, 64, 8, False, seed=2)
    a = check(lg, idx, None, None)
    b = check(lg, idx, None, [0, 4000])
    for name in ("counts", "tokens", "prob", "loss", "z_loss", "lse"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


def test_bounds_that_do_not_ascend_stay_inside():
    announce("balance with descending bounds")
    lg, idx, _ = inputs(90, 16, 2, False, seed=3)
    for cu in ([0, 80, 10, 90], [90, 0], [2 ** 31 - 1, -2 ** 31, 7], [50, 20, 80, 60, 5]):
        cu_d = torch.tensor(cu, dtype=torch.int32, device=DEV)
        f = e4b.moe_balance(dev(lg), torch.from_numpy(idx).to(DEV), cu_tokens=cu_d)
        S = len(cu) - 1
        e4b.moe_balance_backward(f, dev(lg), torch.ones(S, device=DEV), torch.ones(S, device=DEV), cu_tokens=cu_d)
    torch.cuda.synchronize()


def test_far_logits_and_masked_rows_of_the_lowest_value():
    lg, idx, _ = inputs(80, 32, 4, False, seed=4)
    lg[3] *= 1e4
    lg[4] += 1e6
    lg[5, 1:] = np.finfo(np.float32).min  # a mask of the type's lowest value
    lg[6] = np.finfo(np.float32).min      # throughout: a row like any other of equal logits, with a z loss beyond fp32
    idx = np.argsort(-lg.astype(np.float64), axis=1, kind="stable")[:, :4].astype(np.int32)
    mask = np.ones(80, bool)
    mask[6] = False
    check(lg, idx, mask, None)


def test_a_nan_shows_in_its_own_sequence_only():
    lg, idx, _ = inputs(60, 16, 2, False, seed=5)
    lg[25, 3] = np.nan
    cu = torch.tensor([0, 20, 40, 60], dtype=torch.int32, device=DEV)
    f = e4b.moe_balance(dev(lg), torch.from_numpy(idx).to(DEV), cu_tokens=cu)
    assert f.loss.isnan().tolist() == [False, True, False] and f.z_loss.isnan().tolist() == [False, True, False]
    g = e4b.moe_balance_backward(f, dev(lg), torch.ones(3, device=DEV), torch.ones(3, device=DEV), cu_tokens=cu)
    bad = g.isnan().any(dim=1).nonzero()[:, 0].tolist()
    assert bad == [25]


def test_counts_summed_over_ranks():
    """The gradient of the loss over two ranks' tokens, from each rank's own call."""
    lg, idx, _ = inputs(300, 32, 4, False, seed=6)
    one = torch.ones(1, device=DEV)
    call = lambda s: e4b.moe_balance(dev(lg[s]), torch.from_numpy(idx[s].copy()).to(DEV))  # noqa: E731
    whole = call(slice(None))
    want = e4b.moe_balance_backward(whole, dev(lg), one, one)
    parts = [(s, call(s)) for s in (slice(0, 111), slice(111, 300))]
    counts, tokens = sum(p.counts for _, p in parts), sum(p.tokens for _, p in parts)
    assert torch.equal(counts, whole.counts.to(counts.dtype)) and int(tokens) == 300
    for s, p in parts:
        p.counts.copy_(counts)
        p.tokens.copy_(tokens)
        assert torch.equal(e4b.moe_balance_backward(p, dev(lg[s]), one, one), want[s])


def test_gradient_by_differences():
    """Central differences of the library's own losses: d 2^-6 wide they are off by its square times the
    third derivative (below 1 for p of a few tokens) and by the losses' own few steps over d."""
    lg, idx, _ = inputs(12, 8, 2, False, seed=7)
    idx_d = torch.from_numpy(idx).to(DEV)
    f = e4b.moe_balance(dev(lg), idx_d)
    one = torch.ones(1, device=DEV)
    for name, kw in (("loss", dict(grad_loss=one)), ("z_loss", dict(grad_z=one))):
        g = host(e4b.moe_balance_backward(f, dev(lg), **kw))
        for t, e in ((0, 0), (3, 5), (7, 2), (11, 7)):
            h = 2.0 ** -6
            up, dn = lg.copy(), lg.copy()
            up[t, e] += h
            dn[t, e] -= h
            width = float(up[t, e]) - float(dn[t, e])
            v = [float(getattr(e4b.moe_balance(dev(x), idx_d), name)) for x in (up, dn)]
            size = max(abs(v[0]), 1.0)
            assert abs((v[0] - v[1]) / width - g[t, e]) <= h * h + 64 * U * size / width, (name, t, e)


def test_refusals_on_the_device():
    lg, idx = torch.zeros(4, 8, device=DEV), torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    f = e4b.moe_balance(lg, idx)
    cu = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    one = torch.ones(1, device=DEV)
    bad = [
        lambda: e4b.moe_balance(lg, idx[:3]),
        lambda: e4b.moe_balance(lg.t(), idx),
        lambda: e4b.moe_balance(lg, idx.view(-1)),
        lambda: e4b.moe_balance(lg, torch.zeros(4, 9, dtype=torch.int32, device=DEV)),
        lambda: e4b.moe_balance(lg, idx, cu_tokens=cu[:1]),
        lambda: e4b.moe_balance(lg, idx, cu_tokens=cu.view(1, 3)),
        lambda: e4b.moe_balance(lg, idx, token_mask=torch.ones(3, dtype=torch.bool, device=DEV)),
        lambda: e4b.moe_balance(lg, idx, cu_tokens=cu, workspace=torch.empty(1, device=DEV)),
        lambda: e4b.moe_balance_backward(f, lg, one, cu_tokens=cu),
        lambda: e4b.moe_balance_backward(f, lg, torch.ones(2, device=DEV)),
        lambda: e4b.moe_balance_backward(f, lg, one, add=lg[:3]),
        lambda: e4b.moe_balance_backward(f, lg, one, out=lg),
        lambda: e4b.moe_balance_backward(f, torch.zeros(5, 8, device=DEV), one),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    for call in (lambda: e4b.moe_balance(lg.bfloat16(), idx), lambda: e4b.moe_balance(lg, idx.long()),
                 lambda: e4b.moe_balance(lg, idx, token_mask=torch.ones(4, device=DEV)),
                 lambda: e4b.moe_balance(lg, idx, cu_tokens=cu.long()), lambda: e4b.moe_balance_backward(f, lg, one.double())):
        with pytest.raises(TypeError):
            call()


def test_two_runs_another_stream_and_a_graph():
    """The same bits on every run, on another stream, and captured and replayed on new inputs with eager
    runs between the replays (workspaces of garbage)."""
    T, E, k = 3000, 48, 4
    lg, idx, mask = inputs(T, E, k, True, seed=8)
    cu = torch.from_numpy(bounds(T, 7, np.random.default_rng(0))).to(DEV)
    mask_d = torch.from_numpy(mask).to(DEV)
    gl, gz, add = torch.randn(7, device=DEV), torch.randn(7, device=DEV), torch.randn(T, E, device=DEV)
    need = e4b.moe_balance_workspace_bytes(dev(lg), k, cu)

    def both(lg_d, idx_d, ws):
        f = e4b.moe_balance(lg_d, idx_d, cu_tokens=cu, token_mask=mask_d, workspace=ws)
        return [f.counts, f.tokens, f.prob, f.loss, f.z_loss, f.lse,
                e4b.moe_balance_backward(f, lg_d, gl, gz, cu_tokens=cu, add=add)]

    bits = lambda ts: [t.view(torch.int32) for t in ts]  # noqa: E731
    same = lambda a, b: all(torch.equal(p, q) for p, q in zip(bits(a), bits(b)))  # noqa: E731
    garbage = lambda: torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)  # noqa: E731
    lg_d, idx_d, ws = dev(lg), torch.from_numpy(idx).to(DEV), garbage()
    want = both(lg_d, idx_d, None)
    assert same(want, both(lg_d, idx_d, garbage()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = both(lg_d, idx_d, ws)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert same(want, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(lg_d, idx_d, ws)
    for rep in range(4):
        lg2, idx2, _ = inputs(T, E, k, True, seed=20 + rep)
        lg_d.copy_(dev(lg2))
        idx_d.copy_(torch.from_numpy(idx2).to(DEV))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, both(dev(lg2), torch.from_numpy(idx2).to(DEV), None)), rep
