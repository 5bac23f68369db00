"""GPU tests of the router's balance on arguments that are parts of longer tensors."""

import numpy as np
import pytest
import torch

import bit_quantized_mixture_nf4_amd as e4b
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu


def _batch(T=300, E=24, k=3, seed=0):
    rng = np.random.default_rng(seed)
    lg = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
    mask = torch.from_numpy(rng.random(T + 40) > 0.3).to(DEV)
    cu = torch.from_numpy(np.concatenate([[-1] * 9, np.sort(rng.integers(0, T + 1, 7))]).astype(np.int32)).to(DEV)
    return lg, e4b.moe_route(lg, k)[0], mask, cu


def _both(lg, idx, cu, mask, workspace=None):
    f = e4b.moe_balance(lg, idx, cu_tokens=cu, token_mask=mask, workspace=workspace)
    S = f.loss.shape[0]
    weights = torch.arange(1.0, S + 1, device=DEV), torch.full((S,), 0.5, device=DEV)
    return [f.counts, f.tokens, f.prob, f.loss, f.z_loss, f.lse, e4b.moe_balance_backward(f, lg, *weights, cu_tokens=cu)]


def _same(a, b):
    return all(torch.equal(p.view(torch.int32), q.view(torch.int32)) for p, q in zip(a, b))


@pytest.mark.parametrize("first", [0, 1, 3, 8, 16, 33])
def test_parts_of_longer_masks_and_bounds(first):
    announce(f"balance of views that begin at {first}")
    lg, idx, mask, cu = _batch()
    m = mask[first:first + lg.shape[0]]
    for c in [None] + [cu[at:] for at in (9, 10, 11, 12)]:
        want = _both(lg, idx, None if c is None else c.clone(), m.clone())
        assert _same(_both(lg, idx, c, m), want) and _same(_both(lg, idx, c, m.clone()), want)
        need = e4b.moe_balance_workspace_bytes(lg, idx.shape[1], c)
        assert need == e4b.moe_balance_workspace_bytes(lg, idx.shape[1], None if c is None else c.clone()) > 0
        assert _same(_both(lg, idx, c, m, torch.empty(need, dtype=torch.uint8, device=DEV)), want)


def test_a_captured_call_reads_the_views_again():
    announce("balance of views in a graph")
    lg, idx, mask, cu = _batch(seed=1)
    T = lg.shape[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _both(lg, idx, cu[10:], mask[5:5 + T])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _both(lg, idx, cu[10:], mask[5:5 + T])
    for rep in range(4):
        lg2, idx2, mask2, cu2 = _batch(seed=10 + rep)
        for a, b in ((lg, lg2), (idx, idx2), (mask, mask2), (cu, cu2)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert _same(out, _both(lg2, idx2, cu2[10:].clone(), mask2[5:5 + T].clone())), rep


@pytest.mark.parametrize("first", [1, 2, 4, 7])
def test_parts_of_longer_selections_and_gradients(first):
    announce(f"balance of selections that begin at {first}")
    lg, idx, _, cu = _batch(T=203, k=2, seed=3)
    cu = cu[9:].clamp(max=200)
    lg, idx = lg[first:first + 196], idx[first:first + 196]
    f, want = e4b.moe_balance(lg, idx, cu_tokens=cu), e4b.moe_balance(lg, idx.clone(), cu_tokens=cu)
    assert _same([f.counts, f.prob, f.loss, f.lse], [want.counts, want.prob, want.loss, want.lse])
    g = torch.randn(2, 16, device=DEV)
    gl, gz = g[0, first:first + 6], g[1, first:first + 6]
    assert _same([e4b.moe_balance_backward(f, lg, gl, gz, cu_tokens=cu)],
                 [e4b.moe_balance_backward(f, lg, gl.clone(), gz.clone(), cu_tokens=cu)])


def test_no_place_among_what_is_read():
    lg, idx, _, _ = _batch(T=40, E=8, k=2)
    f = e4b.moe_balance(lg, idx)
    one = torch.ones(1, device=DEV)
    place = torch.zeros(2, 40, 8, device=DEV)
    lse = place[0].view(-1)[100:140].copy_(f.lse)
    inside = e4b.Balance(f.counts, f.tokens, f.prob, f.loss, f.z_loss, lse, f.top_k)
    counts = e4b.Balance(place[0].view(torch.int32)[3:4].copy_(f.counts), f.tokens, f.prob, f.loss, f.z_loss, f.lse, f.top_k)
    for call in (lambda: e4b.moe_balance_backward(inside, lg, one, out=place[0]),
                 lambda: e4b.moe_balance_backward(counts, lg, one, out=place[0]),
                 lambda: e4b.moe_balance_backward(f, lg, place[0, 5, :1], out=place[0]),
                 lambda: e4b.moe_balance_backward(f, lg, one, place[0, 39, 7:], out=place[0]),
                 lambda: e4b.moe_balance_backward(f, lg, one, add=place.view(-1)[8:328].view(40, 8), out=place[0])):
        with pytest.raises(ValueError, match="overlap"):
            call()
    want = e4b.moe_balance_backward(f, lg, one)
    assert _same([e4b.moe_balance_backward(f, lg, one, out=place[1])], [want])  # next to them is a place
