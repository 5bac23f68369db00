"""GPU tests of the router's balance on batches of millions of tokens."""

import pytest
import torch

import bit_quantized_mixture_nf4_amd as e4b
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _parts(T, n=1 << 18):
    return [slice(a, min(a + n, T)) for a in range(0, T, n)]


@pytest.mark.parametrize("T,E,k,cu,masked", [
    ((1 << 24) - 1, 4, 2, None, True), ((1 << 24) - 1, 7, 2, [3, 9, 9, 5000000, (1 << 24) - 9], False),
    (2100000, 64, 8, [0, 1, 1000000, 2100000], True), (4300000, 512, 2, [7, 4300000], False)])
def test_millions_of_tokens(T, E, k, cu, masked):
    """Against the definition in 64 bits, summed by torch part by part (the last batch's logits lie beyond 2^31
    values). A probability is off by E + 8 steps and d (the distance to the row's largest) half steps, d below 24 here;
    a sum of n values in the kernels' order by 2 log2(n) + n / 2^13 steps at most: a lane adds up at most n / 2^13 of
    them in turn, and so does the join's row by row, before they are joined."""
    announce(f"balance T={T} E={E} k={k} cu={cu}")
    gen = torch.Generator(device=DEV).manual_seed(E)
    lg = torch.randn(T, E, device=DEV, generator=gen).add_(torch.randn(E, device=DEV, generator=gen))
    idx = torch.randint(0, E, (T, k), device=DEV, generator=gen, dtype=torch.int32)
    mask = torch.rand(T, device=DEV, generator=gen) > 0.25 if masked else None
    cu_d = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    f = e4b.moe_balance(lg, idx, cu_tokens=cu_d, token_mask=mask)
    ends = cu or [0, T]
    S = len(ends) - 1
    gl, gz = torch.linspace(1, 2, S, device=DEV), torch.linspace(-1, 1, S, device=DEV)
    add = torch.ones(T, E, device=DEV)
    grad = e4b.moe_balance_backward(f, lg, gl, gz, cu_tokens=cu_d, add=add, out=add)
    assert grad.data_ptr() == add.data_ptr()
    r_p, r_lse = (E + 8 + 24) * U, (E + 8 + 24) * U
    outside = torch.ones(T, dtype=torch.bool, device=DEV)
    for s in range(S):
        a, b = ends[s], ends[s + 1]
        outside[a:b] = False
        if mask is not None:
            outside[a:b] = ~mask[a:b]
        counts = torch.zeros(E, dtype=torch.int64, device=DEV)
        prob, z, n = torch.zeros(E, dtype=torch.float64, device=DEV), 0.0, 0
        kept = []
        for part in _parts(b - a):
            t = slice(a + part.start, a + part.stop)
            live = torch.ones(t.stop - t.start, dtype=torch.bool, device=DEV) if mask is None else mask[t]
            rows = lg[t][live].double()
            lse = torch.logsumexp(rows, 1)
            assert ((f.lse[t][live].double() - lse).abs() <= r_lse * (1 + lse.abs())).all()
            prob += torch.exp(rows - lse[:, None]).sum(0)
            z, n = z + float(lse.square().sum()), n + rows.shape[0]
            counts += torch.bincount(idx[t][live].view(-1).long(), minlength=E)
            kept.append((t, live))
        assert int(f.tokens[s]) == n and torch.equal(f.counts[s].long(), counts)
        if not n:
            assert float(f.loss[s]) == float(f.z_loss[s]) == 0.0 and not f.prob[s].any()
            continue
        r_sum = (2 * 24 + n / 2 ** 13) * U
        assert ((f.prob[s].double() - prob).abs() <= (r_p + r_sum) * prob).all()
        want = E / (k * n * n) * float((counts.double() * prob).sum())
        assert abs(float(f.loss[s]) - want) <= (r_p + r_sum + 4 * U) * want
        assert abs(float(f.z_loss[s]) - z / n) <= (8 * r_lse + r_sum) * (z / n + 1)
        # the gradient of the first and last part's tokens
        factor = float(gl[s]) * E / (k * n * n)
        for t, live in {0: kept[0], 1: kept[-1]}.values():
            rows = lg[t][live].double()
            lse = torch.logsumexp(rows, 1, keepdim=True)
            p, c, zf = torch.exp(rows - lse), counts.double(), float(gz[s]) * 2 / n
            dot = (p * c).sum(1, keepdim=True)
            g = 1 + p * (factor * (c - dot) + zf * lse)
            # dot is off by r_p and E + 4 steps of its terms, lse by r_lse (1 + |lse|); the terms, c - dot no smaller
            # than which may cancel, by r_p and 8 steps of products and sums; 1 + them by a step of both
            terms = p * (abs(factor) * (c + dot) + abs(zf) * lse.abs())
            err = terms * (r_p + 8 * U) + p * (abs(factor) * dot * (r_p + (E + 4) * U) + abs(zf) * r_lse * (1 + lse.abs()))
            assert ((grad[t][live].double() - g).abs() <= err + 2 * U * (1 + terms)).all()
    for part in _parts(T):
        off = outside[part]
        assert f.lse[part][off].eq(-float("inf")).all() and grad[part][off].eq(1.0).all()
