"""GPU checks of the expert router and its gradient against the oracle; choices and counts are exact.

Tolerances, with u = 2^-24: a logit's distance to the row's largest is off by u of itself and the
exponential by 4 u, so a softmax term by (5 + d) u of it, d the largest such distance; a sum of E such
terms adds E u, the division 1 u.  A weight is then off by 2 (E + d + 8) u of itself, a sum over T tokens
by (T + E + d + 16) u more, the loss (products of both) by twice that.  A gradient is a sum of at most E +
top_k terms of a few such factors: 8 (E + top_k + d + 8) u of its terms' magnitudes, plus the rounding
to its type."""
import numpy as np
import pytest
import torch

import oracle as O
from mxfp4_microscaling_quantization_amd import mx
from tests.gpu_util import DEV, assert_bytes_equal, host, oracle_input
from tests.test_gpu_moe_routing import STEP, dev_f32, stored, strided, torch_type, values

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SIZES = [(1, 1, 1), (1, 2, 2), (3, 8, 2), (16, 16, 16), (17, 17, 3), (24, 32, 4), (65, 33, 1), (100, 128, 8), (256, 5, 4),
         (257, 60, 6), (300, 64, 8), (4100, 100, 2), (1000, 128, 16),
         (33, 128, 8), (64, 30, 3), (8192, 12, 2), (8193, 70, 3)]


def inputs(rng, tokens, experts, dtype, ties=False):
    x = rng.integers(-2, 3, (tokens, experts)) * 1.0 if ties else rng.standard_normal((tokens, experts)) * 3
    if tokens > 3 and experts > 1:
        x[:, rng.integers(0, experts)] = -np.inf          # an expert that is closed
        x[2] = -np.inf                                    # a token without any
        x[3, 1:] = -np.inf                                # a token with one at most
    return stored(x, dtype)


def distance(v):
    f = np.where(np.isfinite(v), v, np.nan)
    f = f[np.isfinite(v).any(axis=1)]
    return float(np.nanmax(np.nanmax(f, axis=1) - np.nanmin(f, axis=1))) if len(f) else 0.0


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,experts,top_k", SIZES)
def test_forward_and_backward(tokens, experts, top_k, dtype, renormalize):
    rng = np.random.default_rng(tokens + experts)
    for ties, masked in ((False, True), (True, False)):
        a = inputs(rng, tokens, experts, dtype, ties)
        v = oracle_input(a, dtype)
        mask = rng.random(tokens) < 0.8 if masked else None
        dead = np.zeros(tokens, bool) if mask is None else ~mask
        x = strided(a, dtype, experts + 3)
        x[torch.from_numpy(dead).to(DEV)] = float("nan")   # a masked token's logits are not looked at
        m = None if mask is None else torch.from_numpy(mask).to(DEV)
        want = O.route(v, top_k, renormalize, mask)
        ids, p, counts, sums, loss = mx.moe_route(x, top_k, renormalize, m)
        assert_bytes_equal(host(ids), want[0], "ids")
        assert_bytes_equal(host(counts), want[2], "counts")
        d = distance(v)
        few = (experts + d + 8) * U
        assert np.all(np.abs(values(p) - want[1]) <= 2 * few * want[1])
        many = (tokens + experts + d + 16) * U
        assert np.all(np.abs(values(sums) - want[3]) <= (2 * few + many) * want[3])
        assert abs(values(loss)[0] - want[4]) <= 2 * (2 * few + many) * want[4] + U * want[4]
        dp = rng.standard_normal((tokens, top_k)).astype(np.float32)
        dp[host(ids) < 0] = np.nan
        dloss = dev_f32([0.7])
        for g, dl in ((dp, 0.7), (None, 0.7), (dp, 0.0)):
            got = mx.moe_route_bwd(x, ids, counts, None if g is None else dev_f32(g), dloss if dl else None, renormalize, m)
            w, mag = O.route_bwd(v, want[0], want[2], np.zeros_like(dp) if g is None else g, float(np.float32(dl)),
                                 renormalize, mask)
            tol = 8 * (experts + top_k + d + 8) * U * mag + STEP[dtype] * np.abs(w) + 2.0 ** -130
            assert got.dtype == torch_type(dtype)
            err = np.abs(values(got) - w)
            assert np.all(err <= tol), (float((err / tol).max()), ties)


def test_many_tokens_and_repeated_calls():
    tokens, experts, top_k = 70000, 32, 4
    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randn((tokens, experts), generator=g, device=DEV)
    first = mx.moe_route(x, top_k)
    s = torch.softmax(x.double(), dim=1)
    top = torch.topk(s, top_k, dim=1)
    assert torch.equal(first[0].long(), top.indices)
    counts = torch.bincount(top.indices.flatten(), minlength=experts)
    assert torch.equal(first[2].long(), torch.cat((counts, torch.tensor([tokens], device=DEV))))
    sums = s.sum(dim=0)
    assert torch.all((first[3].double() - sums).abs() <= (tokens + 2 * experts + 80) * U * sums)
    loss = experts * (counts.double() / (tokens * top_k) * sums / tokens).sum()
    assert abs(first[4].double() - loss) <= 2 * (tokens + 2 * experts + 80) * U * loss
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(mx.moe_route(x, top_k), first))


def test_no_token_takes_part():
    x = torch.full((300, 8), float("-inf"), device=DEV)
    for logits, mask in ((x, None), (torch.randn_like(x), torch.zeros(300, dtype=torch.bool, device=DEV)),
                         (x[:0], None)):
        ids, p, counts, sums, loss = mx.moe_route(logits, 2, mask=mask)
        assert torch.all(ids == -1) and not p.any() and not counts.any() and not sums.any() and not loss.any()
        d = mx.moe_route_bwd(logits, ids, counts, torch.ones_like(p), torch.ones(1, device=DEV), mask=mask)
        assert d.shape == logits.shape and not d.any()


def test_nan_and_infinite_logits():
    x = torch.randn((4, 6), device=DEV)
    x[1, 2], x[2, 4] = float("nan"), float("inf")
    ids, p, counts, sums, loss = mx.moe_route(x, 2)
    assert torch.isnan(p[1:3]).all() and torch.isfinite(p[[0, 3]]).all() and torch.isnan(loss).all()
    assert not (ids[1] == 2).any() and ids[2, 0] == 4 and counts[-1] == 4
    d = mx.moe_route_bwd(x, ids, counts, torch.ones_like(p))
    assert torch.isnan(d[1:3]).all() and torch.isfinite(d[[0, 3]]).all()
    x[1] = float("-inf")
    x[1, 0] = float("nan")                              # NaN alone is open
    ids, p, counts, _, loss = mx.moe_route(x, 2)
    assert torch.all(ids[1] == -1) and counts[-1] == 4 and torch.isnan(loss).all()


@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_against_differences(renormalize):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 12)).astype(np.float32)
    dp = rng.standard_normal((40, 3)).astype(np.float32)
    ids, p, counts, _, _ = mx.moe_route(dev_f32(x), 3, renormalize)
    d = values(mx.moe_route_bwd(dev_f32(x), ids, counts, dev_f32(dp), dev_f32([5.0]), renormalize))
    step = 2.0 ** -8

    def value(v):
        i, p, _, _, loss = mx.moe_route(dev_f32(v), 3, renormalize)
        assert torch.equal(i, ids)
        return (values(p) * dp).sum(axis=1), values(loss)[0]

    order = np.sort(x, axis=1)
    safe = np.nonzero((np.diff(order, axis=1).min(axis=1) > 4 * step))[0]
    for t, e in [(t, e) for t in safe[:3] for e in range(12)]:
        up, down = x.copy(), x.copy()
        up[t, e] += step
        down[t, e] -= step
        (a, la), (b, lb) = value(up), value(down)
        diff = ((a - b)[t] + 5.0 * (la - lb)) / (2 * step)
        # third derivatives of a softmax term are below 1; float32 weights and loss around 1
        assert abs(diff - d[t, e]) < (np.abs(dp[t]).sum() + 5) * step ** 2 + (np.abs(dp[t]).sum() + 5) * 32 * U / step


def test_streams_and_graphs():
    x = torch.randn((3000, 40), device=DEV)
    dp, dl = torch.randn((3000, 4), device=DEV), torch.ones(1, device=DEV)

    def step(stream=None):
        r = mx.moe_route(x, 4, stream=stream)
        return (*r, mx.moe_route_bwd(x, r[0], r[2], dp, dl, stream=stream))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        x.copy_(torch.randn_like(x))
        want = step()
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def lanes(experts):
    """Experts of a lane: 16 lanes hold a token."""
    return 1 if experts <= 16 else 2 if experts <= 32 else 4 if experts <= 64 else 8


@pytest.mark.parametrize("tokens,experts,top_k,dtype,renormalize", [
    (70000, 32, 4, torch.float32, True), (70001, 128, 8, torch.bfloat16, False), (66000, 7, 2, torch.float32, False),
    (140000, 60, 6, torch.bfloat16, True)])
def test_many_masked_tokens_in_loops(tokens, experts, top_k, dtype, renormalize):
    """More tokens than 256 workgroups hold at once, forward and backward, some masked: every row.

    The kernel's own chains set the bounds, with u, d as above and L experts a lane.  An exponential is off by (4 + d) u,
    a row's sum by L + 3 roundings more, so a softmax term by (2 d + L + 12) u of it.  A lane adds one token a pass,
    passes = tokens / (256 * 64), two exchanges follow, the workgroup's sum and the whole are rounded once each and
    added in float64 between: (2 d + L + 16 + passes) u of sums, and of the loss, whose counts are exact.  A weight
    divided by the sum of its choices: (2 d + top_k + 9) u.  (A pass left out of sums would be 64 / tokens = 9e-4 of
    them, 15000 u.)"""
    g = torch.Generator(device=DEV).manual_seed(tokens)
    x = (3 * torch.randn((tokens, experts), generator=g, device=DEV)).to(dtype)
    mask = torch.rand(tokens, generator=g, device=DEV) < 0.8
    x[:, experts // 2] = float("-inf")            # an expert that is closed
    x[11:tokens:1000] = float("-inf")             # tokens without any
    part = mask & (x > float("-inf")).any(dim=1)
    v = torch.where(part[:, None], x.double(), float("-inf"))
    x[~mask] = float("nan")                       # a masked token's logits are not looked at
    s = torch.softmax(torch.where(part[:, None], v, 0.0), dim=1) * part[:, None]
    finite = torch.where(v > float("-inf"), v, float("nan"))[part]
    d = float((v[part].max(dim=1).values - torch.nan_to_num(finite, nan=float("inf")).min(dim=1).values).max())
    term = 2 * d + lanes(experts) + 12
    order = torch.sort(v, dim=1, descending=True, stable=True)
    choice = order.indices[:, :top_k]
    there = order.values[:, :top_k] > float("-inf")
    weight = torch.gather(s, 1, choice) * there
    share = weight.sum(dim=1, keepdim=True) if renormalize else torch.ones((tokens, 1), dtype=torch.float64, device=DEV)
    share = torch.where(part[:, None], share, 1.0)
    n, slots = int(part.sum()), torch.bincount(choice[there], minlength=experts)

    ids, p, counts, sums, loss = mx.moe_route(x, top_k, renormalize, mask)
    assert torch.equal(ids.long(), torch.where(there, choice, -1))
    assert torch.equal(counts.long(), torch.cat((slots, torch.tensor([n], device=DEV))))
    want = weight / share
    assert torch.all((p.double() - want).abs() <= (2 * d + top_k + 9 if renormalize else term) * U * want)
    passes = -(-tokens // (256 * 64))
    want = s.sum(dim=0)
    assert passes > 4 and torch.all((sums.double() - want).abs() <= (term + 4 + passes) * U * want)
    want = experts * float((slots.double() * want).sum()) / (n * n * top_k)
    assert abs(float(loss) - want) <= (term + 4 + passes) * U * want

    dp = torch.randn((tokens, top_k), generator=g, device=DEV)
    dp = torch.where(there, dp, float("nan"))     # nor at the gradients of slots left out
    value = torch.where(there, dp.double(), 0.0)
    for dloss in (None, 0.7 * n):                 # the loss's gradients as large as the weights'
        d_loss = None if dloss is None else torch.full((1,), dloss, device=DEV)
        G0 = (0.0 if dloss is None else float(d_loss)) * experts * slots.double() / (n * n * top_k)
        inner = (weight / share * value).sum(dim=1, keepdim=True) * renormalize
        bound = (weight / share * value.abs()).sum(dim=1, keepdim=True) * renormalize
        G = G0.expand(tokens, experts).scatter_add(1, choice, torch.where(there, (value - inner) / share, 0.0))
        A = G0.expand(tokens, experts).scatter_add(1, choice, torch.where(there, (value.abs() + bound) / share, 0.0))
        want = s * (G - (s * G).sum(dim=1, keepdim=True))
        mag = s * (A + (s * A).sum(dim=1, keepdim=True))
        got = mx.moe_route_bwd(x, ids, counts, dp, d_loss, renormalize, mask)
        step = STEP["bf16" if dtype == torch.bfloat16 else "f32"]
        tol = 8 * (experts + top_k + d + 8) * U * mag + step * want.abs() + 2.0 ** -130
        bad = ~((got.double() - want).abs() <= tol)
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
        assert not got[~part].any()
