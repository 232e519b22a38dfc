"""Routing and the experts' block against the fp64 oracle.

Tolerances. Choices are compared exactly, on logits whose keys are either equal
or at least 2^-12 apart. Weights are fp32 quotients of exponentials (2 ulp each,
sums of at most 1024 in a tree): within 2^-18 relative. The experts' block is
held to the bound the oracle carries through both products, with chains of at
most K / 32 + 160 fp32 additions and h rounded to 2^-8 (bf16), 2^-11 (fp16).
"""

import numpy as np
import pytest

from oracle import mx

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lutq():
    import weight_only_lut_amd as m
    m.load_library()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def spaced_logits(rng, T, E, ties=True):
    """Logits on a grid of 2^-4 (exact in every type), each row's in random order; with repeats if asked."""
    l = np.stack([rng.permutation(E) for _ in range(T)]).astype(np.float64)
    if ties:
        l = np.floor(l / 2)
    return (l - E / 4) * min(0.0625, 16.0 / E)


def check(r, logits, k, **kw):
    ids, w = mx.route(f64(logits), k, **kw)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.allclose(f64(r.weights), w, rtol=2.0 ** -18, atol=1e-30, equal_nan=True)
    offsets, order = mx.plan(ids, logits.shape[1])
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.order.cpu().numpy(), order)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (3, 5, 5), (64, 16, 2), (65, 60, 4), (70, 128, 32),
                                   (700, 96, 3), (300, 200, 8), (33, 513, 10), (2, 1024, 32), (1, 1000, 6)])
def test_softmax_routing(lutq, T, E, k, dtype):
    l = torch.from_numpy(spaced_logits(np.random.default_rng(T + E), T, E)).to(dtype).cuda()
    check(lutq.moe_route(l, k), l, k)
    check(lutq.moe_route(l, k, renorm=False, scale=0.5), l, k, renorm=False, scale=0.5)


@pytest.mark.parametrize("T,E,k,groups,top_groups,best", [
    (1, 64, 6, 8, 3, 2), (9, 256, 8, 8, 4, 2), (700, 256, 8, 8, 4, 1), (5, 12, 3, 6, 2, 2), (40, 60, 4, 3, 1, 1),
    (3, 64, 4, 64, 7, 1), (2, 1024, 8, 32, 4, 2), (17, 96, 8, 1, 1, 2)])
def test_sigmoid_routing_with_bias_and_groups(lutq, T, E, k, groups, top_groups, best):
    rng = np.random.default_rng(E + k)
    # keys: sigmoids of a few values, biases a grid that keeps distinct keys apart
    l = dev(rng.choice([-1.5, -0.5, 0.5, 2.0], (T, E)).astype(np.float32))
    bias = dev((rng.integers(-4, 5, E) / 16).astype(np.float32))
    kw = dict(score="sigmoid", groups=groups, top_groups=top_groups, group_best=best, scale=2.5)
    check(lutq.moe_route(l, k, bias=bias, **kw), l, k, bias=bias.cpu().numpy(), **kw)
    check(lutq.moe_route(l, k, renorm=False, **kw), l, k, renorm=False, **kw)


def test_softmax_routing_with_bias(lutq):
    rng = np.random.default_rng(2)
    l = dev(np.log(rng.choice([1.0, 2.0, 4.0, 8.0], (30, 32))).astype(np.float32))
    bias = dev((np.arange(32) / 7).astype(np.float32))     # steps of 1/7 order the experts by themselves
    check(lutq.moe_route(l, 5, bias=bias), l, 5, bias=bias.cpu().numpy())
    check(lutq.moe_route(l, 5, bias=bias, renorm=False), l, 5, bias=bias.cpu().numpy(), renorm=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [6, 300])
def test_masked_experts_and_empty_rows(lutq, T, score):
    """Rows of -infinity choose nothing; rows with fewer experts than places fill up with -1."""
    rng = np.random.default_rng(T)
    l = spaced_logits(rng, T, 24, ties=False)
    l[rng.random((T, 24)) < 0.7] = -np.inf
    l[1] = l[T - 1] = -np.inf
    l[2, :] = -np.inf
    l[2, 23] = -3.0e38
    l[3, 0] = np.nan if score == "sigmoid" else 1.0
    l = dev(l.astype(np.float32))
    check(lutq.moe_route(l, 8, score=score), l, 8, score=score)
    check(lutq.moe_route(l, 8, score=score, groups=4, top_groups=2), l, 8, score=score, groups=4, top_groups=2)
    allinf = torch.full((T, 24), float("-inf"), device="cuda")
    r = lutq.moe_route(allinf, 3, score=score)
    assert bool((r.ids == -1).all()) and not r.weights.any() and not r.offsets.any() and bool((r.order == -1).all())


def test_nan_and_infinite_softmax_rows(lutq):
    l = torch.zeros(3, 8)
    l[0, 3], l[1, 5], l[2, 6] = float("nan"), float("inf"), 60000.0
    l = l.cuda()
    r = lutq.moe_route(l, 2)
    assert r.ids.tolist() == [[0, 1], [5, 0], [6, 0]]
    assert bool(torch.isnan(r.weights[:2]).all()) and r.weights[2].tolist() == [1.0, 0.0]


def test_strided_logits_and_a_negative_zero(lutq):
    wide = torch.randn(50, 80, device="cuda")
    l = wide[:, 3:67]
    check(lutq.moe_route(l, 4), l, 4)
    l = torch.tensor([[-0.0, 0.0, -0.0, -1.0]], device="cuda")
    assert lutq.moe_route(l, 3).ids.tolist() == [[0, 1, 2]]


@pytest.mark.parametrize("T,E,k", [(0, 8, 2), (4, 8, 2), (300, 16, 4), (5000, 64, 6), (2049, 1024, 1), (3000, 3, 3)])
def test_plan_of_given_ids(lutq, T, E, k):
    rng = np.random.default_rng(T + E)
    # a skewed spread, with ids outside the range
    ids = (E * rng.random((T, k)) ** 3).astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    ids[rng.random((T, k)) < 0.05] = E + 3
    r = lutq.moe_plan(dev(ids), torch.zeros((T, k), device="cuda"), E)
    offsets, order = mx.plan(ids, E)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets) and np.array_equal(r.order.cpu().numpy(), order)


def test_large_routing_is_a_stable_grouping(lutq):
    T, E, k = 40000, 256, 8
    l = torch.randn(T, E, device="cuda")
    r = lutq.moe_route(l, k)
    top = torch.sort(l, dim=-1, descending=True, stable=True)[1][:, :k]
    assert torch.equal(r.ids, top.int())
    assert torch.equal(r.order, torch.sort(top.reshape(-1), stable=True)[1].int())
    again = lutq.moe_route(l, k)
    assert torch.equal(again.order, r.order) and torch.equal(again.weights, r.weights)


# ---- the experts' block ---------------------------------------------------------------

def experts(rng, E, D, F):
    def one(N, K):
        return (rng.integers(0, 256, (E, N, K // 2)).astype(np.uint8),
                rng.integers(118, 122, (E, N, K // 32)).astype(np.uint8))
    return one(2 * F, D), one(D, F)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,D,F", [
    (1, 4, 2, 64, 32), (1, 16, 16, 96, 160), (2, 40, 20, 64, 64), (7, 8, 3, 160, 96), (16, 8, 4, 128, 64),
    (40, 60, 6, 96, 32), (90, 4, 2, 288, 224), (150, 3, 1, 64, 320), (300, 5, 2, 32, 64), (64, 1, 1, 544, 96),
    # row tiles of 16, 32 and 64 with enough of them for the wide columns, and widths that end inside a tile
    (24, 64, 2, 96, 64), (600, 40, 2, 1056, 544), (1500, 3, 3, 800, 416), (900, 64, 4, 96, 2080)])
def test_moe_mlp(lutq, T, E, k, D, F, dtype):
    rng = np.random.default_rng(T * 3 + E + D)
    gu, dn = experts(rng, E, D, F)
    x = torch.from_numpy(rng.standard_normal((T, D)) / 8).to(dtype).cuda()
    l = rng.standard_normal((T, E)) + np.linspace(0, 2, E)      # some experts full, some empty
    l[rng.random((T, E)) < 0.2] = -np.inf
    if T > 2:
        l[T // 2] = -np.inf                                     # a token without experts
    r = lutq.moe_route(dev(l.astype(np.float32)), k)
    y = lutq.moe_mlp(x, lutq.mx_pack(dev(gu[0]), dev(gu[1])), lutq.mx_pack(dev(dn[0]), dev(dn[1])), r)
    u = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    ref, err = mx.moe_mlp(f64(x), mx.dequantize(*gu), mx.dequantize(*dn), r.ids.cpu().numpy(), f64(r.weights), u,
                          D / 32 + 160, F / 32 + 160)
    bound = err + u * (np.abs(ref) + err) + 2.0 ** -24
    assert (np.abs(f64(y) - ref) <= bound).all(), float((np.abs(f64(y) - ref) / bound).max())
    if T > 2:
        assert not y[T // 2].any()


def test_few_tokens_keep_h_above_16_bits(lutq):
    """With few pairs h is not rounded to bf16, so y is within its own rounding and 2^-15 of h."""
    rng = np.random.default_rng(12)
    E, D, F = 8, 256, 512
    gu, dn = experts(rng, E, D, F)
    W = lutq.mx_pack(dev(gu[0]), dev(gu[1])), lutq.mx_pack(dev(dn[0]), dev(dn[1]))
    for T in (1, 3):
        x = torch.from_numpy(rng.standard_normal((T, D)) / 8).to(torch.bfloat16).cuda()
        r = lutq.moe_route(torch.randn(T, E, device="cuda"), 4)
        ref, err = mx.moe_mlp(f64(x), mx.dequantize(*gu), mx.dequantize(*dn), r.ids.cpu().numpy(),
                              f64(r.weights), 2.0 ** -15, D / 32 + 160, F / 32 + 160)
        bound = err + 2.0 ** -8 * (np.abs(ref) + err)
        assert (np.abs(f64(lutq.moe_mlp(x, *W, r)) - ref) <= bound).all()


@pytest.mark.parametrize("T", [1, 13, 400])
def test_moe_mlp_with_another_routers_ids(lutq, T):
    """ids and weights of the caller's own; an id outside the range is no expert,
    also where its weight is NaN, and a repeated expert counts twice."""
    rng = np.random.default_rng(T)
    E, D, F, k = 6, 64, 96, 3
    gu, dn = experts(rng, E, D, F)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[0] = [2, 9, 2]
    w = rng.random((T, k)).astype(np.float32)
    w[0, 1] = np.nan
    x = torch.from_numpy(rng.standard_normal((T, D)) / 8).to(torch.bfloat16).cuda()
    r = lutq.moe_plan(dev(ids), dev(w), E)
    y = lutq.moe_mlp(x, lutq.mx_pack(dev(gu[0]), dev(gu[1])), lutq.mx_pack(dev(dn[0]), dev(dn[1])), r)
    ref, err = mx.moe_mlp(f64(x), mx.dequantize(*gu), mx.dequantize(*dn), ids, w.astype(np.float64), 2.0 ** -8,
                          D / 32 + 160, F / 32 + 160)
    bound = err + 2.0 ** -8 * (np.abs(ref) + err)
    assert (np.abs(f64(y) - ref) <= bound).all()


def test_moe_mlp_strided_rows_out_and_empty(lutq):
    rng = np.random.default_rng(1)
    E, D, F = 4, 96, 64
    gu, dn = experts(rng, E, D, F)
    W = lutq.mx_pack(dev(gu[0]), dev(gu[1])), lutq.mx_pack(dev(dn[0]), dev(dn[1]))
    for T in (3, 50, 200):
        wide = torch.full((T, D + 16), float("nan"), dtype=torch.float16, device="cuda")
        wide[:, 8:8 + D] = torch.randn(T, D, device="cuda").half() / 8
        r = lutq.moe_route(torch.randn(T, E, device="cuda"), 2)
        out = torch.empty((T, D), dtype=torch.float16, device="cuda")
        y = lutq.moe_mlp(wide[:, 8:8 + D], *W, r, out=out)
        assert y is out and torch.equal(y, lutq.moe_mlp(wide[:, 8:8 + D].contiguous(), *W, r))
        assert torch.isfinite(y).all()
    r = lutq.moe_route(torch.zeros((0, E), device="cuda"), 2)
    assert lutq.moe_mlp(torch.zeros((0, D), dtype=torch.float16, device="cuda"), *W, r).shape == (0, D)


@pytest.mark.parametrize("T", [1, 30, 300])
def test_graph_replays(lutq, T):
    """Routing and the block in one graph: replays on new inputs give the eager bits."""
    rng = np.random.default_rng(T)
    E, D, F, k = 8, 128, 96, 2
    gu, dn = experts(rng, E, D, F)
    W = lutq.mx_pack(dev(gu[0]), dev(gu[1])), lutq.mx_pack(dev(dn[0]), dev(dn[1]))
    x = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")
    l = torch.empty((T, E), device="cuda")

    def step():
        return lutq.moe_mlp(x, *W, lutq.moe_route(l, k))
    x.normal_(), l.normal_()
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = step()
    for _ in range(4):
        x.normal_(), l.normal_()
        y.fill_(5)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, step())
