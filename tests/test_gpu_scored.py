"""Routing by scores on the GPU against the fp64 oracle: ids equal, weights
within two roundings of fp32 (the weight's own, 2^-24, and what 64-bit sums
and exponentials leave, far below the second)."""
import numpy as np
import pytest

from oracle import scored_oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TOL = 2 * 2.0 ** -24


@pytest.fixture(scope="module")
def router():
    from packed_bit_grouped_amd import router as m
    return m


def check(router, logits, k, **kw):
    dev = {**kw, "bias": None if kw.get("bias") is None else torch.from_numpy(kw["bias"]).to(DEV)}
    ids, w = router.route_scored(torch.from_numpy(logits).to(DEV), k, **dev)
    want_ids, want_w = O.route_scored(logits, k, **kw)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = w.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want_w))
    fin = ~np.isnan(want_w)
    assert (np.abs(got - want_w)[fin] <= TOL * np.abs(want_w)[fin] + 2.0 ** -149).all()


CASES = [  # T, E, k, score, bias, n_group, topk_group, group_best, renormalize, scale
    (1, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
    (1, 1, 1, "softmax", False, 1, 1, 2, True, 1.0),
    (3, 2, 2, "sigmoid", True, 2, 2, 1, False, 1.0),
    (5, 7, 3, "softmax", True, 1, 1, 1, False, 16.0),
    (33, 159, 6, "softmax", True, 3, 2, 1, True, 16.0),
    (64, 128, 8, "softmax", False, 1, 1, 1, False, 1.0),
    (65, 160, 6, "softmax", False, 8, 3, 1, True, 1.0),
    (7, 64, 4, "sigmoid", True, 64, 5, 2, True, 1.0),        # groups of one expert
    (7, 62, 30, "sigmoid", False, 31, 16, 2, True, 1.0),     # two lanes a group
    (9, 1023, 17, "sigmoid", True, 33, 20, 2, True, 1.0),    # one lane a group, 31 experts each
    (9, 1020, 13, "softmax", True, 17, 3, 2, False, 0.5),    # 60 experts on two lanes
    (6, 1024, 1024, "softmax", True, 1, 1, 2, True, 1.0),    # every expert, in order
    (6, 512, 100, "sigmoid", True, 4, 2, 2, True, 1.0),      # more choices than lanes
    (6, 512, 65, "sigmoid", True, 1, 1, 2, False, 1.0),
    (4, 300, 64, "sigmoid", True, 2, 1, 2, True, 1.0),
    (2, 1000, 10, "softmax", False, 2, 1, 2, True, 1.0),     # 32 lanes a group
    (513, 18, 7, "sigmoid", False, 2, 1, 2, False, 1.0),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("coarse", [False, True])
def test_matches_oracle(router, case, coarse):
    T, E, k, score, bias, n_group, topk_group, best, renorm, scale = case
    rng = np.random.default_rng(T * E + k)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    if coarse:      # many ties
        logits = np.round(logits * 2) / 2
    b = (rng.standard_normal(E) * 0.1).astype(np.float32) if bias else None
    if coarse and bias:
        b = (np.round(b * 20) / 16).astype(np.float32)
    check(router, logits, k, score=score, bias=b, n_group=n_group, topk_group=topk_group,
          group_best=best, renormalize=renorm, scale=scale)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_scores_that_32_bits_cannot_tell_apart(router, score):
    rng = np.random.default_rng(3)
    logits = (20 + rng.standard_normal((40, 64)) * 0.5).astype(np.float32)   # sigmoids of 1 - 2e-9
    check(router, logits, 8, score=score, n_group=8, topk_group=3)
    tiny = (-60 + rng.standard_normal((40, 64))).astype(np.float32)          # scores of 1e-26
    check(router, tiny, 8, score=score, n_group=8, topk_group=3)
    bias = (1 + rng.standard_normal(64) * 1e-3).astype(np.float32)
    check(router, logits, 8, score=score, bias=bias, n_group=8, topk_group=3)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups", [(1, 1), (4, 2)])
def test_masked_infinite_and_nan_logits(router, score, groups):
    rng = np.random.default_rng(4)
    l = rng.standard_normal((10, 32)).astype(np.float32)
    l[0] = -np.inf                       # nothing left
    l[1, 1:] = -np.inf                   # one left
    l[2, ::2] = -np.inf
    l[3] = np.finfo(np.float32).min      # masks of the type's lowest value
    l[4, 5:] = np.finfo(np.float32).min
    l[5, 7] = np.nan
    l[6] = np.nan
    l[7, 3] = np.inf
    l[8] = 0.0
    l[8, 9] = -0.0
    l[9] = 200.0                         # scores of 1 and of 1/32
    check(router, l, 5, score=score, n_group=groups[0], topk_group=groups[1])
    bias = np.zeros(32, dtype=np.float32)
    bias[::3] = -np.inf
    check(router, l, 5, score=score, bias=bias, n_group=groups[0], topk_group=groups[1],
          renormalize=False)


def test_equals_the_plain_router_where_they_meet(router):
    from packed_bit_grouped_amd import _lib as L
    torch.manual_seed(0)
    logits = torch.randn(300, 128, device=DEV)
    ids, w = router.route_scored(logits, 8, score="softmax")
    ids2, w2 = torch.empty_like(ids), torch.empty_like(w)
    L.moe_route_topk(logits, 300, 128, 8, 1, ids2, w2)
    assert torch.equal(ids, ids2)
    assert torch.allclose(w, w2, rtol=1e-5)


def test_rows_past_32_bit_offsets(router):
    T, E = (1 << 21) + 5, 1024                 # 2^31 logits and more
    logits = torch.zeros((T, E), device=DEV)
    rng = np.random.default_rng(6)
    rows = [0, 1, (1 << 20) - 1, 1 << 20, (1 << 21) - 1, 1 << 21, T - 1]
    part = rng.standard_normal((len(rows), E)).astype(np.float32)
    logits[rows] = torch.from_numpy(part).to(DEV)
    ids, w = router.route_scored(logits, 4, n_group=4, topk_group=2)
    want_ids, want_w = O.route_scored(part, 4, n_group=4, topk_group=2)
    assert np.array_equal(ids[rows].cpu().numpy(), want_ids)
    assert np.abs(w[rows].cpu().numpy() - want_w).max() <= TOL
    del logits
    torch.cuda.empty_cache()


def test_given_outputs_streams_and_graphs(router):
    torch.manual_seed(1)
    logits = torch.randn(50, 96, device=DEV)
    bias = torch.randn(96, device=DEV) * 0.1
    kw = dict(bias=bias, n_group=6, topk_group=2)
    ids = torch.full((52, 7), -7, dtype=torch.int32, device=DEV)
    w = torch.full((52, 7), -7.0, device=DEV)
    a, b = router.route_scored(logits, 7, ids=ids[1:51], w=w[1:51], **kw)
    want_ids, want_w = router.route_scored(logits, 7, **kw)
    assert torch.equal(ids[1:51], want_ids) and torch.equal(w[1:51], want_w)
    for t in (ids, w):
        assert (t[0] == -7).all() and (t[51] == -7).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ids2, w2 = router.route_scored(logits, 7, stream=side, **kw)
    side.synchronize()
    assert torch.equal(ids2, want_ids) and torch.equal(w2, want_w)
    graph = torch.cuda.CUDAGraph()
    out_i, out_w = torch.empty_like(want_ids), torch.empty_like(want_w)
    src = logits.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        router.route_scored(src, 7, ids=out_i, w=out_w, **kw)
    for i in range(3):
        src.copy_(torch.randn(50, 96, device=DEV))
        graph.replay()
        e_i, e_w = router.route_scored(src, 7, **kw)
        torch.cuda.synchronize()
        assert torch.equal(out_i, e_i) and torch.equal(out_w, e_w)


def test_no_tokens_and_refusals(router):
    ids, w = router.route_scored(torch.empty((0, 16), device=DEV), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    l = torch.zeros((4, 16), device=DEV)
    with pytest.raises(ValueError, match="bias"):
        router.route_scored(l, 4, bias=torch.zeros(8, device=DEV))
    with pytest.raises(ValueError, match="device"):
        router.route_scored(l, 4, bias=torch.zeros(16))
    with pytest.raises(TypeError, match="ids"):
        router.route_scored(l, 4, ids=torch.zeros((4, 4), dtype=torch.int64, device=DEV))
    from packed_bit_grouped_amd import _lib as L
    with pytest.raises(L.MoeError):
        router.route_scored(l, 17)


@pytest.mark.parametrize("T", [(1 << 26) - 5, (1 << 26) - 1])
def test_the_most_tokens(router, T):
    """Workgroups of 256 lanes for four tokens each: 2^32 lanes and the most that are less."""
    logits = torch.zeros((T, 1), device=DEV)
    ids = torch.full((T, 1), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, 1), -7.0, device=DEV)
    router.route_scored(logits, 1, renormalize=False, scale=4.0, ids=ids, w=w)
    assert (ids == 0).all() and (w == 2.0).all()
    del logits, ids, w
    torch.cuda.empty_cache()
