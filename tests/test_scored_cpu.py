"""Routing by scores without a GPU: the oracle against hand-worked choices, the
plain router and a brute force; the refusals of the C ABI and of the Python
call (nothing is launched)."""
import itertools

import numpy as np
import pytest

import oracle
from oracle import scored_oracle as O
from packed_bit_grouped_amd import _lib as L

FAKE = 1 << 20


def logit(p):
    return np.log(p / (1 - np.asarray(p)))


def test_hand_worked_groups():
    # three groups of two; best two: 0.9, 1.1, 1.0; the first leaves though it holds the best expert
    l = logit([[0.8, 0.1, 0.6, 0.5, 0.7, 0.3]])
    ids, w = O.route_scored(l, 3, n_group=3, topk_group=2)
    assert ids.tolist() == [[4, 2, 3]]
    assert w[0] == pytest.approx(np.array([0.7, 0.6, 0.5]) / 1.8, rel=1e-14)
    # by their best one: 0.8, 0.6, 0.7
    ids, w = O.route_scored(l, 3, n_group=3, topk_group=2, group_best=1, renormalize=False, scale=2.0)
    assert ids.tolist() == [[0, 4, 5]]
    assert w[0] == pytest.approx([1.6, 1.4, 0.6], rel=1e-14)


def test_bias_chooses_but_does_not_weigh():
    l = logit([[0.8, 0.6, 0.4, 0.2]])
    ids, w = O.route_scored(l, 2, bias=[-1.0, 0.0, 0.0, 0.5], renormalize=False)
    assert ids.tolist() == [[3, 1]] and w[0] == pytest.approx([0.2, 0.6], rel=1e-14)


def test_ties_and_empty_rows():
    ids, w = O.route_scored([[1.0, 1.0, 1.0, 1.0], [-np.inf] * 4], 2, n_group=2, topk_group=1)
    assert ids.tolist() == [[0, 1], [0, 1]]
    assert w.tolist() == [[0.5, 0.5], [0.0, 0.0]]
    ids, w = O.route_scored([[-np.inf] * 3], 2, score="softmax")
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]


@pytest.mark.parametrize("renormalize", [0, 1])
def test_plain_softmax_router_is_a_special_case(renormalize):
    logits = np.random.default_rng(0).standard_normal((20, 12)).astype(np.float32)
    ids, w = O.route_scored(logits, 4, score="softmax", renormalize=bool(renormalize))
    want_ids, want_w = oracle.route_topk(logits, 4, renormalize)
    assert np.array_equal(ids, want_ids) and w == pytest.approx(want_w, rel=1e-12)


def test_brute_force_over_subsets():
    rng = np.random.default_rng(1)
    for _ in range(30):
        l = rng.standard_normal(8)
        bias = rng.standard_normal(8) * 0.3
        ids, _ = O.route_scored(l[None], 3, bias=bias, n_group=4, topk_group=2)
        c = 1 / (1 + np.exp(-l)) + bias
        pairs = max(itertools.combinations(range(4), 2),
                    key=lambda q: sum(c[2 * g] + c[2 * g + 1] for g in q))
        among = [e for g in pairs for e in (2 * g, 2 * g + 1)]
        best = max(itertools.combinations(among, 3), key=lambda q: c[list(q)].sum())
        assert sorted(ids[0].tolist()) == sorted(best)


# ---------------------------------------------------------------------------
# refusals


def _route(**kw):
    a = dict(logits=FAKE, T=4, E=64, k=8, score=1, bias=FAKE, n_group=8, topk_group=4,
             group_best=2, renormalize=1, scale=2.5, topk_ids=FAKE, topk_w=FAKE)
    a.update(kw)
    return L.moe_route_scored(*a.values(), stream=0, check=False)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(E=0), dict(k=0), dict(k=33), dict(score=2),
                                dict(score=-1), dict(n_group=0), dict(n_group=7), dict(topk_group=0),
                                dict(topk_group=9), dict(group_best=0), dict(group_best=3),
                                dict(renormalize=2), dict(scale=float("nan")),
                                dict(scale=float("inf")), dict(logits=None), dict(topk_ids=None),
                                dict(topk_w=None), dict(n_group=64, topk_group=1, k=2)])
def test_invalid_arguments(kw):
    assert _route(**kw) == L.MOE_E_INVAL


@pytest.mark.parametrize("kw", [dict(E=1032), dict(E=1000, n_group=100, topk_group=100),
                                dict(T=1 << 26)])
def test_unsupported_sizes(kw):
    assert _route(**kw) == L.MOE_E_UNSUPPORTED


def test_accepted_arguments_reach_the_device_check():
    for kw in (dict(), dict(bias=None), dict(T=(1 << 26) - 1), dict(E=1024, k=512),
               dict(n_group=64, topk_group=64, k=64)):
        assert _route(**kw) == L.MOE_E_DEVICE, kw
    assert _route(T=0, logits=None, topk_ids=None, topk_w=None) == L.MOE_OK


def test_python_call_refuses():
    torch = pytest.importorskip("torch")
    from packed_bit_grouped_amd import router
    l = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="score"):
        router.route_scored(l, 2, score="tanh")
    with pytest.raises(TypeError, match="logits"):
        router.route_scored(l.double(), 2)
    with pytest.raises(ValueError, match="contiguous"):
        router.route_scored(torch.zeros(8, 4).t(), 2)
    with pytest.raises(ValueError, match="GPU"):
        router.route_scored(l, 2)
    with pytest.raises(ValueError, match="logits"):
        router.route_scored(torch.zeros(8), 2)
