"""Low-rank adapters on the GPU against the fp64 oracle (oracle/lora_oracle.py):
every value within the bound of fp32 sums and one rounding to the output's type."""
import numpy as np
import pytest

import oracle
from oracle import lora_oracle as O
from oracle import mx_oracle, scored_oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def lora():
    from packed_bit_grouped_amd import lora as m
    return m


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).bfloat16().to(DEV)


def test_tiled_layouts_match_their_definition(lora):
    from packed_bit_grouped_amd import _lib as L
    rng = np.random.default_rng(0)
    for n, rows, cols, is_b in ((1, 8, 32, 0), (3, 16, 96, 0), (2, 24, 64, 0), (2, 256, 160, 0), (1, 32, 8, 1),
                                (3, 96, 24, 1), (2, 64, 128, 1)):
        m = rng.integers(-30000, 30000, (n, rows, cols)).astype(np.int16)
        held = rows if is_b else (rows + 15) // 16 * 16
        dst = torch.zeros((n, held * cols), dtype=torch.int16, device=DEV)
        L.moe_lora_tile(dev(m), n, rows, cols, is_b, dst)
        want = np.zeros((n, held * cols), dtype=np.int16)
        for i in range(n):
            if is_b:
                want[i] = m[i].reshape(rows // 32, 32, cols // 8, 8).transpose(0, 2, 1, 3).ravel()
            else:
                full = np.zeros((held, cols), dtype=np.int16)
                full[:rows] = m[i]
                want[i] = full.reshape(held // 16, 16, cols // 32, 4, 8).transpose(0, 2, 3, 1, 4).ravel()
        assert np.array_equal(dst.cpu().numpy(), want)


def tables(rng, T, k, E, gone=0.0):
    """Routing tables of random choices; gone: that share of pairs has no expert."""
    ids = np.array([rng.permutation(E)[:k] for _ in range(T)], dtype=np.int32).reshape(T, k)
    ids[rng.random((T, k)) < gone] = -1
    flat = ids.ravel()
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable").astype(np.int32)
    m = int((flat >= 0).sum())
    pos = np.full(T * k, -1, dtype=np.int32)
    pos[order[:m]] = np.arange(m)
    order[m:] = -1
    off = np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=E))]).astype(np.int32)
    return ids, off, order, pos


def make(lora, T, H, I, E, k, n_shared=0, I_shared=0, n=2, ranks=(8,), h_f32=False, out_f32=False,
         runs=False, none=0.2, gone=0.0, seed=0):
    """A layer's rows and adapters of mixed ranks: device tensors, and the oracle's view."""
    rng = np.random.default_rng(seed)
    d = dict(T=T, H=H, I=I, E=E, k=k, n_shared=n_shared, I_shared=I_shared, h_f32=h_f32, out_f32=out_f32)
    d["widths"] = [I] * E + [I_shared] * n_shared
    d["ld"] = max(I, I_shared if n_shared else 0)
    d["ids"], d["off"], d["sp"], d["pos"] = tables(rng, T, k, E, gone)
    d["rows"] = O.rows_of(d["sp"], d["ids"], T, k, E, n_shared)
    R = len(d["rows"])
    adapter = np.sort(rng.integers(0, n, T)) if runs else rng.integers(0, n, T)
    adapter[rng.random(T) < none] = rng.choice([-1, n, -2**31, 2**31 - 1])
    d["adapter"] = adapter.astype(np.int32)
    d["ad"] = lora.Adapters(n, E, H, I, n_shared, I_shared, max_rank=max(ranks), device=DEV)
    d["up"], d["dn"] = [[None] * (E + n_shared) for _ in range(n)], [[None] * (E + n_shared) for _ in range(n)]
    for i in range(n):
        for e, width in enumerate(d["widths"]):
            if rng.random() < 0.1 and E + n_shared > 1:
                continue                                   # this adapter leaves the expert alone
            r, s = int(rng.choice(ranks)), float(2.0 ** rng.integers(-2, 2))
            a13, b13 = bf16(rng, 1, 2 * r, H, scale=H ** -0.5), bf16(rng, 1, 2 * width, r, scale=0.5)
            a2, b2 = bf16(rng, 1, r, width, scale=width ** -0.5), bf16(rng, 1, H, r, scale=0.5)
            d["ad"].load(i, a13, b13, a2, b2, s, first=e)
            d["up"][i][e], d["dn"][i][e] = (f64(a13[0]), f64(b13[0]), s), (f64(a2[0]), f64(b2[0]), s)
    d["B"] = lora.LoraBuffers(T, H, I, E, k, n_shared, I_shared, max(ranks), h_f32, out_f32, device=DEV)
    d["x"] = bf16(rng, T, H)
    d["gu"] = dev(rng.standard_normal((R, 2 * d["ld"])).astype(np.float32))
    h = (rng.standard_normal((R, d["ld"])) * 0.7).astype(np.float32)
    d["h"] = dev(h) if h_f32 else dev(h).bfloat16()
    d["base"] = dev(rng.standard_normal((T, H)).astype(np.float32))
    d["w"] = dev(rng.random((T, k)).astype(np.float32))
    d["gate"] = dev(rng.standard_normal((T, n_shared)).astype(np.float32)) if n_shared else None
    d["t"] = [dev(d[x]) for x in ("ids", "off", "sp", "pos")]
    d["tad"] = dev(d["adapter"])
    return d


def run_gateup(lora, d, **kw):
    ids, off, sp, _ = d["t"]
    return lora.gateup_silu(d["ad"], d["x"], d["tad"], d["gu"], ids, off, sp, d["B"], **kw)


def run_down(lora, d, **kw):
    ids, off, sp, pos = d["t"]
    kw.setdefault("shared_gate", d["gate"])
    return lora.down_combine(d["ad"], d["h"], d["base"], d["tad"], d["w"], ids, off, sp, pos, d["B"], **kw)


def check_gateup(d, h):
    want, bound = O.gateup(f64(d["gu"]), f64(d["x"]), d["rows"], d["adapter"], d["up"], d["widths"],
                           d["ld"], not d["h_f32"])
    got = f64(h)
    there = ~np.isnan(want)
    err = np.abs(got - want)[there]
    worst = (err / bound[there]).max() if err.size else 0.0
    assert worst <= 1.0, worst
    return there


def gates(d):
    return np.ones((d["T"], d["n_shared"])) if d["gate"] is None else 1 / (1 + np.exp(-f64(d["gate"])))


def check_down(d, out):
    want, bound = O.down(f64(d["base"]), f64(d["h"]), d["rows"], d["adapter"], d["dn"], d["widths"],
                         f64(d["w"]), d["pos"], gates(d), d["T"], d["k"], not d["out_f32"])
    worst = (np.abs(f64(out) - want) / bound).max()
    assert worst <= 1.0, worst


CASES = [  # T, H, I, E, k, n_shared, I_shared, adapters, ranks, runs
    (1, 32, 32, 1, 1, 0, 0, 1, (8,), False),
    (1, 64, 96, 4, 2, 1, 96, 2, (16,), False),
    (3, 96, 32, 5, 5, 2, 64, 3, (8, 24), False),
    (5, 1056, 352, 12, 3, 0, 0, 5, (24,), False),
    (12, 2048, 512, 8, 4, 1, 512, 4, (16,), False),
    (17, 128, 160, 3, 1, 1, 32, 64, (8, 16, 40, 128), False),
    (64, 224, 64, 16, 4, 1, 128, 9, (8, 64), False),
    (77, 1056, 352, 12, 3, 0, 0, 5, (24,), False),
    (130, 64, 32, 2, 2, 0, 0, 1, (8,), True),
    (33, 64, 64, 40, 20, 1, 64, 3, (128,), False),     # 336 pieces of rank 8 a token: several passes
    # more than 2048 rows
    (700, 64, 64, 7, 3, 0, 0, 3, (8, 16), True),
    (700, 96, 32, 3, 3, 1, 64, 40, (16, 40), False),
    (1031, 160, 96, 5, 2, 1, 96, 2, (8, 72, 128), True),
    (2100, 32, 32, 4, 1, 1, 32, 1, (16,), True),
    # the sums of a block of tokens in LDS: ranks up to 32, 64 and 128, blocks of 64 tokens and more
    (1100, 2080, 384, 6, 3, 1, 416, 3, (8, 24, 32), False),
    (900, 1056, 352, 12, 4, 0, 0, 2, (8, 64), True),
    (1500, 992, 96, 5, 2, 1, 32, 40, (16, 72, 128), False),
    (4200, 8224, 32, 3, 1, 0, 0, 1, (16,), False),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("wide", [False, True])
def test_gateup_matches_oracle(lora, case, wide):
    T, H, I, E, k, s, Is, n, ranks, runs = case
    d = make(lora, T, H, I, E, k, s, Is, n, ranks, h_f32=wide, runs=runs, seed=T + H)
    d["B"].h.fill_(7.0)
    h = run_gateup(lora, d)
    there = check_gateup(d, h)
    assert (f64(h)[~there] == 7.0).all()              # columns past a row's own width
    assert d["B"].error_word() == 0


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("out_f32", [False, True])
def test_down_matches_oracle(lora, case, wide, out_f32):
    T, H, I, E, k, s, Is, n, ranks, runs = case
    d = make(lora, T, H, I, E, k, s, Is, n, ranks, h_f32=wide, out_f32=out_f32, runs=runs, seed=T + H)
    for r, (t, e) in enumerate(d["rows"]):            # what no row owns is not read
        d["h"][r, d["widths"][e]:] = float("nan")
    out = run_down(lora, d)
    d["h"] = torch.nan_to_num(d["h"])
    check_down(d, out)
    assert d["B"].error_word() == 0


# tokens and ranks: one launch; three of gate/up; three of both
@pytest.mark.parametrize("T,ranks", [(5, (8, 16)), (70, (8, 16)), (900, (8, 16)), (2000, (8, 128))])
def test_unrouted_pairs(lora, T, ranks):
    """Pairs that no expert took: their rows of h stay as they were, and what
    lies in them reaches no output."""
    d = make(lora, T, 96, 64, 6, 3, 1, 32, 3, ranks, gone=0.3, none=0.1, seed=T)
    d["B"].h.fill_(3.0)
    h = run_gateup(lora, d)
    there = check_gateup(d, h)
    assert (f64(h)[~there] == 3.0).all()
    m = int(d["off"][-1])
    d["h"][m:T * 3] = float("nan")
    out = run_down(lora, d)
    d["h"][m:T * 3] = 0
    check_down(d, out)


@pytest.mark.parametrize("T,ranks", [(9, (8,)), (1200, (8,)), (4500, (128,))])
def test_unrouted_tokens_without_shared_experts_give_base(lora, T, ranks):
    d = make(lora, T, 64, 32, 4, 2, n=2, ranks=ranks, gone=1.0, out_f32=True, seed=1)
    assert torch.equal(run_down(lora, d), d["base"])
    d["B"].h.fill_(5.0)
    assert (run_gateup(lora, d) == 5.0).all()


@pytest.mark.parametrize("T,rank", [(6, 8), (1000, 8), (3500, 128)])
@pytest.mark.parametrize("n", [0, 3])
def test_no_adapter_at_all(lora, T, rank, n):
    d = make(lora, T, 64, 32, 4, 2, 1, 64, n=max(n, 1), ranks=(rank,), none=1.0, out_f32=True, seed=2)
    if n == 0:
        d["ad"] = lora.Adapters(0, 4, 64, 32, 1, 64, max_rank=rank, device=DEV)
        d["tad"] = torch.zeros(T, dtype=torch.int32, device=DEV)
    check_gateup(d, run_gateup(lora, d))
    assert torch.equal(run_down(lora, d), d["base"])


@pytest.mark.parametrize("T,ranks", [(8, (8, 16)), (900, (8, 16)), (3000, (8, 128))])
def test_unusable_entries_count_as_none_and_are_reported(lora, T, ranks):
    d = make(lora, T, 64, 32, 3, 3, 0, 0, 1, ranks, none=0.0, seed=3)
    a13, b13 = bf16(np.random.default_rng(0), 1, 16, 64), bf16(np.random.default_rng(0), 1, 64, 8)
    a2, b2 = bf16(np.random.default_rng(0), 1, 8, 32), bf16(np.random.default_rng(0), 1, 64, 8)
    d["ad"].load(0, a13, b13, a2, b2, first=1)
    d["up"][0][1] = d["dn"][0][1] = None
    for change in (dict(N=32), dict(K=96), dict(rank=ranks[1] + 8), dict(rank=12), dict(rank=-8), dict(a=0), dict(b=0),
                   dict(a=a13.data_ptr() + 2)):
        for tag in ("13", "2"):
            d["ad"].load(0, a13, b13, a2, b2, first=1)
            for f, v in change.items():
                setattr(d["ad"]._host[tag][1], f, v)
            d["ad"]._put(tag, 0, 1, 1, None)
            d["B"].ws[:4].zero_()
            if tag == "13":
                check_gateup(d, run_gateup(lora, d))
            else:
                check_down(d, run_down(lora, d))
            assert d["B"].error_word() == 1, change
    d["ad"].unload(0)
    d["up"], d["dn"] = [[None] * 3], [[None] * 3]
    d["B"].ws[:4].zero_()
    check_gateup(d, run_gateup(lora, d))
    check_down(d, run_down(lora, d))
    assert d["B"].error_word() == 0


@pytest.mark.parametrize("e", range(4))
def test_an_unusable_entry_is_reported_whichever_choice_meets_it(lora, e):
    d = make(lora, 1, 64, 32, 3, 3, 1, 32, 1, (8,), none=0.0, seed=14)
    for tag, run in (("13", run_gateup), ("2", run_down)):
        rng = np.random.default_rng(1)
        d["ad"].load(0, bf16(rng, 1, 16, 64), bf16(rng, 1, 64, 8), bf16(rng, 1, 8, 32), bf16(rng, 1, 64, 8), first=e)
        d["B"].ws[:4].zero_()
        run(lora, d)
        assert d["B"].error_word() == 0
        d["ad"]._host[tag][e].rank = 24
        d["ad"]._put(tag, 0, e, 1, None)
        run(lora, d)
        assert d["B"].error_word() == 1


@pytest.mark.parametrize("T,ranks", [(20, (8, 16)), (900, (8, 16)), (2000, (8, 128))])
def test_nan_and_inf_stay_in_their_rows(lora, T, ranks):
    d = make(lora, T, 96, 64, 4, 2, 1, 64, 3, ranks, none=0.0, out_f32=True, seed=4)
    keep_h, keep_o = f64(run_gateup(lora, d)), f64(run_down(lora, d))
    d["x"][2, 9] = float("nan")
    d["x"][5, 1] = float("inf")
    h = f64(run_gateup(lora, d))
    bad = np.array([t in (2, 5) and d["up"][d["adapter"][t]][e] is not None for t, e in d["rows"]])
    assert np.array_equal(h[~bad], keep_h[~bad]) and not np.isfinite(h[bad]).any()
    # a NaN in one adapter's matrices of one expert
    d["x"][2, 9] = d["x"][5, 1] = 0
    i, e = next((i, e) for i in range(3) for e in range(4) if d["up"][i][e] is not None)
    for at, b in (("13", 1), ("2", 1)):
        d["ad"]._held[at, i, e][b].fill_(float("nan"))
    h, o = f64(run_gateup(lora, d)), f64(run_down(lora, d))
    hit = np.array([d["adapter"][t] == i and q == e for t, q in d["rows"]])
    clean = np.array([t not in (2, 5) for t, _ in d["rows"]])
    assert np.isnan(h[hit]).all() and np.array_equal(h[~hit & clean], keep_h[~hit & clean])
    tok = np.zeros(T, dtype=bool)
    tok[[t for (t, _), x in zip(d["rows"], hit) if x]] = True
    assert np.isnan(o[tok]).all() and np.array_equal(o[~tok], keep_o[~tok])


def test_large_and_tiny_values_keep_their_bits(lora):
    """The three bf16 parts of an fp32 operand lose nothing of it."""
    d = make(lora, 24, 64, 32, 2, 1, 0, 0, 1, (8,), h_f32=True, out_f32=True, none=0.0, seed=5)
    rng = np.random.default_rng(5)
    d["h"] = (d["h"].double() * torch.from_numpy(2.0 ** rng.integers(-60, 60, (24, 1))).to(DEV)).float()
    d["base"].zero_()
    check_down(d, run_down(lora, d))
    d["gu"] *= 30.0
    check_gateup(d, run_gateup(lora, d))
    d["gu"][:, :32] = -100.0
    d["gu"][:, 32:] = 1e30
    d["tad"].fill_(-1)
    got = f64(run_gateup(lora, d))
    assert got == pytest.approx(np.full(got.shape, -100 * np.exp(-100.0) * 1e30), rel=1e-5)


def test_down_in_place(lora):
    from packed_bit_grouped_amd import _lib as L
    d = make(lora, 40, 96, 64, 4, 2, 1, 64, 3, (8, 16), out_f32=True, seed=6)
    want = run_down(lora, d).clone()
    B, (ids, off, sp, pos) = d["B"], d["t"]
    L.moe_lora_down_combine(d["h"], 40, 96, 64, 4, 2, 1, 64, d["tad"], 3, 16, d["ad"].table["2"], d["w"], ids, off,
                            sp, pos, d["base"], d["base"], B.ws, B.ws_bytes, L.MOE_OUT_F32, shared_gate=d["gate"])
    assert torch.equal(d["base"], want)


@pytest.mark.parametrize("T,ranks", [(30, (8, 16)), (800, (8, 16)), (2000, (8, 128))])
def test_same_results_every_time_on_streams_and_in_graphs(lora, T, ranks):
    d = make(lora, T, 128, 64, 6, 3, 1, 64, 4, ranks, seed=7)
    h, o = run_gateup(lora, d).clone(), run_down(lora, d).clone()
    e = make(lora, T, 128, 64, 6, 3, 1, 64, 4, ranks, seed=7)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):                                # two at once, with buffers each
        h1, h2 = run_gateup(lora, d, stream=a), run_gateup(lora, e, stream=b)
        o1, o2 = run_down(lora, d, stream=a), run_down(lora, e, stream=b)
        torch.cuda.synchronize()
        for x in (h1, h2):
            assert torch.equal(x, h)
        for x in (o1, o2):
            assert torch.equal(x, o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_gateup(lora, d)
        run_down(lora, d)
    for i in range(3):
        d["x"].copy_(torch.randn(T, 128, device=DEV))
        d["tad"].copy_(torch.randint(-1, 4, (T,), device=DEV))
        d["h"].copy_(torch.randn_like(d["h"]))
        graph.replay()
        torch.cuda.synchronize()
        h1, o1 = d["B"].h.clone(), d["B"].out.clone()
        assert torch.equal(h1, run_gateup(lora, d)) and torch.equal(o1, run_down(lora, d))


def test_adapters_are_loaded_and_emptied_between_steps(lora):
    d = make(lora, 25, 64, 32, 4, 2, 0, 0, 2, (8,), none=0.0, seed=8)
    check_gateup(d, run_gateup(lora, d))
    rng = np.random.default_rng(9)
    a13, b13 = bf16(rng, 4, 16, 64, scale=0.1), bf16(rng, 4, 64, 8)
    a2, b2 = bf16(rng, 4, 8, 32, scale=0.1), bf16(rng, 4, 64, 8)
    d["ad"].load(1, a13, b13, a2, b2, scale=3.0, stream=torch.cuda.current_stream())
    for e in range(4):
        d["up"][1][e], d["dn"][1][e] = (f64(a13[e]), f64(b13[e]), 3.0), (f64(a2[e]), f64(b2[e]), 3.0)
    check_gateup(d, run_gateup(lora, d))
    check_down(d, run_down(lora, d))
    d["ad"].unload(0)
    d["up"][0], d["dn"][0] = [None] * 4, [None] * 4
    check_gateup(d, run_gateup(lora, d))
    check_down(d, run_down(lora, d))


def test_python_refusals_on_the_device(lora):
    d = make(lora, 4, 64, 32, 4, 2, 0, 0, 2, (8,), seed=10)
    ids, off, sp, pos = d["t"]
    with pytest.raises(ValueError, match="adapter"):
        lora.gateup_silu(d["ad"], d["x"], d["tad"][:3], d["gu"], ids, off, sp, d["B"])
    with pytest.raises(ValueError, match="gu"):
        lora.gateup_silu(d["ad"], d["x"], d["tad"], d["gu"][:, :32], ids, off, sp, d["B"])
    with pytest.raises(TypeError, match="h:"):
        lora.down_combine(d["ad"], d["h"].float(), d["base"], d["tad"], d["w"], ids, off, sp, pos, d["B"])
    with pytest.raises(ValueError, match="device"):
        lora.gateup_silu(d["ad"], d["x"], d["tad"].cpu(), d["gu"], ids, off, sp, d["B"])
    other = lora.Adapters(2, 4, 64, 64, max_rank=8, device=DEV)
    with pytest.raises(ValueError, match="I = 64"):
        lora.gateup_silu(other, d["x"], d["tad"], d["gu"], ids, off, sp, d["B"])
    other = lora.Adapters(2, 4, 64, 32, max_rank=16, device=DEV)
    with pytest.raises(ValueError, match="ranks"):
        lora.gateup_silu(other, d["x"], d["tad"], d["gu"], ids, off, sp, d["B"])


# ---------------------------------------------------------------------------
# the shared projections' sums, and whole layers


def silu_rows(gu, widths, rows, ld):
    """SiLU(g) * u in 64 bits of fp32 sums, NaN where nothing is."""
    h = np.full((len(rows), ld), np.nan)
    for r, (_, e) in enumerate(rows):
        g, u = gu[r, :widths[e]], gu[r, ld:ld + widths[e]]
        h[r, :widths[e]] = g / (1 + np.exp(-g)) * u
    return h


def w4_layer(T, H, I, E, k, n_shared, I_shared, act, seed, n_int2=1):
    from packed_bit_grouped_amd import layer as W
    from synth import LayerConfig, make_layer
    cfg = LayerConfig("lora_w4", seed, T=T, H=H, E=E, k=k, I=I, group=32, n_int2=n_int2, group_int2=64,
                      n_shared=n_shared, I_shared=I_shared, act=act)
    return W.DeviceLayer.from_synth(make_layer(cfg), DEV)


@pytest.mark.parametrize("act,path,T,tile_m,prepacked", [
    ("a16", 0, 1, 16, False), ("a16", 1, 9, 16, False), ("a16", 3, 40, 16, False), ("a16", 2, 300, 160, False),
    ("a16", 2, 300, 160, True), ("a8", 0, 5, 16, False), ("a8", 1, 30, 16, False), ("a8", 3, 50, 16, False)])
def test_w4_sums_are_what_silu_joins(act, path, T, tile_m, prepacked):
    from packed_bit_grouped_amd import _lib as L
    H, I, E, k, Is = 256, 128, 4, 2, 256
    dl = w4_layer(T, H, I, E, k, 1, Is, act, 200 + T)
    B = dl.buffers(act, tile_m)
    bank = dl.bank.prepack() if prepacked else dl.bank
    flags = path | (L.MOE_W_PREPACKED if prepacked else 0)
    L.moe_route_topk(dl.logits, T, E, k, 1, B.ids, B.w)
    L.moe_permute(B.ids, T, k, E, tile_m, B.counts, B.offsets, B.sorted_pair, B.pair_pos, B.tiles, B.n_tiles)
    gu = torch.full((B.R, 2 * B.ld_h), 7.0, device=DEV)
    args = (B.act, dl.x, T, H, I, E, k, bank.w13, bank.w13_sh, 1, Is, B.offsets, B.sorted_pair, B.tiles, B.n_tiles,
            tile_m)
    L.moe_w4_gateup_silu(*args, gu, B.ws, B.ws_bytes, flags | L.MOE_GU_F32)
    L.moe_w4_gateup_silu(*args, B.h, B.ws, B.ws_bytes, flags)
    h = f64(B.h.view(torch.bfloat16) if act == "a16" else B.h)
    rows = O.rows_of(B.sorted_pair.cpu().numpy(), B.ids.cpu().numpy(), T, k, E, 1)
    widths = [I] * E + [Is]
    want = silu_rows(f64(gu), widths, rows, B.ld_h)
    there = ~np.isnan(want)
    # the same sums, where both calls run the same kernel: SiLU * u in fp32 and one
    # rounding; a single token's h comes from another kernel (sums of K = H products)
    loose = 2.0 ** -14 if path == 0 and act == "a16" else 2.0 ** -18
    rel = 2.0 ** -8 if act == "a16" else 0.0
    err = np.abs(h - want)[there]
    near0 = 1.0 if path == 0 and act == "a16" else 1e-2
    assert (err <= (rel + loose) * np.abs(want[there]) + loose * np.abs(want[there]).max() * near0).all()
    for half in (slice(0, I), slice(B.ld_h, B.ld_h + I)):
        assert not (gu[:T * k, half] == 7.0).any()
    assert (gu[:T * k, I:Is] == 7.0).all() and (gu[:T * k, Is + I:] == 7.0).all()
    assert B.error_word() == 0


def mx_layer(T, H, I, E, k, n_shared, I_shared, act, seed):
    from packed_bit_grouped_amd import mx
    rng = np.random.default_rng(seed)
    pair = lambda n, N, K: tuple(map(dev, mx_oracle.quantise((rng.standard_normal((n, N, K)) * 0.08).astype(np.float32))))
    bank = mx.MxBank(pair(E, 2 * I, H), pair(E, H, I), *((pair(n_shared, 2 * I_shared, H), pair(n_shared, H, I_shared))
                                                         if n_shared else (None, None)))
    return bank, mx.MxBuffers(T, H, I, E, k, n_shared, I_shared, act=act, device=DEV)


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("T,H,I", [(1, 96, 64), (50, 160, 96), (700, 512, 256), (1500, 512, 256)])
def test_mx_sums_are_what_silu_joins(act, T, H, I):
    from packed_bit_grouped_amd import mx
    E, k = 4, 2
    bank, B = mx_layer(T, H, I, E, k, 1, I + 32, act, T)
    rng = np.random.default_rng(T)
    ids, off, sp, _ = tables(rng, T, k, E)
    x, toff, tsp = bf16(rng, T, H), dev(off), dev(sp)
    gu = torch.full((B.R, 2 * B.ld_h), 7.0, device=DEV)
    assert mx.gateup_silu(bank, x, toff, tsp, B, gu=gu) is gu
    h = f64(mx.gateup_silu(bank, x, toff, tsp, B))
    rows = O.rows_of(sp, ids, T, k, E, 1)
    want = silu_rows(f64(gu), [I] * E + [I + 32], rows, B.ld_h)
    there = ~np.isnan(want)
    err = np.abs(h - want)[there]
    assert (err <= (2.0 ** -8 + 2.0 ** -18) * np.abs(want[there]) + 1e-30).all()
    assert (gu[:T * k, I:B.ld_h] == 7.0).all() and (gu[:T * k, B.ld_h + I:] == 7.0).all()


def run_and_check_layer(lora, bank, M, dims, act, routing, seed, x, logits, gate, flags=0):
    T, H, I, E, k, n_shared, I_shared = dims
    d = make(lora, T, H, I, E, k, n_shared, I_shared, 3, (8, 16), h_f32=act == "a8", out_f32=True, seed=seed)
    d["x"], B = x, d["B"]
    B.gu.fill_(float("nan"))
    out = lora.run_layer(bank, M, d["ad"], B, x, d["tad"], logits, routing=routing, shared_gate=gate, flags=flags)
    lg = logits.cpu().numpy()
    ids, w = oracle.route_topk(lg, k, 1) if routing is None else scored_oracle.route_scored(
        lg, k, **{**routing, "bias": routing["bias"].cpu().numpy()})
    assert np.array_equal(M.ids.cpu().numpy()[:T], ids)
    assert np.abs(f64(M.w)[:T] - w).max() <= 1e-6
    # each part from the parts before it, as the device left them
    d["ids"] = ids
    d["sp"], d["pos"] = M.sorted_pair.cpu().numpy()[:T * k], M.pair_pos.cpu().numpy()[:T * k]
    order = np.argsort(ids.ravel(), kind="stable")
    assert np.array_equal(d["sp"], order) and np.array_equal(d["pos"], np.argsort(order))
    d["rows"] = O.rows_of(d["sp"], ids, T, k, E, n_shared)
    d["gu"] = torch.nan_to_num(B.gu)
    check_gateup(d, B.h)
    d["h"], d["base"], d["w"], d["gate"] = B.h, B.base, M.w[:T], gate
    check_down(d, out)
    assert B.error_word() == 0
    # without adapters it is the layer itself
    plain = lora.run_layer(bank, M, d["ad"], B, x, torch.full_like(d["tad"], -1), logits, routing=routing,
                           shared_gate=gate, flags=flags).clone()
    assert torch.equal(plain, B.base)
    return plain


ROUTING = dict(score="sigmoid", n_group=4, topk_group=2, scale=2.5)


@pytest.mark.parametrize("routed", [False, True])
@pytest.mark.parametrize("T", [1, 12, 70, 1100])
@pytest.mark.parametrize("act", ["a16", "a8"])
def test_w4_layer_with_adapters(lora, act, T, routed):
    H, I, E, k, Is = 256, 128, 8, 2, 128
    dl = w4_layer(T, H, I, E, k, 1, Is, act, 300 + T)
    gate = torch.randn(T, 1, device=DEV)
    routing = dict(ROUTING, bias=torch.randn(E, device=DEV) * 0.1) if routed else None
    M = dl.buffers(act)
    plain = run_and_check_layer(lora, dl.bank, M, (T, H, I, E, k, 1, Is), act, routing, T,
                                dl.x.view(torch.bfloat16), dl.logits, gate)
    if not routed:                                   # next to the layer's own call
        from packed_bit_grouped_amd import layer as W
        N = dl.buffers(act, out_f32=True)
        W.run_layer(dl.bank, dl.x, dl.logits, N, shared_gate=gate)
        err = (plain - N.out[:T]).abs().max() / N.out[:T].abs().max()
        # h in bf16 from other kernels' sums: a step of bf16 here and there; 8-bit codes move with theirs
        assert err <= (2.0 ** -8 if act == "a16" else 2.0 ** -6)


@pytest.mark.parametrize("routed", [False, True])
@pytest.mark.parametrize("T", [1, 40, 900])
@pytest.mark.parametrize("act", ["a16", "a4"])
def test_mx_layer_with_adapters(lora, act, T, routed):
    H, I, E, k, Is = 288, 96, 8, 2, 160
    bank, M = mx_layer(T, H, I, E, k, 1, Is, act, T)
    rng = np.random.default_rng(T + 1)
    routing = dict(ROUTING, bias=torch.randn(E, device=DEV) * 0.1) if routed else None
    run_and_check_layer(lora, bank, M, (T, H, I, E, k, 1, Is), act, routing, T, bf16(rng, T, H),
                        dev(rng.standard_normal((T, E)).astype(np.float32)),
                        dev(rng.standard_normal((T, 1)).astype(np.float32)))


def test_layer_in_a_graph(lora):
    T, H, I, E, k = 20, 256, 128, 8, 2
    bank, M = mx_layer(T, H, I, E, k, 1, 128, "a16", 5)
    d = make(lora, T, H, I, E, k, 1, 128, 3, (8, 16), seed=11)
    logits = torch.randn(T, E, device=DEV)
    bias = torch.randn(E, device=DEV) * 0.1
    go = lambda: lora.run_layer(bank, M, d["ad"], d["B"], d["x"], d["tad"], logits, routing=dict(ROUTING, bias=bias))
    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(3):
        d["x"].copy_(torch.randn(T, H, device=DEV))
        logits.copy_(torch.randn(T, E, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = d["B"].out.clone()
        assert torch.equal(got, go())


def test_layer_refuses_what_does_not_fit_before_it_runs(lora):
    T, H, I, E, k, Is = 6, 256, 128, 8, 2, 128
    dl = w4_layer(T, H, I, E, k, 1, Is, "a16", 77)
    M = dl.buffers("a16", 16)
    ad = lora.Adapters(2, E, H, I, 1, Is, max_rank=8, device=DEV)
    B = lora.LoraBuffers(T, H, I, E, k, 1, Is, 8, device=DEV)
    x, tad = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV), torch.zeros(T, dtype=torch.int32, device=DEV)
    M.ids.fill_(-7)
    go = lambda bank=dl.bank, M=M, ad=ad, B=B, x=x, tad=tad, logits=dl.logits, **kw: lora.run_layer(
        bank, M, ad, B, x, tad, logits, **kw)
    for kw, word in ((dict(x=x[:3]), "x"), (dict(x=x.float()), "x"), (dict(tad=tad[:2]), "adapter"),
                     (dict(tad=tad.long()), "adapter"), (dict(logits=dl.logits[:, :4]), "logits"),
                     (dict(shared_gate=torch.zeros(T, 2, device=DEV)), "shared_gate"),
                     (dict(B=lora.LoraBuffers(T, H, I, E, k, 1, 2 * Is, 8, device=DEV)), "different layers"),
                     (dict(B=lora.LoraBuffers(T, H, I, E, k, 1, 64, 8, device=DEV)), "different layers"),
                     (dict(B=lora.LoraBuffers(T, H, I, E, k, 1, Is, 8, h_f32=True, device=DEV)), "h_f32"),
                     (dict(ad=lora.Adapters(2, E, H, 64, 1, Is, max_rank=8, device=DEV)), "adapters"),
                     (dict(ad=lora.Adapters(2, E, H, I, 1, Is, max_rank=16, device=DEV)), "ranks")):
        with pytest.raises((ValueError, TypeError), match=word):
            go(**kw)
    bank, X = mx_layer(T, H, I, E, k, 1, Is, "a16", 1)
    with pytest.raises(ValueError, match="flags"):
        go(bank=bank, M=X, flags=1)
    torch.cuda.synchronize()
    assert (M.ids == -7).all()


@pytest.mark.parametrize("T,ranks", [(6, (8, 16)), (700, (8, 16)), (2100, (8, 16)), (4200, (16, 128))])
def test_a_token_that_lists_an_expert_twice(lora, T, ranks):
    """Both of its rows count, alone and between others of their expert."""
    d = make(lora, T, 64, 32, 4, 3, 0, 0, 2, ranks, out_f32=True, runs=True, none=0.0, seed=12)
    rng = np.random.default_rng(12)
    ids = d["ids"].copy()
    ids[::2, 1] = ids[::2, 0]
    ids[1::6, 2] = ids[1::6, 1] = ids[1::6, 0]
    flat = ids.ravel()
    order = np.argsort(flat, kind="stable").astype(np.int32)
    d["ids"], d["sp"], d["pos"] = ids, order, np.argsort(order).astype(np.int32)
    d["off"] = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=4))]).astype(np.int32)
    d["rows"] = O.rows_of(d["sp"], ids, T, 3, 4, 0)
    d["t"] = [dev(d[x]) for x in ("ids", "off", "sp", "pos")]
    check_gateup(d, run_gateup(lora, d))
    check_down(d, run_down(lora, d))


def test_more_experts_than_the_sums_of_a_block_hold(lora):
    """Shared experts beside 1024 routed ones: many rows, down in one launch."""
    d = make(lora, 40, 256, 32, 1024, 2, 70, 32, 1, (128,), none=0.0, seed=13)
    check_gateup(d, run_gateup(lora, d))
    check_down(d, run_down(lora, d))
    assert d["B"].error_word() == 0


@pytest.mark.parametrize("kind", ["mx", "w4"])
def test_layer_on_another_stream_with_fresh_buffers(lora, kind):
    """The first step on a stream of its own, while the current one is busy: nothing is
    made in the step, and the result is the one of the current stream."""
    T, H, I, E, k, Is = 300, 256, 128, 8, 2, 128
    if kind == "mx":
        bank, M = mx_layer(T, H, I, E, k, 1, Is, "a16", 21)
        x, logits = torch.randn(T, H, device=DEV).bfloat16(), torch.randn(T, E, device=DEV)
    else:
        dl = w4_layer(T, H, I, E, k, 1, Is, "a16", 321)
        bank, M, x, logits = dl.bank, dl.buffers("a16"), dl.x, dl.logits
    d = make(lora, T, H, I, E, k, 1, Is, 3, (8, 16), seed=22)
    sized = (T, H, I, E, k, 1, Is, 16)
    want = lora.run_layer(bank, M, d["ad"], lora.LoraBuffers(*sized, device=DEV), x, d["tad"], logits).clone()
    a, side = torch.randn(4096, 4096, device=DEV), torch.cuda.Stream()
    for _ in range(3):
        B = lora.LoraBuffers(*sized, device=DEV)
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(5):
            a @ a                                     # the current stream is busy
        before = torch.cuda.memory_stats()["allocation.all.allocated"]
        out = lora.run_layer(bank, M, d["ad"], B, x, d["tad"], logits, stream=side)
        assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
        side.synchronize()
        assert torch.equal(out, want) and B.error_word() == 0
        torch.cuda.synchronize()
    with pytest.raises(ValueError, match="layer=False"):
        lora.run_layer(bank, M, d["ad"], lora.LoraBuffers(*sized, device=DEV, layer=False), x, d["tad"], logits)


def test_layer_takes_no_flags_but_paths(lora):
    """MOE_X_PREPARED would read a copy of x that no call of the layer makes."""
    from packed_bit_grouped_amd import _lib as L
    T, H, I, E, k, Is = 6, 256, 128, 8, 2, 128
    dl = w4_layer(T, H, I, E, k, 1, Is, "a16", 78)
    M = dl.buffers("a16", 16)
    ad = lora.Adapters(2, E, H, I, 1, Is, max_rank=8, device=DEV)
    B = lora.LoraBuffers(T, H, I, E, k, 1, Is, 8, device=DEV)
    tad = torch.zeros(T, dtype=torch.int32, device=DEV)
    M.ids.fill_(-7)
    for flags in (L.MOE_X_PREPARED, L.MOE_LAYER_ONE_LAUNCH, L.MOE_OUT_F32, L.MOE_W_PREPACKED, L.MOE_GU_F32, L.MOE_H_F32):
        with pytest.raises(ValueError, match="flags"):
            lora.run_layer(dl.bank, M, ad, B, dl.x, tad, dl.logits, flags=flags)
    torch.cuda.synchronize()
    assert (M.ids == -7).all()
    lora.run_layer(dl.bank, M, ad, B, dl.x, tad, dl.logits, flags=L.MOE_PATH_MFMA16 | L.MOE_QUANT_SEPARATE)
    assert (M.ids >= 0).all()


def test_layer_refuses_banks_paths_and_flags_before_it_runs(lora):
    from packed_bit_grouped_amd import _lib as L
    T, H, I, E, k, Is = 6, 256, 128, 8, 2, 128
    dl = w4_layer(T, H, I, E, k, 1, Is, "a16", 78)
    M = dl.buffers("a16", 16)
    ad = lora.Adapters(2, E, H, I, 1, Is, max_rank=8, device=DEV)
    B = lora.LoraBuffers(T, H, I, E, k, 1, Is, 8, device=DEV)
    tad = torch.zeros(T, dtype=torch.int32, device=DEV)
    bank, X = mx_layer(T, H, I, E, k, 1, Is, "a16", 2)
    small = w4_layer(T, H, I, E - 4, k, 1, Is, "a16", 79).bank
    bare = w4_layer(T, H, I, E, k, 0, 0, "a16", 79).bank
    x = dl.x.view(torch.bfloat16)
    odd = torch.zeros(T * H + 4, dtype=torch.bfloat16, device=DEV)[4:].view(T, H)
    wide = dl.buffers("a16", 160)
    M.ids.fill_(-7), X.ids.fill_(-7), wide.ids.fill_(-7)
    go = lambda bank=dl.bank, M=M, x=x, **kw: lora.run_layer(bank, M, ad, B, x, tad, dl.logits, **kw)
    for kw, kind, word in (
            (dict(bank=bank), TypeError, "bank"), (dict(M=X), TypeError, "bank"), (dict(bank=small), ValueError, "w13"),
            (dict(bank=bare), ValueError, "w13_sh"), (dict(x=odd), ValueError, "aligned"),
            (dict(bank=mx_layer(T, H, I, E - 1, k, 1, Is, "a16", 3)[0], M=X), ValueError, "w13"),
            (dict(bank=mx_layer(T, H, I + 32, E, k, 1, Is, "a16", 3)[0], M=X), ValueError, "w13"),
            (dict(bank=mx_layer(T, H, I, E, k, 0, 0, "a16", 3)[0], M=X), ValueError, "w13_shared"),
            (dict(flags=L.MOE_X_PREPARED), ValueError, "flags"), (dict(flags=L.MOE_LAYER_ONE_LAUNCH), ValueError, "flags"),
            (dict(flags=L.MOE_OUT_F32), ValueError, "flags"), (dict(flags=L.MOE_H_F32), ValueError, "flags"),
            (dict(flags=L.MOE_PATH_MFMA16, M=wide), L.MoeError, "moe_w4_covers"),
            (dict(bank=dl.bank.prepack()), L.MoeError, "moe_w4_covers"),
            (dict(routing=dict(n_group=3)), L.MoeError, "moe_route_scored"),
            (dict(routing=dict(n_group=8, topk_group=1)), L.MoeError, "moe_route_scored")):
        with pytest.raises(kind, match=word):
            go(**kw)
    torch.cuda.synchronize()
    assert all((m.ids == -7).all() for m in (M, X, wide))
    assert B.error_word() == M.error_word() == 0
    go(), go(flags=L.MOE_PATH_MFMA16 | L.MOE_QUANT_SEPARATE)       # what fits runs
    assert (M.ids >= 0).all()
