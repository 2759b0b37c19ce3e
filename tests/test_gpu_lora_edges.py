"""The adapters' calls where their other tests do not go: the sums of a block of
tokens over several segments of windows and more units than are taken at a time;
fp32 operands to their last bit."""
import numpy as np
import pytest

from oracle import lora_oracle as O
from packed_bit_grouped_amd import _lib as L

torch = pytest.importorskip("torch")
from test_gpu_lora import DEV, check_down, check_gateup, dev, f64, make, run_down, run_gateup, tables  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lora():
    from packed_bit_grouped_amd import lora as m
    return m


# ---------------------------------------------------------------------------
# down of many rows: a block's rows, experts in order, in windows of 64, 16
# windows (a segment) at a time, of which 128 units at a time

WINDOW, SEGMENT, UNITS = 64, 16, 128


def units_by_segment(d, block):
    """Units (up to 16 rows of one adapter and expert, a token once) of every
    block's segments, counted from the tables."""
    T, k, E, out = d["T"], d["k"], d["E"], []
    for t0 in range(0, T, block):
        rows = [(t, e) for t, e in d["rows"][:T * k] if t0 <= t < t0 + block and e >= 0]
        rows += [(t, E + s) for s in range(d["n_shared"]) for t in range(t0, min(T, t0 + block))]
        counts = []
        for w in range(0, len(rows), WINDOW):
            groups = {}
            for i, (t, e) in enumerate(rows[w:w + WINDOW]):
                a = int(d["adapter"][t])
                if 0 <= a < len(d["dn"]) and d["dn"][a][e] is not None:
                    again = sum(1 for q in rows[w:w + i] if q == (t, e))
                    groups[a, e, again] = groups.get((a, e, again), 0) + 1
            counts.append(sum((n + 15) // 16 for n in groups.values()))
        out.append([sum(counts[i:i + SEGMENT]) for i in range(0, len(counts), SEGMENT)])
    return out


def block_of(d):
    return L.moe_lora_block(d["T"], d["H"], d["I"], d["E"], d["k"], d["n_shared"], d["I_shared"], d["ad"].n,
                            d["B"].max_rank, 1)


def leave_alone(d, experts):
    """No adapter has matrices for these experts."""
    for i in range(d["ad"].n):
        for e in experts:
            d["ad"]._entries("2", i, e, 1)[:] = 0
            d["dn"][i][e] = None
        d["ad"]._put("2", i, 0, d["ad"].per, None)


SEGMENTS = [  # T, H, I, E, k, n_shared, I_shared, adapters, ranks, runs, h and out in fp32
    (600, 8192, 64, 16, 8, 1, 96, 2, (8, 16), True, False, False),   # 73 windows of a block: the fifth segment is partial
    (600, 8192, 64, 16, 8, 1, 96, 2, (8, 16), True, True, True),
    (1100, 5632, 64, 12, 5, 0, 0, 3, (8, 40, 64), True, False, True),    # 40 windows, ranks up to 64
    (600, 8192, 32, 5, 3, 2, 64, 3, (16, 104, 128), True, False, False),  # and up to 128
    (600, 8192, 64, 12, 8, 1, 96, 32, (8, 24, 32), False, False, True),  # a unit for two or three rows
    (530, 8192, 96, 10, 5, 1, 32, 20, (72, 128), False, True, False),
]


@pytest.mark.parametrize("case", SEGMENTS)
def test_sums_of_a_block_over_several_segments(lora, case):
    T, H, I, E, k, s, Is, n, ranks, runs, wide, out_f32 = case
    d = make(lora, T, H, I, E, k, s, Is, n, ranks, h_f32=wide, out_f32=out_f32, runs=runs, none=0.1, seed=T + n)
    block = block_of(d)
    assert block == 512
    units = units_by_segment(d, block)
    assert len(units[0]) >= 3 and min(units[0]) > 0
    if not runs:                       # the next units of a segment, once and more often
        assert max(units[0]) > 2 * UNITS
    check_down(d, run_down(lora, d))
    assert d["B"].error_word() == 0


@pytest.mark.parametrize("silent,empty", [((0, 1), (0,)), ((2, 3), (1,)), ((2, 3, 4, 5), (1, 2)),
                                          ((0, 1, 4, 5, 6, 7, 8), (0, 2, 3, 4)), (range(9), (0, 1, 2, 3, 4))])
def test_segments_without_units_between_others(lora, silent, empty):
    T, H, I, E = 600, 8192, 32, 8      # every token takes all experts: two experts a segment
    d = make(lora, T, H, I, E, 8, 1, 64, 2, (16,), out_f32=True, runs=True, none=0.0, seed=31)
    leave_alone(d, silent)
    assert block_of(d) == 512
    units = units_by_segment(d, 512)
    assert [i for i, u in enumerate(units[0]) if u == 0] == list(empty) and len(units[0]) == 5
    check_down(d, run_down(lora, d))
    assert d["B"].error_word() == 0


# ---------------------------------------------------------------------------
# Fp32 operands go into the matrix cores as three parts of 8 bits.  With matrices
# whose rows hold powers of two a result has the 24 bits of one operand, and every
# partial sum on the way is a run of its bits: nothing may be rounded, so the
# calls have to be exact.  (A bound of worst-case sums of K products is above what
# a lost third part changes.)


def power(rng, *shape):
    return 2.0 ** rng.integers(-3, 4, shape) * rng.choice([-1.0, 1.0], shape)


def one_entry_rows(rng, n, K):
    """[n][K] with a power of two in one column of each row; the columns, the entries."""
    col, val = rng.integers(0, K, n), power(rng, n)
    m = np.zeros((n, K))
    m[np.arange(n), col] = val
    return m, col, val


def bits24(rng, *shape):
    """Numbers of [1, 2) with 24 bits, the last one set."""
    return 1.0 + (rng.integers(0, 1 << 22, shape) * 2 + 1) * 2.0 ** -23


def two_parts(f):
    """f without its last 8 bits."""
    return (f.astype(np.float32).view(np.uint32) & 0xFFFFFF00).view(np.float32)


def bf(a):
    t = torch.from_numpy(np.ascontiguousarray(a).astype(np.float32)).bfloat16()
    assert np.array_equal(t.double().numpy(), a)
    return t.to(DEV)


@pytest.mark.parametrize("T,H,I,rank,many", [
    (1, 64, 32, 8, False), (40, 416, 96, 24, False), (300, 64, 64, 128, False), (9, 2048, 512, 40, False),
    (20000, 512, 64, 16, True), (4000, 544, 96, 72, True), (4000, 512, 64, 128, True)])
def test_down_keeps_every_bit_of_h_and_v(lora, T, H, I, rank, many):
    rng = np.random.default_rng(T + rank)
    E, scale = 3, 0.25
    ids, off, sp, pos = tables(rng, T, 1, E)
    assert (L.moe_lora_block(T, H, I, E, 1, 0, 0, 1, rank, 1) > 0) == many
    ad, a2, b2 = lora.Adapters(1, E, H, I, max_rank=rank, device=DEV), [], []
    for e in range(E):
        a2.append(one_entry_rows(rng, rank, I))
        b2.append(one_entry_rows(rng, H, rank))
    ad.load(0, a2=bf(np.stack([m for m, _, _ in a2])), b2=bf(np.stack([m for m, _, _ in b2])), scale=scale)
    h, w = bits24(rng, T, I) * power(rng, T, I), power(rng, T, 1)
    want = np.zeros((T, H))
    for t in range(T):
        e = ids[t, 0]
        v = scale * a2[e][2] * h[pos[t], a2[e][1]]
        want[t] = w[t, 0] * b2[e][2] * v[b2[e][1]]
    assert (two_parts(want) != want).all()
    B = lora.LoraBuffers(T, H, I, E, 1, max_rank=rank, h_f32=True, out_f32=True, device=DEV)
    out = lora.down_combine(ad, dev(h.astype(np.float32)), torch.zeros(T, H, device=DEV),
                            torch.zeros(T, dtype=torch.int32, device=DEV), dev(w.astype(np.float32)),
                            *map(dev, (ids, off, sp, pos)), B)
    assert np.array_equal(f64(out), want)


@pytest.mark.parametrize("T,I,rank,many", [
    (1, 32, 8, False), (9, 160, 128, False), (300, 96, 40, False), (640, 64, 16, False),
    (3000, 96, 8, True), (3000, 320, 40, True), (2100, 64, 128, True)])
@pytest.mark.parametrize("half", ["gate", "up"])
def test_gateup_keeps_every_bit_of_v(lora, T, I, rank, many, half):
    """v of 24 bits from x of 8: columns 3 q, 3 q + 1 and 3 q + 2 hold 8 bits each, the
    next ones behind the last.  Through up: SiLU(64) = 64 in fp32.  Through gate: SiLU(g)
    = g for g >= 64, u = 1."""
    rng = np.random.default_rng(T + rank)
    E, H, scale = 3, 96, 2.0
    ids, off, sp, pos = tables(rng, T, 1, E)
    assert (L.moe_lora_block(T, H, I, E, 1, 0, 0, 1, rank, 0) > 0) == many
    x = rng.integers(128, 256, (T, H)) * 2.0 ** (-8 * (np.arange(H) % 3))
    x[:, 2::3] += 2.0 ** -16 * (x[:, 2::3] * 2 ** 16 % 2 == 0)        # the last bit set
    a13, b13 = np.zeros((E, 2 * rank, H)), np.zeros((E, 2 * I, rank))
    want = np.zeros((T, I))
    for e in range(E):
        q, pa = rng.integers(0, H // 3, rank), 2.0 ** rng.integers(0, 4, rank)
        b, col, pb = one_entry_rows(rng, I, rank)
        first = 0 if half == "gate" else rank
        for i in range(3):
            a13[e, first + np.arange(rank), 3 * q + i] = pa
        if half == "gate":
            b, pb = np.abs(b), np.abs(pb) * 8                            # g of 128 and more
            b *= 8
        b13[e, :I] = b if half == "gate" else 0.0
        b13[e, I:] = b if half == "up" else 0.0
        t = np.nonzero(ids[:, 0] == e)[0]
        v = scale * pa * x[t].reshape(len(t), H // 3, 3).sum(2)[:, q]
        want[pos[t]] = pb * v[:, col] * (64.0 if half == "up" else 1.0)
    assert (two_parts(want) != want).all() and (half == "up" or (want >= 64).all())
    ad = lora.Adapters(1, E, H, I, max_rank=rank, device=DEV)
    ad.load(0, bf(a13), bf(b13), scale=scale)
    gu = np.zeros((T, 2 * I), dtype=np.float32)
    gu[:, :I], gu[:, I:] = (64.0, 0.0) if half == "up" else (0.0, 1.0)
    B = lora.LoraBuffers(T, H, I, E, 1, max_rank=rank, h_f32=True, device=DEV)
    h = lora.gateup_silu(ad, bf(x), torch.zeros(T, dtype=torch.int32, device=DEV), dev(gu),
                         *map(dev, (ids, off, sp)), B)
    assert np.array_equal(f64(h), want)


# ---------------------------------------------------------------------------
# the routing's tables


@pytest.mark.parametrize("T,ranks", [(5, (8, 16)), (70, (8, 16)), (2400, (8, 16)), (2400, (8, 128))])
@pytest.mark.parametrize("wide", [False, True])
def test_a_pair_without_a_place_adds_nothing(lora, T, ranks, wide):
    """pair_pos -1 takes a pair out of the sum whatever the other tables say, as in
    the shared down projection."""
    d = make(lora, T, 4096, 64, 6, 3, 1, 32, 3, ranks, h_f32=wide, out_f32=True, none=0.1, seed=T)
    assert (block_of(d) > 0) == (T > 70)
    d["pos"][np.random.default_rng(1).random(3 * T) < 0.3] = -1
    d["pos"][:3] = -1
    d["t"][3] = dev(d["pos"])
    check_down(d, run_down(lora, d))
    assert d["B"].error_word() == 0


@pytest.mark.parametrize("T,ranks", [(6, (8, 16)), (2400, (8, 16)), (2400, (8, 128))])
@pytest.mark.parametrize("gone", [0, 1, 2])
def test_a_token_s_places_of_one_expert_one_of_them_taken_out(lora, T, ranks, gone):
    """Three times the same expert, the first, second or third of them without a place."""
    d = make(lora, T, 4096, 64, 4, 3, 0, 0, 2, ranks, out_f32=True, runs=True, none=0.0, seed=41)
    ids = np.repeat(d["ids"][:, :1], 3, 1)
    order = np.argsort(ids.ravel(), kind="stable").astype(np.int32)
    pos = np.argsort(order).astype(np.int32).reshape(T, 3)
    pos[::2, gone] = -1
    d["ids"], d["sp"], d["pos"] = ids, order, pos.ravel()
    d["off"] = np.concatenate([[0], np.cumsum(np.bincount(ids.ravel(), minlength=4))]).astype(np.int32)
    d["rows"] = [(int(p) // 3, int(ids.ravel()[p])) for p in order]
    d["t"] = [dev(d[x]) for x in ("ids", "off", "sp", "pos")]
    assert (block_of(d) > 0) == (T > 6)
    check_down(d, run_down(lora, d))


@pytest.mark.parametrize("ranks", [(8, 16), (8, 128)])
def test_rows_that_the_offsets_leave_out_touch_no_other_token(lora, ranks):
    """Lists that contradict each other: rows of valid pairs that no expert's offsets
    hold.  What an earlier call left in the workspace is not taken for their places."""
    T, E = 2400, 6
    d = make(lora, T, 4096, 64, E, 1, 0, 0, 3, ranks, out_f32=True, none=0.0, seed=43)
    assert block_of(d) > 0
    check_down(d, run_down(lora, d))                  # a place for every row
    cut = int(d["off"][3] - 40)                       # expert 2 ends early: its last 40 rows are nobody's
    d["off"][3] = cut
    left = [d["rows"][r][0] for r in range(cut, cut + 40)]
    rng = np.random.default_rng(44)
    d["adapter"] = rng.integers(0, 3, T).astype(np.int32)      # other places than before
    d["tad"], d["t"][1] = dev(d["adapter"]), dev(d["off"])
    out = run_down(lora, d)
    others = np.setdiff1d(np.arange(T), left)
    pos = d["pos"].copy()
    pos[left] = -1
    want, bound = O.down(f64(d["base"]), f64(d["h"]), d["rows"], d["adapter"], d["dn"], d["widths"], f64(d["w"]), pos,
                         np.ones((T, 0)), T, 1, False)
    assert (np.abs(f64(out) - want)[others] <= bound[others]).all()


# ---------------------------------------------------------------------------
# sizes, streams and graphs


class Far:
    """Rows of a device tensor, fetched one at a time, as the oracle indexes them."""

    def __init__(self, t):
        self.t = t

    def __getitem__(self, at):
        return f64(self.t[at[0], at[1]])


@pytest.mark.parametrize("wide", [False, True])
def test_more_sums_and_rows_of_h_than_32_bits_count(lora, wide):
    """gu of 2^31 values and more, h of 2^31 bytes and more."""
    T, H, I, E, k, rank = 70000, 64, 2048, 8, 8, 8
    rng = np.random.default_rng(51)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    order = np.argsort(ids.ravel(), kind="stable").astype(np.int32)
    pos = np.argsort(order).astype(np.int32)
    off = np.concatenate([[0], np.cumsum(np.bincount(ids.ravel(), minlength=E))]).astype(np.int32)
    adapter = rng.integers(-1, 2, T).astype(np.int32)
    ad = lora.Adapters(2, E, H, I, max_rank=rank, device=DEV)
    up, dn = [[None] * E for _ in range(2)], [[None] * E for _ in range(2)]
    for i in range(2):
        a13, b13, a2, b2 = (torch.randn(E, *s, device=DEV).bfloat16() * 0.3
                            for s in ((2 * rank, H), (2 * I, rank), (rank, I), (H, rank)))
        ad.load(i, a13, b13, a2, b2, scale=0.5)
        for e in range(E):
            up[i][e], dn[i][e] = (f64(a13[e]), f64(b13[e]), 0.5), (f64(a2[e]), f64(b2[e]), 0.5)
    x, R = torch.randn(T, H, device=DEV).bfloat16(), T * k
    t = list(map(dev, (ids, off, order, pos)))
    tad, w = dev(adapter), torch.rand(T, k, device=DEV)
    B = lora.LoraBuffers(T, H, I, E, k, max_rank=rank, h_f32=wide, out_f32=True, device=DEV)
    assert B.gu.numel() > 1 << 31 and B.h.numel() * 2 > 1 << 31
    for i in range(0, R, 1 << 17):
        B.gu[i:i + (1 << 17)].normal_()
    h = lora.gateup_silu(ad, x, tad, B.gu, *t[:3], B)
    some = np.unique(np.concatenate([[0, R - 1], rng.integers(0, R, 60), rng.integers(R - 2000, R, 20)]))
    rows = [(int(order[r]) // k, int(ids.ravel()[order[r]])) for r in some]
    want, bound = O.gateup(f64(B.gu[some]), f64(x), rows, adapter, up, [I] * E, I, not wide)
    assert (np.abs(f64(h[some]) - want) <= bound).all()
    base = torch.randn(T, H, device=DEV)
    out = lora.down_combine(ad, h, base, tad, w, *t, B)
    tok = np.unique(np.concatenate([[0, T - 1], rng.integers(0, T, 20)]))
    n = len(tok)
    all_rows = {int(r): (i, int(ids[q, j])) for i, q in enumerate(tok) for j, r in enumerate(pos.reshape(T, k)[q])}
    want, bound = O.down(f64(base[tok]), Far(h), all_rows, adapter[tok], dn, [I] * E, f64(w[tok]),
                         pos.reshape(T, k)[tok].ravel(), np.ones((n, 0)), n, k, False)
    assert (np.abs(f64(out[tok]) - want) <= bound).all()
    assert B.error_word() == 0
    del B, h, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [20, 900])
def test_two_graphs_share_buffers_and_adapters_change_between_replays(lora, T):
    d = make(lora, T, 128, 64, 6, 3, 1, 64, 3, (8, 16), none=0.0, seed=61)
    other = {**d, "x": torch.randn_like(d["x"]), "h": torch.randn(d["h"].shape, device=DEV).to(d["h"].dtype)}
    graphs = []
    torch.cuda.synchronize()
    for q in (d, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run_gateup(lora, q)
            run_down(lora, q)
        graphs.append(g)
    rng = np.random.default_rng(62)
    for i in range(4):
        for g, q in zip(graphs, (d, other)):
            g.replay()
            h, out = d["B"].h.clone(), d["B"].out.clone()
            assert torch.equal(h, run_gateup(lora, q)) and torch.equal(out, run_down(lora, q))
        torch.cuda.synchronize()
        r = (8, 16)[i % 2]
        bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32) * 0.2).bfloat16().to(DEV)
        d["ad"].load(i % 3, bf(6, 2 * r, 128), bf(6, 128, r), bf(6, r, 64), bf(6, 128, r), scale=0.5)


@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_adapters_are_loaded_on_the_stream_that_uses_them(lora, kind):
    d = make(lora, 40, 128, 64, 4, 2, 0, 0, 2, (8,), none=0.0, seed=63)
    side = torch.cuda.Stream()
    arg = side if kind == "stream" else side.cuda_stream
    busy = torch.randn(4096, 4096, device=DEV)
    rng = np.random.default_rng(64)
    for i in range(4):
        m = [torch.from_numpy(rng.standard_normal(s).astype(np.float32) * 0.2).bfloat16().to(DEV)
             for s in ((4, 16, 128), (4, 128, 8), (4, 8, 64), (4, 128, 8))]
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(5):
            busy @ busy                               # the current stream is behind
        d["ad"].load(i % 2, *m, scale=0.5, stream=arg)
        for e in range(4):
            d["up"][i % 2][e] = (f64(m[0][e]), f64(m[1][e]), 0.5)
            d["dn"][i % 2][e] = (f64(m[2][e]), f64(m[3][e]), 0.5)
        del m                                         # its memory may go to the current stream's work
        torch.randn(4, 128, 8, device=DEV)
        h, out = run_gateup(lora, d, stream=arg), run_down(lora, d, stream=arg)
        side.synchronize()
        check_gateup(d, h)
        check_down(d, out)


@pytest.mark.parametrize("T,held,room", [(5, 8, 128), (60, 24, 40), (2400, 8, 40), (2400, 16, 128)])
def test_buffers_for_higher_ranks_than_the_adapters_have(lora, T, held, room):
    d = make(lora, T, 4096, 64, 5, 3, 1, 96, 3, (8, held), seed=71)
    d["B"] = lora.LoraBuffers(T, 4096, 64, 5, 3, 1, 96, room, device=DEV)
    assert (block_of(d) > 0) == (T > 60)
    check_gateup(d, run_gateup(lora, d))
    check_down(d, run_down(lora, d))
    assert d["B"].error_word() == 0


def test_no_tokens(lora):
    d = make(lora, 0, 64, 32, 4, 2, 1, 64, 2, (8,), seed=72)
    assert run_gateup(lora, d).shape == (0, 64) and run_down(lora, d).shape == (0, 64)
    assert d["B"].error_word() == 0
