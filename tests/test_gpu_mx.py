"""The MXFP4 operators on the GPU against the fp64 oracle (oracle/mx_oracle.py):
codes, scales and values bit for bit; projections within the bound of fp32
sums and one rounding to bf16."""
import numpy as np
import pytest

import oracle
from oracle import mx_oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def mx():
    from packed_bit_grouped_amd import mx as m
    return m


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def bf16_rows(rng, R, C, scale=1.0):
    return torch.from_numpy((rng.standard_normal((R, C)) * scale).astype(np.float32)).bfloat16()


def matrices(rng, n, N, K, scale=0.05):
    """n quantised matrices: device (codes, scales) and their fp64 values."""
    codes, scales = O.quantise((rng.standard_normal((n, N, K)) * scale).astype(np.float32))
    pair = (torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV))
    return pair, O.values(codes, scales)


# ---------------------------------------------------------------------------
# rows


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,C,pad", [(1, 32, 0), (3, 96, 0), (12, 2048, 0), (7, 1056, 8), (5, 64, 3),
                                     (257, 352, 1), (1000, 4096, 0)])
def test_rows_match_oracle(mx, dtype, R, C, pad):
    rng = np.random.default_rng(R * C + pad)
    v = rng.standard_normal((R, C + pad)) * np.exp(rng.standard_normal((R, 1)) * 10)
    v[:, :32] *= rng.random((R, 1)) > 0.3
    src = torch.from_numpy(v.astype(np.float32)).to(dtype).to(DEV)[:, :C]
    codes, scales = mx.quantize_rows(src)
    want_c, want_s = O.quantise(f64(src))
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    want = O.values(want_c, want_s)
    assert np.array_equal(f64(mx.dequantize_rows(codes, scales)), want)
    assert np.array_equal(f64(mx.dequantize_rows(codes, scales, torch.float32)), want)


def test_every_bf16_value(mx):
    """Every bf16 bit pattern in blocks of neighbours, of its own alone, and
    under a large first value (codes of everything that rounds to 0, ties)."""
    bits = np.arange(65536, dtype=np.uint32)
    all_v = (bits << 16).astype(np.uint32).view(np.float32)
    alone = np.zeros((65536, 32), dtype=np.float32)
    alone[:, 3] = all_v
    under = np.zeros((4096, 32), dtype=np.float32)
    under[:, 1:17] = all_v.reshape(4096, 16)
    fin = np.where(np.isfinite(under), np.abs(under), 0).max(-1)
    under[:, 0] = np.where(fin < 8e37, fin, 0) * 4
    for v in (all_v.reshape(2048, 32), alone, under):
        src = torch.from_numpy(v).bfloat16().to(DEV)
        codes, scales = mx.quantize_rows(src)
        want_c, want_s = O.quantise(f64(src))
        assert np.array_equal(scales.cpu().numpy(), want_s)
        assert np.array_equal(codes.cpu().numpy(), want_c)


def test_fp32_ties_and_their_neighbours(mx):
    mids = (O.GRID[1:] + O.GRID[:-1]) / 2
    v = []
    for e in (-126, -3, 0, 40, 120):
        for m in np.float32(mids):
            for x in (m, np.nextafter(m, np.float32(9)), np.nextafter(m, np.float32(0))):
                row = np.zeros(32, dtype=np.float32)
                row[:3] = [4, x, -x]
                v.append(np.ldexp(row, e).astype(np.float32))
    src = torch.from_numpy(np.stack(v)).to(DEV)
    codes, scales = mx.quantize_rows(src)
    want_c, want_s = O.quantise(f64(src))
    assert np.array_equal(codes.cpu().numpy(), want_c) and np.array_equal(scales.cpu().numpy(), want_s)


def test_every_code_and_scale_back(mx):
    codes = np.tile(O.pack(np.tile(np.arange(16, dtype=np.uint8), 2)[None]), (256, 1))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    c, s = torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV)
    want = O.values(codes, scales)
    for dtype, top in ((torch.bfloat16, 253), (torch.float32, 253)):
        got = f64(mx.dequantize_rows(c, s, dtype))
        assert np.array_equal(got[:top], want[:top])
        assert np.isnan(got[255]).all()
        big = np.abs(want[253:255]) >= 2.0 ** 128    # beyond the type: inf
        assert np.isinf(got[253:255][big]).all()
        assert np.array_equal(got[253:255][~big], want[253:255][~big])


def test_rows_of_other_layouts(mx):
    """Given outputs are filled and nothing else is; one row of any stride; no rows."""
    rng = np.random.default_rng(5)
    src = bf16_rows(rng, 40, 128).to(DEV)
    big_c = torch.full((42, 64), 77, dtype=torch.uint8, device=DEV)
    big_s = torch.full((42, 4), 77, dtype=torch.uint8, device=DEV)
    mx.quantize_rows(src, big_c[1:41], big_s[1:41])
    c, s = mx.quantize_rows(src)
    assert torch.equal(big_c[1:41], c) and torch.equal(big_s[1:41], s)
    for b in (big_c, big_s):
        assert (b[0] == 77).all() and (b[41] == 77).all()
    c1, s1 = mx.quantize_rows(src[7:8])
    assert torch.equal(c1, c[7:8]) and torch.equal(s1, s[7:8])
    c0, s0 = mx.quantize_rows(src[:0])
    assert c0.shape == (0, 64) and mx.dequantize_rows(c0, s0).shape == (0, 128)


def test_rows_past_32_bit_offsets(mx):
    R, C = 66000, 65536                       # 4.3e9 values, 8.7 GB of bf16
    src = torch.zeros((R, C), dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(6)
    rows = [0, 32767, 32768, 65535, 65536, R - 1]
    for r in rows:
        src[r] = bf16_rows(rng, 1, C)[0].to(DEV)
    codes, scales = mx.quantize_rows(src)
    back = mx.dequantize_rows(codes, scales)
    for r in rows:
        want_c, want_s = O.quantise(f64(src[r:r + 1]))
        assert np.array_equal(codes[r].cpu().numpy(), want_c[0])
        assert np.array_equal(scales[r].cpu().numpy(), want_s[0])
        assert np.array_equal(f64(back[r]), O.values(want_c, want_s)[0])
    del src, codes, scales, back
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n,N,K", [(1, 16, 32), (2, 48, 128), (3, 32, 352), (2, 64, 2080), (1, 128, 512)])
def test_tiles_match_their_definition(mx, n, N, K):
    """The header's layout, built here from plain rows."""
    rng = np.random.default_rng(K)
    codes = rng.integers(0, 256, (n, N, K // 2), dtype=np.uint8)
    scales = rng.integers(0, 256, (n, N, K // 32), dtype=np.uint8)
    pieces = -(-K // 128)
    words = -(-pieces // 4)
    blk = np.zeros((n, N // 16, 16, pieces * 4, 16), dtype=np.uint8)
    blk[:, :, :, :K // 32] = codes.reshape(n, N // 16, 16, K // 32, 16)
    want = blk.reshape(n, N // 16, 16, pieces, 4, 16).transpose(0, 1, 3, 4, 2, 5)   # s, g, c
    sc = np.zeros((n, N // 16, 16, words * 16), dtype=np.uint8)
    sc[..., :K // 32] = scales.reshape(n, N // 16, 16, K // 32)
    want_s = sc.reshape(n, N // 16, 16, words, 4, 4).transpose(0, 1, 3, 5, 2, 4)    # S, g, c, j
    bank = mx.MxBank((torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV)))
    tc, ts = bank.tiles["w13"]
    assert np.array_equal(tc.cpu().numpy(), want.ravel())
    assert np.array_equal(ts.cpu().numpy(), want_s.ravel())


# ---------------------------------------------------------------------------
# projections


def make(mx, T, H, I, E, k, n_sh=0, I_sh=0, act="a16", seed=0, skew=0.0, out_f32=False):
    """A layer's device inputs and their fp64 values."""
    rng = np.random.default_rng(seed)
    I_sh = I_sh or I
    d = {"dims": (T, H, I, E, k, n_sh, I_sh), "act": act}
    d["x"] = bf16_rows(rng, T, H).to(DEV)
    logits = rng.standard_normal((T, E)) - skew * np.log(1 + rng.permutation(E))
    d["logits"] = torch.from_numpy(logits.astype(np.float32)).to(DEV)
    p13, d["v13"] = matrices(rng, E, 2 * I, H)
    p2, d["v2"] = matrices(rng, E, H, I)
    s13, d["v13s"] = matrices(rng, n_sh, 2 * I_sh, H) if n_sh else (None, None)
    s2, d["v2s"] = matrices(rng, n_sh, H, I_sh) if n_sh else (None, None)
    d["gate"] = torch.from_numpy(rng.standard_normal((T, n_sh)).astype(np.float32)).to(DEV) if n_sh else None
    d["w13"], d["bank"] = p13, mx.MxBank(p13, p2, s13, s2)
    d["B"] = mx.MxBuffers(T, H, I, E, k, n_sh, I_sh if n_sh else 0, act=act, device=DEV, out_f32=out_f32)
    d["B"].ws.fill_(255)     # nothing in the workspace may matter
    return d


def tables(d):
    T, H, I, E, k, n_sh, I_sh = d["dims"]
    ids, w = oracle.route_topk(d["logits"].cpu().numpy(), k)
    perm = oracle.permute(ids, E, 16)
    return ids, w, perm


def check_h(d, h, perm):
    T, H, I, E, k, n_sh, I_sh = d["dims"]
    x = O.activations(f64(d["x"]), d["act"])
    got = f64(h)
    off = perm["offsets"]
    for e in range(E + n_sh):
        lo, hi = (off[e], off[e + 1]) if e < E else (T * k + (e - E) * T, T * k + (e - E + 1) * T)
        if hi == lo:
            continue
        tok = perm["sorted_pair"][lo:hi] // k if e < E else np.arange(T)
        Ie = I if e < E else I_sh
        want, bound = O.gateup(x[tok], d["v13"][e] if e < E else d["v13s"][e - E], Ie)
        assert (np.abs(got[lo:hi, :Ie] - want) <= bound).all(), (e, np.abs(got[lo:hi, :Ie] - want).max())


def check_out(d, out, h, perm, w, gates):
    """out against the oracle applied to the h that the kernel read."""
    T, H, I, E, k, n_sh, I_sh = d["dims"]
    hv = f64(h)
    y = np.zeros((T * k + n_sh * T, H))
    dy = np.zeros_like(y)
    off = perm["offsets"]
    for e in range(E + n_sh):
        lo, hi = (off[e], off[e + 1]) if e < E else (T * k + (e - E) * T, T * k + (e - E + 1) * T)
        if hi == lo:
            continue
        Ie = I if e < E else I_sh
        y[lo:hi], dy[lo:hi] = O.project(O.activations(hv[lo:hi, :Ie], d["act"]),
                                        d["v2"][e] if e < E else d["v2s"][e - E])
    want, bound = O.combine(w, y, dy, perm["pair_pos"], T, k, gates)
    if out.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(want) + bound) + 2.0 ** -133
    got = f64(out)
    assert (np.abs(got - want) <= bound).all(), np.abs(got - want).max()


def gates_of(d, gated):
    T, n_sh = d["dims"][0], d["dims"][5]
    if not gated or not n_sh:
        return np.ones((T, n_sh))
    return 1 / (1 + np.exp(-f64(d["gate"])))


SHAPES = [
    # T, H, I, E, k, n_shared, I_shared
    (1, 32, 32, 1, 1, 0, 0),
    (1, 256, 128, 8, 2, 1, 128),
    (2, 64, 96, 4, 4, 0, 0),
    (5, 96, 32, 3, 2, 2, 64),
    (16, 512, 128, 2, 1, 0, 0),
    (17, 1056, 352, 12, 3, 1, 32),
    (37, 288, 160, 70, 5, 0, 0),
    (64, 2048, 768, 16, 2, 0, 0),
    (130, 544, 64, 3, 2, 1, 224),
    (300, 256, 96, 5, 2, 0, 0),
    (700, 640, 192, 4, 1, 1, 192),
    (3, 2080, 1056, 13, 8, 1, 1056),
]


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gateup(mx, shape, act):
    d = make(mx, *shape, act=act, seed=sum(shape), skew=1.0)
    ids, w, perm = tables(d)
    B = d["B"]
    h = mx.gateup_silu(d["bank"], d["x"], torch.from_numpy(perm["offsets"]).to(DEV),
                       torch.from_numpy(perm["sorted_pair"]).to(DEV), B)
    assert h is B.h
    check_h(d, h, perm)


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_down(mx, shape, act):
    d = make(mx, *shape, act=act, seed=sum(shape) + 1, skew=0.5, out_f32=sum(shape) % 2 == 0)
    ids, w, perm = tables(d)
    B, rng = d["B"], np.random.default_rng(9)
    h = bf16_rows(rng, B.R, B.ld_h).to(DEV)
    w32 = torch.from_numpy(w.astype(np.float32)).to(DEV)
    gated = shape[0] % 2 == 1
    out = mx.down_combine(d["bank"], h, w32, torch.from_numpy(perm["offsets"]).to(DEV),
                          torch.from_numpy(perm["pair_pos"]).to(DEV), B,
                          shared_gate=d["gate"] if gated else None)
    check_out(d, out, h, perm, f64(w32), gates_of(d, gated))


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_layer(mx, shape, act):
    d = make(mx, *shape, act=act, seed=sum(shape) + 2, skew=1.1, out_f32=sum(shape) % 2 == 1)
    B = d["B"]
    ids, w, perm = tables(d)
    out = mx.run_layer(d["bank"], d["x"], d["logits"], B, shared_gate=d["gate"])
    assert np.array_equal(B.ids.cpu().numpy(), ids)
    for name in ("counts", "offsets", "sorted_pair", "pair_pos"):
        assert np.array_equal(getattr(B, name).cpu().numpy(), perm[name]), name
    assert (np.abs(f64(B.w) - w) <= 16 * O.EPS32 * w).all()
    check_h(d, B.h, perm)
    check_out(d, out, B.h, perm, f64(B.w), gates_of(d, True))
    # and it is the parts, bit for bit
    h1, o1 = B.h.clone(), out.clone()
    h2 = mx.gateup_silu(d["bank"], d["x"], B.offsets, B.sorted_pair, B)
    assert torch.equal(h1.view(torch.int16), h2.view(torch.int16))
    o2 = mx.down_combine(d["bank"], h2, B.w, B.offsets, B.pair_pos, B, shared_gate=d["gate"])
    assert torch.equal(o1, o2)


def test_plain_softmax_weights(mx):
    d = make(mx, 9, 64, 32, 6, 2)
    mx.run_layer(d["bank"], d["x"], d["logits"], d["B"], renormalize=0)
    _, w = oracle.route_topk(d["logits"].cpu().numpy(), 2, 0)
    assert (np.abs(f64(d["B"].w) - w) <= 16 * O.EPS32 * w).all()


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("T", [3, 40, 200])
def test_unrouted_pairs(mx, act, T):
    """Pairs that no expert took: their rows of h stay as they were, nothing of
    them reaches the outputs, and a token without any gives zeros."""
    d = make(mx, T, 96, 64, 5, 2, act=act, seed=T)
    ids, w, _ = tables(d)
    gone = np.zeros((T, 2), dtype=bool)
    gone[::3, 0] = True
    gone[1] = True
    flat = np.where(gone, -1, ids).ravel()
    order = np.argsort(np.where(flat < 0, 99, flat), kind="stable")
    n = int((flat >= 0).sum())
    pos = np.full(2 * T, -1, dtype=np.int32)
    pos[order[:n]] = np.arange(n)
    sp = np.full(2 * T, -1, dtype=np.int32)
    sp[:n] = order[:n]
    off = np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=5))]).astype(np.int32)
    perm = {"offsets": off, "sorted_pair": sp, "pair_pos": pos}
    B = d["B"]
    B.h.fill_(3.0)
    h = mx.gateup_silu(d["bank"], d["x"], torch.from_numpy(off).to(DEV), torch.from_numpy(sp).to(DEV), B)
    check_h(d, h, perm)
    assert (h[n:] == 3.0).all()
    h[n:] = float("nan")
    w32 = torch.from_numpy(w.astype(np.float32)).to(DEV)
    out = mx.down_combine(d["bank"], h, w32, torch.from_numpy(off).to(DEV), torch.from_numpy(pos).to(DEV), B)
    assert (out[1] == 0).all()
    hz = h.clone()
    hz[n:] = 0
    check_out(d, out, hz, perm, f64(w32), np.ones((T, 0)))


@pytest.mark.parametrize("T", [6, 80])
def test_experts_without_rows_and_with_all(mx, T):
    d = make(mx, T, 128, 64, 9, 1, seed=4)
    logits = torch.full((T, 9), -5.0, device=DEV)
    logits[:, 8] = 1.0
    d["logits"] = logits
    out = mx.run_layer(d["bank"], d["x"], logits, d["B"])
    ids, w, perm = tables(d)
    assert (ids == 8).all()
    check_h(d, d["B"].h, perm)
    check_out(d, out, d["B"].h, perm, f64(d["B"].w), np.ones((T, 0)))


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("T", [4, 50, 160])
def test_nan_and_inf_stay_in_their_token(mx, act, T):
    d = make(mx, T, 160, 64, 3, 2, 1, 64, act=act, seed=8)
    d["x"][1, 37] = float("nan")
    d["x"][3, 5] = float("inf")
    out = f64(mx.run_layer(d["bank"], d["x"], d["logits"], d["B"], shared_gate=d["gate"]))
    bad = np.zeros(T, dtype=bool)
    bad[[1, 3]] = True
    assert np.isfinite(out[~bad]).all()
    assert np.isnan(out[1]).all()
    assert np.isnan(out[3]).all() if act == "a4" else not np.isfinite(out[3]).any()
    x0 = d["x"].clone()
    x0[1] = x0[3] = 0
    keep = mx.run_layer(d["bank"], x0, d["logits"], d["B"], shared_gate=d["gate"])
    assert np.array_equal(f64(keep)[~bad], out[~bad])


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("T", [2, 40, 300])
def test_marked_weight_block_makes_nan(mx, act, T):
    """A weight block with scale 255 is NaN in its unit and nowhere else."""
    d = make(mx, T, 128, 64, 2, 1, act=act, seed=3)
    codes, scales = d["w13"]
    scales[1, 5, 2] = 255                          # expert 1, gate row 5
    d["bank"] = mx.MxBank((codes, scales))
    ids, w, perm = tables(d)
    h = f64(mx.gateup_silu(d["bank"], d["x"], torch.from_numpy(perm["offsets"]).to(DEV),
                           torch.from_numpy(perm["sorted_pair"]).to(DEV), d["B"]))
    lo = perm["offsets"][1]
    want = np.zeros(h.shape, dtype=bool)
    want[lo:, 5] = True
    assert np.array_equal(np.isnan(h), want)


@pytest.mark.parametrize("act", ["a16", "a4"])
def test_wide_range_of_scales(mx, act):
    """Weights and activations whose block scales span 2^-60..2^60."""
    T, H, I, E = 20, 256, 64, 3
    rng = np.random.default_rng(12)
    d = make(mx, T, H, I, E, 1, act=act, seed=12)
    w = rng.standard_normal((E, 2 * I, H)) * np.exp2(rng.integers(-30, 30, (E, 2 * I, 1)))
    codes, scales = O.quantise(w.astype(np.float32))
    d["v13"] = O.values(codes, scales)
    d["bank"] = mx.MxBank((torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV)))
    d["x"] = (d["x"].float() * torch.exp2(torch.from_numpy(rng.integers(-30, 30, (T, 1))).to(DEV))).bfloat16()
    ids, w_, perm = tables(d)
    h = mx.gateup_silu(d["bank"], d["x"], torch.from_numpy(perm["offsets"]).to(DEV),
                       torch.from_numpy(perm["sorted_pair"]).to(DEV), d["B"])
    check_h(d, h, perm)


def test_bank_past_32_bit_offsets(mx):
    """Codes of 5 GB: the last experts are read where they lie."""
    T, H, I, E = 3, 4096, 4096, 300
    rng = np.random.default_rng(1)
    codes = torch.zeros((E, 2 * I, H // 2), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((E, 2 * I, H // 32), dtype=torch.uint8, device=DEV)
    d = {"dims": (T, H, I, E, 1, 0, 0), "act": "a16", "v13": {}}
    for e in (255, 256, 299):
        c, s = O.quantise((rng.standard_normal((2 * I, H)) * 0.02).astype(np.float32))
        codes[e], scales[e] = torch.from_numpy(c).to(DEV), torch.from_numpy(s).to(DEV)
        d["v13"][e] = O.values(c, s)
    d["x"] = bf16_rows(rng, T, H).to(DEV)
    ids = np.array([[256], [299], [255]], dtype=np.int32)
    perm = oracle.permute(ids, E, 16)
    B = mx.MxBuffers(T, H, I, E, 1, device=DEV)
    h = mx.gateup_silu(mx.MxBank((codes, scales)), d["x"], torch.from_numpy(perm["offsets"]).to(DEV),
                       torch.from_numpy(perm["sorted_pair"]).to(DEV), B)
    check_h(d, h, perm)
    del codes, scales
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# streams, graphs, repeats


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("T", [1, 12, 64, 256])
def test_repeats_and_streams_are_bit_identical(mx, act, T):
    shape = (T, 512, 256, 16, 4, 1, 256)
    d = make(mx, *shape, act=act, seed=T)
    ref = mx.run_layer(d["bank"], d["x"], d["logits"], d["B"], shared_gate=d["gate"]).clone()
    for _ in range(3):
        d["B"].ws.fill_(0)
        again = mx.run_layer(d["bank"], d["x"], d["logits"], d["B"], shared_gate=d["gate"])
        assert torch.equal(again, ref)
    # two streams at once, buffers each
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    bufs = [mx.MxBuffers(*shape, act=act, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        mx.run_layer(d["bank"], d["x"], d["logits"], bufs[0], shared_gate=d["gate"], stream=streams[0])
        with torch.cuda.stream(streams[1]):
            mx.run_layer(d["bank"], d["x"], d["logits"], bufs[1], shared_gate=d["gate"])
    torch.cuda.synchronize()
    assert torch.equal(bufs[0].out, ref) and torch.equal(bufs[1].out, ref)


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("T", [1, 12, 200])
def test_graph_replays_match_eager(mx, act, T):
    shape = (T, 512, 256, 16, 4, 1, 256)
    d = make(mx, *shape, act=act, seed=T + 50)
    B = d["B"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mx.run_layer(d["bank"], d["x"], d["logits"], B, shared_gate=d["gate"])
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.run_layer(d["bank"], d["x"], d["logits"], B, shared_gate=d["gate"])
        codes, scales = mx.quantize_rows(B.out)
    eager = mx.MxBuffers(*shape, act=act, device=DEV)
    rng = np.random.default_rng(T)
    for step in range(4):
        d["x"].copy_(bf16_rows(rng, T, shape[1]))
        d["logits"].copy_(torch.from_numpy(rng.standard_normal((T, shape[3])).astype(np.float32)))
        want = mx.run_layer(d["bank"], d["x"], d["logits"], eager, shared_gate=d["gate"])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(B.out, want) and torch.equal(B.ids, eager.ids), step
        wc, wsc = mx.quantize_rows(want)
        assert torch.equal(codes, wc) and torch.equal(scales, wsc)


def test_quantised_layer_end_to_end(mx):
    """fp32 weights to a bank by the library, a layer on it, against the oracle's own bank."""
    T, H, I, E, k = 21, 256, 96, 6, 2
    rng = np.random.default_rng(2)
    w13 = (rng.standard_normal((E, 2 * I, H)) * 0.05).astype(np.float32)
    w2 = (rng.standard_normal((E, H, I)) * 0.05).astype(np.float32)
    bank = mx.MxBank(mx.quantize_bank(torch.from_numpy(w13).to(DEV)), mx.quantize_bank(torch.from_numpy(w2).to(DEV)))
    d = make(mx, T, H, I, E, k, seed=2)
    d["bank"], d["v13"], d["v2"] = bank, O.values(*O.quantise(w13)), O.values(*O.quantise(w2))
    out = mx.run_layer(bank, d["x"], d["logits"], d["B"])
    ids, w, perm = tables(d)
    check_h(d, d["B"].h, perm)
    check_out(d, out, d["B"].h, perm, f64(d["B"].w), np.ones((T, 0)))


# ---------------------------------------------------------------------------
# many rows: tiles of up to 160

LARGE = [
    # T, H, I, E, k, n_shared, I_shared
    (507, 2080, 352, 20, 3, 1, 224),     # padded rows, shared experts of their own length
    (320, 2048, 512, 24, 4, 0, 0),       # whole steps of K
    (1210, 64, 2080, 60, 2, 0, 0),       # K of half a piece; one block of columns in down
    (1030, 1024, 256, 150, 5, 0, 0),     # more than 128 experts
    (2500, 1056, 416, 3, 2, 2, 32),      # many tiles an expert
]
MANY = (640, 1056, 416, 24, 4, 1, 416)


def on_large_tiles(shape, act):
    """The library's rule, so that a shape that it no longer sends there is noticed."""
    T, H, I, E, k = shape[:5]
    P = T * k
    tiles = P // 160 + min(E, P) // 2
    gu, dn = -(-I // 128) * -(-H // 128), -(-H // 256) * -(-I // 128)
    rows = P >= 16 * E if act == "a4" else P * gu >= 24576 and P * dn >= 40960
    return tiles * min(gu, dn) >= 500 and rows


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_many_rows(mx, shape, act):
    assert on_large_tiles(shape, act)
    test_layer(mx, shape, act)


@pytest.mark.parametrize("act", ["a16", "a4"])
def test_many_rows_with_unrouted_pairs(mx, act):
    """Pairs that no expert took: their rows of h stay as they were, nothing of
    them reaches the outputs, and a token without any gives zeros."""
    T, H, I, E, k = MANY[:5]
    assert on_large_tiles(MANY, act)
    d = make(mx, T, H, I, E, k, act=act, seed=31)
    ids, w, _ = tables(d)
    gone = np.zeros((T, k), dtype=bool)
    gone[::3, 1] = True
    gone[1] = True
    flat = np.where(gone, -1, ids).ravel()
    order = np.argsort(np.where(flat < 0, 999, flat), kind="stable")
    n = int((flat >= 0).sum())
    pos = np.full(k * T, -1, dtype=np.int32)
    pos[order[:n]] = np.arange(n)
    sp = np.full(k * T, -1, dtype=np.int32)
    sp[:n] = order[:n]
    off = np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=E))]).astype(np.int32)
    perm = {"offsets": off, "sorted_pair": sp, "pair_pos": pos}
    B = d["B"]
    B.h.fill_(3.0)
    h = mx.gateup_silu(d["bank"], d["x"], torch.from_numpy(off).to(DEV), torch.from_numpy(sp).to(DEV), B)
    check_h(d, h, perm)
    assert (h[n:] == 3.0).all()
    h[n:] = float("nan")
    w32 = torch.from_numpy(w.astype(np.float32)).to(DEV)
    out = mx.down_combine(d["bank"], h, w32, torch.from_numpy(off).to(DEV), torch.from_numpy(pos).to(DEV), B)
    assert (out[1] == 0).all()
    hz = h.clone()
    hz[n:] = 0
    check_out(d, out, hz, perm, f64(w32), np.ones((T, 0)))


@pytest.mark.parametrize("act", ["a16", "a4"])
def test_many_rows_nan_and_inf_stay_in_their_token(mx, act):
    assert on_large_tiles(MANY, act)
    d = make(mx, *MANY, act=act, seed=8)
    d["x"][1, 37] = float("nan")
    d["x"][3, 5] = float("inf")
    out = f64(mx.run_layer(d["bank"], d["x"], d["logits"], d["B"], shared_gate=d["gate"]))
    bad = np.zeros(MANY[0], dtype=bool)
    bad[[1, 3]] = True
    assert np.isfinite(out[~bad]).all()
    assert np.isnan(out[1]).all()
    assert np.isnan(out[3]).all() if act == "a4" else not np.isfinite(out[3]).any()
    x0 = d["x"].clone()
    x0[1] = x0[3] = 0
    keep = mx.run_layer(d["bank"], x0, d["logits"], d["B"], shared_gate=d["gate"])
    assert np.array_equal(f64(keep)[~bad], out[~bad])


@pytest.mark.parametrize("act", ["a16", "a4"])
def test_many_rows_marked_weight_block_makes_nan(mx, act):
    T, H, I, E, k = MANY[:5]
    d = make(mx, T, H, I, E, k, act=act, seed=3)
    codes, scales = d["w13"]
    scales[1, 5, 2] = 255                          # expert 1, gate row 5
    scales[2, I + 33, H // 32 - 1] = 255           # expert 2, up row 33, the last block
    d["bank"] = mx.MxBank((codes, scales))
    ids, w, perm = tables(d)
    h = f64(mx.gateup_silu(d["bank"], d["x"], torch.from_numpy(perm["offsets"]).to(DEV),
                           torch.from_numpy(perm["sorted_pair"]).to(DEV), d["B"]))
    off = perm["offsets"]
    want = np.zeros(h.shape, dtype=bool)
    want[off[1]:off[2], 5] = True
    want[off[2]:off[3], 33] = True
    assert np.array_equal(np.isnan(h), want)


@pytest.mark.parametrize("act", ["a16", "a4"])
def test_many_rows_repeat_and_replay_bit_identical(mx, act):
    d = make(mx, *MANY, act=act, seed=77)
    B = d["B"]
    ref = mx.run_layer(d["bank"], d["x"], d["logits"], B, shared_gate=d["gate"]).clone()
    for fill in (0, 255):
        B.ws.fill_(fill)
        assert torch.equal(mx.run_layer(d["bank"], d["x"], d["logits"], B, shared_gate=d["gate"]), ref)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.run_layer(d["bank"], d["x"], d["logits"], B, shared_gate=d["gate"])
    eager = mx.MxBuffers(*MANY, act=act, device=DEV)
    rng = np.random.default_rng(6)
    for step in range(3):
        d["x"].copy_(bf16_rows(rng, MANY[0], MANY[1]))
        d["logits"].copy_(torch.from_numpy(rng.standard_normal((MANY[0], MANY[3])).astype(np.float32)))
        want = mx.run_layer(d["bank"], d["x"], d["logits"], eager, shared_gate=d["gate"])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(B.out, want), step


# ---------------------------------------------------------------------------
# a few tokens: routing in the gate/up launch


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 512, 64), (2, 130, 32), (3, 65, 20), (3, 64, 21), (2, 5, 5)])
def test_few_tokens_route_as_the_routing_calls(mx, act, T, E, k):
    """The tables and weights of the routed launch are those of the framework's
    routing and sort, ties, infinities and NaN among the logits too."""
    d = make(mx, T, 64, 32, E, k, act=act, seed=E + k)
    B = d["B"]
    rng = np.random.default_rng(E)
    for kind in ("plain", "ties", "special"):
        lg = rng.standard_normal((T, E)).astype(np.float32)
        if kind == "ties":
            lg = np.round(lg)
        if kind == "special" and E > 4:
            lg[0, 0], lg[0, E // 2], lg[T - 1, E - 1] = -np.inf, -np.inf, -3e38
        logits = torch.from_numpy(lg).to(DEV)
        for renorm in (0, 1):
            out = mx.run_layer(d["bank"], d["x"], logits, B, renormalize=renorm)
            ids, w = oracle.route_topk(lg, k, renorm)
            perm = oracle.permute(ids, E, 16)
            assert np.array_equal(B.ids.cpu().numpy(), ids), kind
            for name in ("counts", "offsets", "sorted_pair", "pair_pos"):
                assert np.array_equal(getattr(B, name).cpu().numpy(), perm[name]), (kind, name)
            # logit - max below 16 in size is rounded by at most 8 eps, which the
            # exponential turns into 8 eps relative, and adds 2 of its own; the
            # sum has the same and 14 additions (8 per lane, 6 over lanes), the
            # quotient one: 8 + 2 + 8 + 2 + 14 + 1 = 35 (-inf and -3e38 give 0)
            assert (np.abs(f64(B.w) - w) <= 40 * O.EPS32 * w).all()
            check_h(d, B.h, perm)
            check_out(d, out, B.h, perm, f64(B.w), np.ones((T, 0)))


@pytest.mark.parametrize("T,E,k", [(1, 128, 8), (3, 130, 5), (2, 20, 20)])
def test_few_tokens_route_nan_logits_as_the_routing_calls(mx, T, E, k):
    """NaN logits have no order of their own: the routed launch takes the one
    that moe_route_topk and moe_permute take, and gives the same bits."""
    from packed_bit_grouped_amd import _lib as L
    d = make(mx, T, 64, 32, E, k, seed=E)
    B = d["B"]
    rng = np.random.default_rng(7)
    for vals in ((np.nan,), (-np.nan, np.inf), (np.nan, -np.inf, np.inf, -0.0, 0.0)):
        lg = rng.standard_normal((T, E)).astype(np.float32)
        for i, v in enumerate(vals):
            lg[i % T, 3 * i], lg[(i + 1) % T, E - 1 - i] = v, -v
        logits = torch.from_numpy(lg).to(DEV)
        for renorm in (0, 1):
            mx.run_layer(d["bank"], d["x"], logits, B, renormalize=renorm)
            i32 = dict(dtype=torch.int32, device=DEV)
            ids, w = torch.empty((T, k), **i32), torch.empty((T, k), device=DEV)
            n = L.load().moe_permute_max_tiles(T, k, E, 16)
            t = [torch.empty(m, **i32) for m in (E, E + 1, T * k, T * k, 4 * n, 1)]
            L.moe_route_topk(logits, T, E, k, renorm, ids, w)
            L.moe_permute(ids, T, k, E, 16, *t)
            assert torch.equal(B.ids, ids)
            assert torch.equal(B.w.view(torch.int32), w.view(torch.int32))
            for got, want in zip((B.counts, B.offsets, B.sorted_pair, B.pair_pos), t):
                assert torch.equal(got, want)


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("shape", [
    (80, 40960, 128, 4, 1, 0, 0),    # rows whose scales do not fit beside a tile
    (2, 49152, 32, 2, 1, 0, 0),      # tokens too long to be staged while they are routed
    (5, 64, 32, 512, 40, 0, 0),      # every expert a lane can hold
    (1, 64, 32, 128, 100, 1, 32),    # more pairs than the routed launch takes
    (33, 32, 4096, 2, 2, 3, 32),     # shared experts shorter than the routed ones
], ids=str)
def test_far_sizes(mx, shape, act):
    test_layer(mx, shape, act)


def test_a_pair_without_a_place_adds_nothing(mx):
    T, H, I, E, k = 6, 64, 32, 4, 2
    d = make(mx, T, H, I, E, k, seed=5)
    ids, w, perm = tables(d)
    B = d["B"]
    h = bf16_rows(np.random.default_rng(1), B.R, B.ld_h).to(DEV)
    w32 = torch.from_numpy(w.astype(np.float32)).to(DEV)
    off = torch.from_numpy(perm["offsets"]).to(DEV)
    pos = perm["pair_pos"].copy()
    pos[3] = -1
    want = mx.down_combine(d["bank"], h, w32, off, torch.from_numpy(pos).to(DEV), B).clone()
    check_out(d, want, h, dict(perm, pair_pos=pos), f64(w32), np.ones((T, 0)))


# fewer rows an expert, A4: two workgroups share a compute unit
FEWER = (560, 1056, 416, 24, 4, 1, 416)


@pytest.mark.parametrize("check", [
    test_many_rows_with_unrouted_pairs, test_many_rows_nan_and_inf_stay_in_their_token,
    test_many_rows_marked_weight_block_makes_nan, test_many_rows_repeat_and_replay_bit_identical,
], ids=lambda f: f.__name__[15:])
def test_fewer_rows(mx, monkeypatch, check):
    T, H, I, E, k = FEWER[:5]
    assert on_large_tiles(FEWER, "a4") and T * k <= 96 * E < MANY[0] * MANY[4]
    monkeypatch.setitem(globals(), "MANY", FEWER)
    check(mx, "a4")


@pytest.mark.parametrize("shape", [
    (400, 6144, 128, 24, 1, 0, 0),     # rows too long for two workgroups' LDS
    (1150, 4608, 160, 12, 1, 1, 96),   # the longest that fit
    (2000, 512, 2304, 12, 1, 0, 0),    # more rows an expert than the rule takes
], ids=str)
def test_rows_on_either_side_of_the_two_workgroup_rule(mx, shape):
    test_layer(mx, shape, "a4")
