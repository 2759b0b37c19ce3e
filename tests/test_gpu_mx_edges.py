"""The MXFP4 operators where their other tests do not go: calls on another
stream than the current one, SiLU far below zero, scale bytes next to the
ends, shared experts longer than the routed ones."""
import numpy as np
import pytest

import oracle
from oracle import mx_oracle as O
from packed_bit_grouped_amd import _lib as L

torch = pytest.importorskip("torch")
import test_gpu_mx as G  # noqa: E402
from test_gpu_mx import DEV, bf16_rows, check_h, f64, make, mx, tables  # noqa: E402,F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# another stream than the current one: the other one is held up where the call's
# own work has to be in order, the current one where it must not matter

HOLD = 50_000_000     # clock ticks of a spinning kernel: tens of milliseconds


def hold(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(HOLD)


def other_stream(kind):
    """(a side stream that has seen the work queued so far, the argument for it)"""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    return s, (s if kind == "stream" else s.cuda_stream)


@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_transposed_bank_is_copied_on_the_call_s_stream(mx, kind):
    """The copy that quantize_bank makes of matrices that are not contiguous is
    in front of the quantiser, whatever the current stream is busy with, and
    its memory is not given away while the quantiser reads it."""
    w = torch.randn((3, 128, 96), generator=torch.Generator(DEV).manual_seed(1), device=DEV)
    want = mx.quantize_bank(w.transpose(1, 2))
    torch.cuda.synchronize()
    s, arg = other_stream(kind)
    hold(torch.cuda.current_stream())     # a copy queued here would come late
    got = mx.quantize_bank(w.transpose(1, 2), stream=arg)
    s.synchronize()
    with torch.cuda.stream(s):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    torch.cuda.synchronize()
    hold(s)                               # the copy's memory has to last
    got = mx.quantize_bank(w.transpose(1, 2), stream=arg)
    noise = [torch.full((3 * 96, 128), 7.0, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del noise


@pytest.mark.parametrize("kind", ["stream", "handle"])
@pytest.mark.parametrize("made_on", ["current", "other"])
def test_pairs_may_be_dropped_behind_the_bank(mx, made_on, kind):
    w = torch.randn((4, 64, 256), generator=torch.Generator(DEV).manual_seed(2), device=DEV)
    want = mx.MxBank(mx.quantize_bank(w)).tiles["w13"]
    torch.cuda.synchronize()
    if made_on == "current":
        pair = mx.quantize_bank(w)
        s, arg = other_stream(kind)
        hold(s)
        bank = mx.MxBank(pair, stream=arg)
        shapes = [t.shape for t in pair]
        del pair
    else:
        s, arg = other_stream(kind)
        hold(s)
        bank = mx.MxBank(mx.quantize_bank(w, stream=arg), stream=arg)
        shapes = [(4, 64, 128), (4, 64, 8)]
    noise = [torch.full(sh, 255, dtype=torch.uint8, device=DEV) for sh in shapes for _ in range(4)]
    torch.cuda.synchronize()
    for got, ref in zip(bank.tiles["w13"], want):
        assert torch.equal(got, ref)
    del noise


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_may_be_dropped_behind_the_call(mx, dtype):
    src = bf16_rows(np.random.default_rng(3), 96, 512).to(DEV).to(dtype)
    want_c, want_s = O.quantise(f64(src))
    want_v = torch.from_numpy(O.values(want_c, want_s)).float()
    torch.cuda.synchronize()
    s, arg = other_stream("stream")
    hold(s)
    codes, scales = mx.quantize_rows(src.clone(), stream=arg)
    noise = [torch.full_like(src, 9.0) for _ in range(4)]
    torch.cuda.synchronize()
    c2, s2 = codes.clone(), scales.clone()
    s.wait_stream(torch.cuda.current_stream())
    hold(s)
    back = mx.dequantize_rows(c2, s2, dtype, stream=arg)
    del c2, s2
    noise += [torch.full_like(t, 255) for t in (codes, scales) for _ in range(4)]
    torch.cuda.synchronize()
    assert np.array_equal(codes.cpu().numpy(), want_c) and np.array_equal(scales.cpu().numpy(), want_s)
    assert torch.equal(back.cpu().float(), want_v)
    del noise


@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_results_do_not_lie_where_the_current_stream_still_writes(mx, kind):
    """Memory that was freed on the current stream behind queued work may be
    handed out there again at once, not to a call on another stream."""
    src = bf16_rows(np.random.default_rng(4), 64, 512).to(DEV)
    w = src.float().view(2, 32, 512)
    codes, scales = mx.quantize_rows(src)
    back = mx.dequantize_rows(codes, scales)
    tiles = mx.MxBank(mx.quantize_bank(w)).tiles["w13"]
    torch.cuda.synchronize()
    s, arg = other_stream(kind)
    hold(torch.cuda.current_stream())
    for t in (codes, scales, back, *tiles):      # written late, given back at once
        for _ in range(2):
            junk = torch.full_like(t, 77)
            del junk
    c2, s2 = mx.quantize_rows(src, stream=arg)
    b2 = mx.dequantize_rows(c2, s2, stream=arg)
    t2 = mx.MxBank(mx.quantize_bank(w, stream=arg), stream=arg).tiles["w13"]
    torch.cuda.synchronize()
    for got, ref in zip((c2, s2, b2, *t2), (codes, scales, back, *tiles)):
        assert torch.equal(got, ref)


def test_default_stream_as_a_handle(mx):
    """Handle 0 is the default stream."""
    w = torch.randn((2, 64, 48), generator=torch.Generator(DEV).manual_seed(5), device=DEV)
    want = mx.quantize_bank(w.transpose(1, 2))
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = mx.quantize_bank(w.transpose(1, 2), stream=0)
        tiles = mx.MxBank(got, stream=0).tiles["w13"]
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for a, b in zip(tiles, mx.MxBank(want).tiles["w13"]):
        assert torch.equal(a, b)


def test_stream_of_another_device_is_refused(mx):
    class StreamOfDevice1:
        device_index, cuda_stream = 1, 0
    s = StreamOfDevice1()
    d = make(mx, 2, 64, 32, 2, 1)
    B, w = d["B"], torch.zeros((1, 32, 64), device=DEV)
    codes, scales = mx.quantize_rows(w[0])
    for call in (lambda: mx.quantize_rows(w[0], stream=s), lambda: mx.dequantize_rows(codes, scales, stream=s),
                 lambda: mx.quantize_bank(w, stream=s), lambda: mx.MxBank(mx.quantize_bank(w), stream=s),
                 lambda: mx.run_layer(d["bank"], d["x"], d["logits"], B, stream=s),
                 lambda: mx.gateup_silu(d["bank"], d["x"], B.offsets, B.sorted_pair, B, stream=s),
                 lambda: mx.down_combine(d["bank"], B.h, B.w, B.offsets, B.pair_pos, B, stream=s)):
        with pytest.raises(ValueError, match="device 1"):
            call()


# ---------------------------------------------------------------------------
# the ends of the ranges

# One expert, 16-row tiles; four experts, tiles of up to 160 rows.
FEW_ROWS, MANY_ROWS = (80, 64, 32, 1), (2560, 2048, 256, 4)


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("dims", [FEW_ROWS, MANY_ROWS], ids=["few", "many"])
def test_silu_far_below_zero(mx, dims, act):
    """h = SiLU(g) * u where SiLU(g) is below fp32's smallest number and u
    brings the product back: one weight of 1 each for g and u, so that both
    are exact."""
    T, H, I, E = dims
    w = np.zeros((E, 2 * I, H))
    w[:, :I, 0] = 1.0
    w[:, I:, 32] = 1.0
    codes, scales = O.quantise(w)
    bank = mx.MxBank((torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV)))
    if act == "a4":   # a code and a scale hold these exactly
        g = -np.array([0.5, 4, 12, 48, 64, 96, 128, 192, 256])
    else:
        g = -np.array([0.5, 4, 12, 48, 63.5, 64.5, 80, 86, 87.5, 88, 89, 104, 128, 160, 176, 182, 186])
    u = 2.0 ** np.array([0, 20, 90, 126])
    pairs = np.array([(a, b) for a in g for b in u])
    x = np.zeros((T, H), dtype=np.float32)
    x[:, [0, 32]] = pairs[np.arange(T) % len(pairs)]
    B = mx.MxBuffers(T, H, I, E, 1, act=act, device=DEV)
    ids = (np.arange(T) % E).astype(np.int32)[:, None]
    perm = oracle.permute(ids, E, 16)
    xt = torch.from_numpy(x).bfloat16().to(DEV)
    h = f64(mx.gateup_silu(bank, xt, torch.from_numpy(perm["offsets"]).to(DEV),
                           torch.from_numpy(perm["sorted_pair"]).to(DEV), B))
    xv = O.activations(f64(xt), act)[perm["sorted_pair"]]
    gv, uv = xv[:, 0], xv[:, 32]
    want = gv / (1 + np.exp(-gv)) * uv
    # the exponential's argument is rounded by |g| * 1.45 half units, which it
    # turns into |g| units of relative error at most; with a factor below 2^-126
    # that fp32 holds in steps of 2^-149 (e^(g/2) >= e^-93.5 = 2^-134.9: 2^-15);
    # a few units for the products; then half a step of bf16 and its smallest step
    rel = (2 * np.abs(gv) + 16) * O.EPS32 + 2.0 ** -14
    bound = (rel + 2.0 ** -8 * (1 + rel)) * np.abs(want) + 2.0 ** -133
    assert (np.abs(h - want[:, None]) <= bound[:, None]).all(), sorted(
        {(float(a), float(b)) for a, b, bad in zip(gv, uv, (np.abs(h - want[:, None]) > bound[:, None]).any(1)) if bad})


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("dims", [(20, 256, 64, 3), (2560, 2048, 256, 4)], ids=["few", "many"])
@pytest.mark.parametrize("byte,unit", [(1, 122), (2, 121), (250, -124), (251, -125)])
def test_scale_bytes_next_to_the_ends(mx, dims, act, byte, unit):
    """Weights of one scale byte next to the smallest or the largest, every
    code among them, with x of the size that brings the sums back to order 1."""
    T, H, I, E = dims
    rng = np.random.default_rng(byte)
    d = make(mx, T, H, I, E, 1, act=act, seed=byte)
    codes = rng.integers(0, 256, (E, 2 * I, H // 2), dtype=np.uint8)
    scales = np.full((E, 2 * I, H // 32), byte, dtype=np.uint8)
    d["v13"] = O.values(codes, scales)
    d["bank"] = mx.MxBank((torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV)))
    x = np.ldexp(rng.standard_normal((T, H)) / np.sqrt(H), unit)
    d["x"] = torch.from_numpy(x.astype(np.float32)).bfloat16().to(DEV)
    ids, w, perm = tables(d)
    h = mx.gateup_silu(d["bank"], d["x"], torch.from_numpy(perm["offsets"]).to(DEV),
                       torch.from_numpy(perm["sorted_pair"]).to(DEV), d["B"])
    assert np.abs(f64(h)).max() > 0.1
    check_h(d, h, perm)


# ---------------------------------------------------------------------------
# shared experts longer than the routed ones, on large tiles

# T, H, I, E, k, n_shared, I_shared: whole steps of K and not, with more rows an
# expert than A4's kernel with two workgroups per compute unit takes, and with fewer
LONG_WIDE = [(1300, 4096, 256, 24, 2, 1, 768), (1300, 2080, 160, 24, 2, 2, 416)]
LONG_NARROW = [(1300, 2048, 256, 48, 2, 1, 768), (1300, 2080, 224, 40, 2, 1, 512),
               (1300, 2080, 256, 48, 2, 1, 352)]


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("shape", LONG_WIDE + LONG_NARROW, ids=str)
def test_long_shared_experts_on_large_tiles(mx, shape, act):
    """The layer and its parts; the columns of h past a routed row's own are
    not read, whatever they hold, and not written."""
    T, H, I, E, k, n_sh, I_sh = shape
    for down in (0, 1):
        assert L.moe_mx4_tile_rows(mx.ACTS[act], *shape, down) > 16
    G.test_layer(mx, shape, act)
    d = make(mx, *shape, act=act, seed=1)
    B = d["B"]
    want = mx.run_layer(d["bank"], d["x"], d["logits"], B, shared_gate=d["gate"]).clone()
    assert (B.h[:T * k, I:] == 0).all()
    B.h.fill_(float("nan"))
    assert torch.equal(mx.run_layer(d["bank"], d["x"], d["logits"], B, shared_gate=d["gate"]), want)
    assert torch.isnan(B.h[:T * k, I:]).all() and torch.isfinite(B.h[:T * k, :I]).all()
    assert torch.isfinite(B.h[T * k:]).all()


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("T", [2, 33])
@pytest.mark.parametrize("I,I_sh", [(96, 224), (224, 96)])
def test_columns_past_a_row_s_own_are_not_read(mx, T, I, I_sh, act):
    """The same on 16 rows, the shared experts' columns too."""
    d = make(mx, T, 288, I, 6, 2, 1, I_sh, act=act, seed=T)
    B = d["B"]
    want = mx.run_layer(d["bank"], d["x"], d["logits"], B, shared_gate=d["gate"]).clone()
    B.h.fill_(float("nan"))
    assert torch.equal(mx.run_layer(d["bank"], d["x"], d["logits"], B, shared_gate=d["gate"]), want)
    P = 2 * T
    assert torch.isfinite(B.h[:P, :I]).all() and torch.isnan(B.h[:P, I:]).all()
    assert torch.isfinite(B.h[P:, :I_sh]).all() and torch.isnan(B.h[P:, I_sh:]).all()


def test_calls_on_a_stream_of_their_own_are_captured(mx):
    """The copy and the memory that the calls make belong to the captured
    stream, given as such or as the current one; replays give the eager bits."""
    w = torch.empty((2, 64, 96), device=DEV)

    def calls(stream):
        codes, scales = mx.quantize_bank(w.transpose(1, 2), stream=stream)
        tiles = mx.MxBank((codes, scales), stream=stream).tiles["w13"]
        rows = mx.dequantize_rows(codes.view(-1, 32), scales.view(-1, 2), stream=stream)
        return codes, scales, *tiles, rows

    w.copy_(torch.randn(w.shape, generator=torch.Generator(DEV).manual_seed(0), device=DEV))
    calls(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = torch.cuda.current_stream()
        got = [calls(s), calls(s.cuda_stream), calls(None)]
    for seed in range(3):
        w.copy_(torch.randn(w.shape, generator=torch.Generator(DEV).manual_seed(seed + 1), device=DEV))
        want = calls(None)
        graph.replay()
        torch.cuda.synchronize()
        for outs in got:
            for a, b in zip(outs, want):
                assert torch.equal(a, b), seed


# ---------------------------------------------------------------------------
# the most tokens, choices and units


@pytest.mark.parametrize("act", ["a16", "a4"])
@pytest.mark.parametrize("shape", [
    (65535, 32, 32, 4, 1, 0, 0),      # tokens
    (9, 32, 32, 512, 512, 0, 0),      # choices: more pairs than one routing launch takes
    (1, 64, 32, 512, 512, 1, 64),
    (300, 32, 32768, 2, 1, 0, 0),     # units: a single step of K on large tiles, and a long K behind it
    (2, 32, 65536, 2, 1, 1, 32),
], ids=str)
def test_largest_of_each(mx, shape, act):
    G.test_layer(mx, shape, act)

