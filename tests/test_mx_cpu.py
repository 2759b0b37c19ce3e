"""MXFP4 without a GPU: the oracle's format against hand-worked values and a
search over all codes, and the C ABI's refusals (nothing is launched)."""
import ctypes

import numpy as np
import pytest

from oracle import mx_oracle as O
from packed_bit_grouped_amd import _lib as L

FAKE = 1 << 20


def test_hand_worked_block():
    # largest magnitude 6 = 1.5 * 2^2: scale 2^0; ties to the even mantissa
    v = np.zeros(32)
    v[:14] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -5, 0.26, 4.99, -6]
    codes, scales = O.quantise(v[None])
    assert scales[0, 0] == 127
    assert O.values(codes, scales)[0, :14].tolist() == [
        6, 0, 1, 1, 2, 2, 4, 4, -0.0, -1, -4, 0.5, 4, -6]
    # even index in the low nibble: 6 is code 7, 0.25 code 0; -0.25 code 8, -0.75 code 10
    assert codes[0, 0] == 0x07 and codes[0, 4] == 0xA8


@pytest.mark.parametrize("a,byte", [(0.0, 0), (1.0, 125), (7.99, 127), (8.0, 128), (2.0 ** -149, 0),
                                    (2.0 ** -125, 0), (2.0 ** -124, 1), (3.3e38, 252),
                                    (np.inf, 255), (np.nan, 255)])
def test_scale_of_largest_magnitude(a, byte):
    v = np.zeros(32)
    v[5] = -a
    codes, scales = O.quantise(v[None])
    assert scales[0, 0] == byte
    if byte == 255:
        assert not codes.any() and np.isnan(O.values(codes, scales)).all()


def test_quantise_is_nearest_of_all_codes():
    rng = np.random.default_rng(3)
    v = (rng.standard_normal((64, 96)) * np.exp(rng.standard_normal((64, 1)) * 8)).astype(np.float32)
    codes, scales = O.quantise(v)
    got = O.values(codes, scales)
    unit = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, axis=1)
    grid = np.concatenate([O.GRID, -O.GRID])
    best = np.abs(v[..., None] - grid * unit[..., None]).min(-1)
    assert np.array_equal(np.abs(v - got), best)
    a = np.abs(v).reshape(64, 3, 32).max(-1)
    u = unit[:, ::32]
    assert ((a >= 4 * u) & (a < 8 * u)).all()


def test_round_trip_of_every_code():
    nib = np.tile(np.arange(16, dtype=np.uint8), 2)[None]
    for s in (1, 100, 127, 250):
        v = O.values(O.pack(nib), np.array([[s]], dtype=np.uint8))
        c2, s2 = O.quantise(v)
        assert s2[0, 0] == s and np.array_equal(O.values(c2, s2), v)


def test_one_weight_layer_closed_form():
    # one nonzero weight in gate, up and down each: h = SiLU(2x) * 3x
    x = np.zeros((1, 32))
    x[0, 7] = 1.5
    w13 = np.zeros((64, 32))
    w13[0, 7], w13[32, 7] = 2.0, 3.0
    h, _ = O.gateup(O.activations(x, "a4"), w13, 32)
    assert h[0, 0] == pytest.approx(3.0 / (1 + np.exp(-3.0)) * 4.5, rel=1e-15)
    assert not h[0, 1:].any()


# ---------------------------------------------------------------------------
# refusals


def _quant(**kw):
    a = dict(src=FAKE, src_is_f32=0, R=4, C=64, ld=64, codes=FAKE, scales=FAKE)
    a.update(kw)
    return L.moe_mx4_quant_rows(*a.values(), stream=0, check=False)


def _dequant(**kw):
    a = dict(codes=FAKE, scales=FAKE, R=4, C=64, dst=FAKE, dst_is_f32=0, ld=64)
    a.update(kw)
    return L.moe_mx4_dequant_rows(*a.values(), stream=0, check=False)


@pytest.mark.parametrize("call,out", [(_quant, "codes"), (_dequant, "dst")])
def test_rows_refusals(call, out):
    kind = "src_is_f32" if call is _quant else "dst_is_f32"
    far = "src" if call is _quant else "dst"
    assert call(R=-1) == L.MOE_E_INVAL
    assert call(C=0) == L.MOE_E_INVAL
    assert call(ld=63) == L.MOE_E_INVAL
    assert call(C=48) == L.MOE_E_UNSUPPORTED
    assert call(**{kind: 2}) == L.MOE_E_INVAL
    for name in (out, "codes", "scales", far):
        assert call(**{name: None}) == L.MOE_E_INVAL, name
    assert call(codes=FAKE + 2) == L.MOE_E_INVAL
    assert call(**{far: FAKE + 1}) == L.MOE_E_INVAL
    assert call(**{kind: 1, far: FAKE + 2}) == L.MOE_E_INVAL
    assert call(R=0, codes=None, scales=None, **{far: None}) == L.MOE_OK


def _tile(**kw):
    a = dict(codes=FAKE, scales=FAKE, n=2, N=64, K=96, dst_codes=2 * FAKE, dst_scales=2 * FAKE)
    a.update(kw)
    return L.moe_mx4_tile_bank(*a.values(), stream=0, check=False)


def test_tile_refusals():
    for kw in (dict(n=-1), dict(N=0), dict(K=0), dict(codes=None), dict(scales=None),
               dict(dst_codes=None), dict(dst_scales=None), dict(dst_codes=FAKE),
               dict(dst_scales=FAKE), dict(codes=FAKE + 8), dict(dst_codes=2 * FAKE + 8),
               dict(dst_scales=2 * FAKE + 2)):
        assert _tile(**kw) == L.MOE_E_INVAL, kw
    for kw in (dict(N=40), dict(K=48)):
        assert _tile(**kw) == L.MOE_E_UNSUPPORTED, kw
    assert _tile(n=0) == L.MOE_OK
    assert L.moe_mx4_bank_code_bytes(2, 64, 96) == 2 * 4 * 1024
    assert L.moe_mx4_bank_scale_bytes(2, 64, 96) == 2 * 4 * 256
    assert L.moe_mx4_bank_code_bytes(3, 32, 2080) == 3 * 2 * 17 * 1024
    assert L.moe_mx4_bank_scale_bytes(3, 32, 2080) == 3 * 2 * 5 * 256
    for args in ((0, 64, 96), (2, 40, 96), (2, 64, 48), (2, -16, 96)):
        assert L.moe_mx4_bank_code_bytes(*args) == L.moe_mx4_bank_scale_bytes(*args) == 0


BANK = L.MxBankDesc(FAKE, FAKE)
SHAPE = dict(act=L.MOE_A16, T=4, H=256, I=128, E=8, k=2, n_shared=0, I_shared=0)


def _gateup(**kw):
    a = dict(act=L.MOE_A16, x=FAKE, T=4, H=256, I=128, E=8, k=2, w13=BANK, w13_shared=None,
             n_shared=0, I_shared=0, offsets=FAKE, sorted_pair=FAKE, h=FAKE, workspace=FAKE,
             ws_bytes=1 << 30, flags=0)
    a.update(kw)
    return L.moe_mx4_gateup_silu(*a.values(), stream=0, check=False)


def _down(**kw):
    a = dict(act=L.MOE_A16, h=FAKE, T=4, H=256, I=128, E=8, k=2, w2=BANK, w2_shared=None,
             n_shared=0, I_shared=0, topk_w=FAKE, offsets=FAKE, pair_pos=FAKE, out=FAKE,
             workspace=FAKE, ws_bytes=1 << 30, flags=0)
    a.update(kw)
    return L.moe_mx4_down_combine(*a.values(), stream=0, check=False)


def _layer(**kw):
    a = dict(act=L.MOE_A16, logits=FAKE, x=FAKE, T=4, H=256, I=128, E=8, k=2, renormalize=1,
             w13=BANK, w2=BANK, w13_shared=None, w2_shared=None, n_shared=0, I_shared=0,
             topk_ids=FAKE, topk_w=FAKE, counts=FAKE, offsets=FAKE, sorted_pair=FAKE,
             pair_pos=FAKE, h=FAKE, out=FAKE, workspace=FAKE, ws_bytes=1 << 30, flags=0)
    a.update(kw)
    return L.moe_mx4_layer(*a.values(), stream=0, check=False)


@pytest.mark.parametrize("call", [_gateup, _down, _layer])
def test_projection_refusals(call):
    inval = [dict(act=L.MOE_A8), dict(act=7), dict(T=-1), dict(H=0), dict(I=0), dict(E=0), dict(k=0),
             dict(k=9), dict(n_shared=-1), dict(n_shared=1, I_shared=0), dict(flags=1),
             dict(flags=L.MOE_W_PREPACKED), dict(offsets=None), dict(n_shared=1, I_shared=128)]
    unsupported = [dict(H=250), dict(I=100), dict(E=600), dict(T=70000), dict(T=65000, k=512, E=512),
                   dict(T=60000, k=8, H=1 << 20), dict(n_shared=1, I_shared=100)]
    if call is not _layer:
        bank = "w13" if call is _gateup else "w2"
        inval += [{bank: None}, {bank: L.MxBankDesc(None, FAKE)}, {bank: L.MxBankDesc(FAKE, None)},
                  {bank: L.MxBankDesc(FAKE + 8, FAKE)}, {bank: L.MxBankDesc(FAKE, FAKE + 2)}]
    if call is _gateup:
        inval += [dict(x=None), dict(h=None), dict(sorted_pair=None), dict(x=FAKE + 8),
                  dict(h=FAKE + 8), dict(flags=L.MOE_OUT_F32)]
    elif call is _down:
        inval += [dict(h=None), dict(out=None), dict(topk_w=None), dict(pair_pos=None),
                  dict(h=FAKE + 8), dict(out=FAKE + 8)]
    else:
        inval += [dict(renormalize=2), dict(w13=None), dict(w2=None)]
        inval += [{n: None} for n in ("logits", "x", "topk_ids", "topk_w", "counts", "sorted_pair",
                                      "pair_pos", "h", "out")]
    for kw in inval:
        assert call(**kw) == L.MOE_E_INVAL, kw
    for kw in unsupported:
        assert call(**kw) == L.MOE_E_UNSUPPORTED, kw
    for kw in (dict(workspace=None), dict(workspace=FAKE + 16), dict(ws_bytes=1)):
        assert call(**kw) == L.MOE_E_WORKSPACE, kw
    assert call(T=0) == L.MOE_OK


def test_workspace_size_of_refused_shapes_is_zero():
    def size(**kw):
        return L.moe_mx4_workspace_bytes(*dict(SHAPE, **kw).values())
    assert size() >= 4 * 2 * 256 * 4          # the fp32 rows of the down projection
    assert size(act=L.MOE_A4) >= 4 * 2 * 256 * 4 + 4 * 512 // 2   # and the codes of x
    for kw in (dict(act=1), dict(H=250), dict(k=9), dict(E=600), dict(T=70000)):
        assert size(**kw) == 0, kw


def test_bank_descriptor_is_two_pointers():
    assert ctypes.sizeof(L.MxBankDesc) == 16


def test_python_front_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    from packed_bit_grouped_amd import mx
    with pytest.raises(TypeError):
        mx.quantize_rows(torch.zeros(4, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        mx.quantize_rows(torch.zeros(4, 48))
    with pytest.raises(ValueError):
        mx.quantize_rows(torch.zeros(64))
    with pytest.raises(ValueError):
        mx.quantize_rows(torch.zeros(64, 4).t())
    with pytest.raises(ValueError):
        mx.quantize_rows(torch.zeros(1, 64).expand(4, 64))
    with pytest.raises(ValueError, match="GPU"):
        mx.quantize_rows(torch.zeros(4, 64))
    codes = torch.zeros(4, 32, dtype=torch.uint8)
    with pytest.raises(ValueError):
        mx.dequantize_rows(codes, torch.zeros(4, 3, dtype=torch.uint8))
    with pytest.raises(TypeError):
        mx.dequantize_rows(codes, torch.zeros(4, 2, dtype=torch.uint8), dtype=torch.float16)
    with pytest.raises(ValueError):
        mx.MxBank(w13=(codes, codes))
    pair = (torch.zeros(2, 64, 16, dtype=torch.uint8), torch.zeros(2, 64, 1, dtype=torch.uint8))
    with pytest.raises(ValueError, match="GPU"):
        mx.MxBank(w13=pair)
    with pytest.raises(ValueError, match="unsupported"):
        mx.MxBank(w13=(pair[0][:, :40].contiguous(), pair[1][:, :40].contiguous()))
    bank = mx.MxBank()
    assert bank.need("w13_shared", (0, 64, 32), 0) is None
    with pytest.raises(ValueError):
        bank.need("w2", (2, 64, 32), 0)
    with pytest.raises(ValueError):
        mx.MxBuffers(4, 250, 32, 4, 2, device="cpu")
    with pytest.raises(ValueError):
        mx.MxBuffers(4, 256, 32, 4, 2, act="a8", device="cpu")
    b = mx.MxBuffers(4, 32, 32, 2, 1, device="cpu")
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    offs, sp = torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for bad in (x.float(), x[:3], x.t().contiguous().t()):
        with pytest.raises((TypeError, ValueError)):
            mx.gateup_silu(bank, bad, offs, sp, b)
    with pytest.raises(ValueError):      # no such matrices in the bank
        mx.gateup_silu(bank, x, offs, sp, b)
    with pytest.raises(TypeError):
        mx.gateup_silu(bank, x, offs.long(), sp, b)


class StreamOfDevice1:
    device_index, cuda_stream = 1, 0


def test_stream_of_another_device_is_refused_before_the_library():
    pytest.importorskip("torch")
    from packed_bit_grouped_amd import mx
    for call in (lambda: mx._side(0, StreamOfDevice1()),
                 lambda: mx._launch("moe_mx4_quant_rows", 0, StreamOfDevice1(), None, 0, 0, 32, 32, None, None)):
        with pytest.raises(ValueError, match="device 1"):
            call()


def test_sizes_next_to_the_range_of_int():
    """Sums and products of sizes near 2^31 come out right or are refused
    before anything is launched."""
    K = 2 ** 31 - 32
    assert L.moe_mx4_bank_code_bytes(1, 16, K) == (2 ** 31 // 128) * 1024
    assert L.moe_mx4_bank_scale_bytes(1, 16, K) == (2 ** 31 // 512) * 256
    assert L.moe_mx4_bank_code_bytes(3, 2 ** 31 - 16, 32) == 3 * (2 ** 27 - 1) * 1024
    assert L.moe_mx4_bank_code_bytes(2 ** 31 - 1, 2 ** 31 - 16, K) == 0
    # 2 I rows, and padded rows, are ints
    for kw in (dict(T=0, H=K), dict(T=0, I=K), dict(T=1, k=1, I=2 ** 30), dict(T=1, k=1, H=2 ** 30),
               dict(T=0, n_shared=1, I_shared=K)):
        assert L.moe_mx4_workspace_bytes(*dict(SHAPE, **kw).values()) == 0, kw
    # more threads than a launch holds: many experts of very many units, many shared experts
    for kw in (dict(T=1, H=32, I=1 << 23, E=512, k=128), dict(T=1, H=32, I=32, n_shared=32768, I_shared=16384)):
        assert L.moe_mx4_workspace_bytes(*dict(SHAPE, **kw).values()) == 0, kw
        a = dict(kw, w13_shared=BANK if "n_shared" in kw else None)
        assert _gateup(**a) == L.MOE_E_UNSUPPORTED, kw
    assert L.moe_mx4_workspace_bytes(*dict(SHAPE, T=1, H=32, I=32, n_shared=8192, I_shared=16384).values()) > 0


def test_shapes_of_the_gpu_tests_run_on_the_tiles_that_they_are_for():
    """The library's own choice of kernel for every shape that a GPU test has
    for the larger tiles."""
    pytest.importorskip("torch")
    import test_gpu_mx as G
    import test_gpu_mx_edges as X

    def rows(shape, act, calls=(0, 1)):
        return {L.moe_mx4_tile_rows(act, *shape, d) for d in calls}

    for shape in G.LARGE + [G.MANY] + X.LONG_WIDE + X.LONG_NARROW:
        assert rows(shape, L.MOE_A16) == {160}, shape
    for shape in [G.FEWER] + X.LONG_NARROW:
        assert rows(shape, L.MOE_A4) == {144}, shape
    assert rows((1150, 4608, 160, 12, 1, 1, 96), L.MOE_A4, [0]) == {144}
    for shape in [G.MANY, (2000, 512, 2304, 12, 1, 0, 0)] + X.LONG_WIDE:
        assert rows(shape, L.MOE_A4) == {160}, shape
    assert rows((400, 6144, 128, 24, 1, 0, 0), L.MOE_A4, [0]) == {160}
    for shape in G.LARGE:
        assert rows(shape, L.MOE_A4) <= {144, 160}, shape
    for shape in ((1, 2048, 768, 128, 8, 1, 768), (8, 2048, 768, 128, 8, 0, 0)):
        assert rows(shape, L.MOE_A16) == rows(shape, L.MOE_A4) == {16}, shape
    assert rows((80, 40960, 128, 4, 1, 0, 0), L.MOE_A4, [0]) == {16}   # its scales do not fit beside a tile
    assert L.moe_mx4_tile_rows(L.MOE_A8, 64, 2048, 768, 128, 8) == 0
    assert L.moe_mx4_tile_rows(L.MOE_A16, 64, 2050, 768, 128, 8) == 0
    assert L.moe_mx4_tile_rows(L.MOE_A16, 64, 2048, 768, 128, 8, down=2) == 0


def test_tiles_where_both_were_measured():
    """A16 takes the larger tiles where they were measured faster: with few
    experts not before their rows fill a tile of 16, with many from the first
    rows on."""
    def gateup(T, *layer):
        return L.moe_mx4_tile_rows(L.MOE_A16, T, *layer)

    def down(T, *layer):
        return L.moe_mx4_tile_rows(L.MOE_A16, T, *layer, 0, 0, 1)

    few, many, wide = (4096, 1536, 8, 2), (4096, 1536, 256, 8), (8192, 2048, 8, 2)
    assert [gateup(T, *few) for T in (16, 32, 40, 64, 96)] == [16, 16, 16, 160, 160]
    assert [gateup(T, *wide) for T in (16, 32, 64)] == [16, 16, 160]
    assert [down(T, 4096, 14336, 8, 2) for T in (16, 32, 64)] == [16, 16, 160]
    assert [gateup(T, *many) for T in (4, 8, 16, 64)] == [16, 160, 160, 160]
    assert [gateup(T, 2048, 768, 128, 8) for T in (16, 32, 64)] == [16, 160, 160]
    assert [down(T, 2048, 768, 128, 8) for T in (64, 128)] == [16, 160]
