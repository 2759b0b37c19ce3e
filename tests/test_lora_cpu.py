"""Low-rank adapters without a GPU: the oracle against hand-worked adapters and
merged weights; the refusals of the C ABI and of the Python calls (nothing is
launched)."""
import numpy as np
import pytest

from oracle import lora_oracle as O
from packed_bit_grouped_amd import _lib as L

FAKE = 1 << 20


def test_hand_worked_rank_one():
    # one token, one expert: v = 2 * 3 (gate), 2 * 5 (up); g = 1 + 0.5 * 6 * 7, u = 1 + 0.5 * 10 * 9
    x = np.zeros((1, 4))
    x[0, 2] = 2.0
    A = np.zeros((2, 4))
    A[0, 2], A[1, 2] = 3.0, 5.0
    B = np.array([[7.0], [9.0]])
    h, _ = O.gateup(np.ones((1, 2)), x, [(0, 0)], [0], [[(A, B, 0.5)]], [1], 1, False)
    g, u = 22.0, 46.0
    assert h[0, 0] == pytest.approx(g / (1 + np.exp(-g)) * u, rel=1e-15)
    h, _ = O.gateup(np.ones((1, 2)), x, [(0, 0)], [-1], [[(A, B, 0.5)]], [1], 1, False)
    assert h[0, 0] == pytest.approx(1 / (1 + np.exp(-1.0)), rel=1e-15)


def test_merged_weights():
    """Beside the projection is as in it: W + s B A."""
    rng = np.random.default_rng(0)
    T, H, I, E, k, rank = 5, 16, 8, 3, 2, 4
    x, W13, W2 = rng.standard_normal((T, H)), rng.standard_normal((E, 2 * I, H)), rng.standard_normal((E, H, I))
    up = [[(rng.standard_normal((2 * rank, H)), rng.standard_normal((2 * I, rank)), 0.5) for _ in range(E)]
          for _ in range(2)]
    dn = [[(rng.standard_normal((rank, I)), rng.standard_normal((H, rank)), 0.25) for _ in range(E)]
          for _ in range(2)]
    ids = np.array([rng.permutation(E)[:k] for _ in range(T)])
    order = np.argsort(ids.ravel(), kind="stable")
    pos = np.argsort(order)
    adapter = np.array([0, 1, -1, 1, 0])
    rows = O.rows_of(order, ids, T, k, E, 0)
    gu = np.array([W13[e] @ x[t] for t, e in rows])
    h, _ = O.gateup(gu, x, rows, adapter, up, [I] * E, I, False)
    w = rng.random((T, k))
    y = np.array([W2[e] @ h[r] for r, (t, e) in enumerate(rows)])
    base = np.array([sum(w[t, j] * y[pos[t * k + j]] for j in range(k)) for t in range(T)])
    out, _ = O.down(base, h, rows, adapter, dn, [I] * E, w, pos, np.ones((T, 0)), T, k, False)
    for t in range(T):
        want = np.zeros(H)
        for j, e in enumerate(ids[t]):
            m13, m2 = W13[e].copy(), W2[e].copy()
            if adapter[t] >= 0:
                A, B, s = up[adapter[t]][e]
                m13[:I] += s * B[:I] @ A[:rank]
                m13[I:] += s * B[I:] @ A[rank:]
                A, B, s = dn[adapter[t]][e]
                m2 += s * B @ A
            q = m13 @ x[t]
            want += w[t, j] * (m2 @ (q[:I] / (1 + np.exp(-q[:I])) * q[I:]))
        assert out[t] == pytest.approx(want, rel=1e-10)


# ---------------------------------------------------------------------------
# refusals


def _gateup(**kw):
    a = dict(x=FAKE, T=4, H=64, I=32, E=8, k=2, n_shared=0, I_shared=0, adapter=FAKE, n_adapters=2,
             max_rank=16, table=FAKE, topk_ids=FAKE, sorted_pair=FAKE, gu=FAKE, h=2 * FAKE,
             workspace=FAKE, ws_bytes=1 << 30, flags=0)
    a.update(kw)
    return L.moe_lora_gateup_silu(*a.values(), stream=0, check=False)


def _down(**kw):
    a = dict(h=FAKE, T=4, H=64, I=32, E=8, k=2, n_shared=0, I_shared=0, adapter=FAKE, n_adapters=2,
             max_rank=16, table=FAKE, topk_w=FAKE, topk_ids=FAKE, offsets=FAKE, sorted_pair=FAKE,
             pair_pos=FAKE, base=FAKE, out=2 * FAKE, workspace=FAKE, ws_bytes=1 << 30, flags=0)
    a.update(kw)
    return L.moe_lora_down_combine(*a.values(), stream=0, check=False)


INVALID = [dict(T=-1), dict(H=0), dict(I=0), dict(E=0), dict(k=0), dict(k=9), dict(n_shared=-1),
           dict(n_shared=1, I_shared=0), dict(n_adapters=-1), dict(max_rank=0), dict(max_rank=12),
           dict(adapter=None), dict(table=None), dict(table=FAKE + 4), dict(topk_ids=None),
           dict(sorted_pair=None), dict(h=None), dict(h=FAKE + 8), dict(flags=1), dict(flags=L.MOE_GU_F32)]
UNSUPPORTED = [dict(H=48), dict(I=48), dict(n_shared=1, I_shared=48), dict(max_rank=136), dict(E=1025),
               dict(T=1 << 22, k=4), dict(n_shared=65536, I_shared=32), dict(T=1 << 17, H=1 << 14),
               dict(H=(1 << 20) + 32), dict(I=(1 << 20) + 32), dict(n_adapters=1 << 28),
               dict(T=1 << 16, I=1 << 14), dict(T=(1 << 22) + 1, k=1), dict(T=1 << 16, n_shared=1024, I_shared=32)]


@pytest.mark.parametrize("call,more", [
    (_gateup, [dict(x=None), dict(x=FAKE + 8), dict(gu=None), dict(gu=2 * FAKE), dict(gu=FAKE + 8),
               dict(flags=L.MOE_OUT_F32)]),
    (_down, [dict(topk_w=None), dict(offsets=None), dict(pair_pos=None), dict(base=None),
             dict(base=FAKE + 8), dict(out=None), dict(out=FAKE), dict(out=FAKE + 4),
             dict(out=FAKE + 8, flags=L.MOE_OUT_F32)])])
def test_invalid_arguments(call, more):
    for kw in INVALID + more:
        assert call(**kw) == L.MOE_E_INVAL, kw


@pytest.mark.parametrize("call", [_gateup, _down])
def test_unsupported_sizes_and_workspace(call):
    for kw in UNSUPPORTED:
        assert call(**kw) == L.MOE_E_UNSUPPORTED, kw
    need = L.moe_lora_workspace_bytes(4, 64, 32, 8, 2, 0, 0, 16)
    assert need >= 256
    assert call(ws_bytes=need - 1) == L.MOE_E_WORKSPACE
    assert call(workspace=None) == L.MOE_E_WORKSPACE
    assert call(workspace=FAKE + 16) == L.MOE_E_WORKSPACE
    for kw in (dict(), dict(ws_bytes=need), dict(n_adapters=0, table=None), dict(flags=L.MOE_H_F32),
               dict(n_shared=2, I_shared=96), dict(max_rank=128)):
        assert call(**kw) == L.MOE_E_DEVICE, kw
    assert call(T=0, h=None) == L.MOE_OK


def test_down_in_place_is_for_fp32():
    assert _down(out=FAKE, flags=L.MOE_OUT_F32) == L.MOE_E_DEVICE


def test_workspace_sizes():
    size = lambda T, k, s, r: L.moe_lora_workspace_bytes(T, 64, 32, 64, k, s, 32, r)
    assert size(4, 2, 0, 12) == size(4, 2, 0, 136) == size(-1, 2, 0, 16) == size(4, 0, 0, 16) == 0
    for T, k, s, r in ((0, 1, 0, 8), (1, 1, 0, 8), (64, 8, 1, 16), (4096, 8, 1, 16), (65535, 8, 0, 128)):
        assert size(T, k, s, r) >= 256 + (T * (k + s) * 2 * r * 4 if T * (k + s) > 2048 else 0)


def test_shared_sums_flag_belongs_to_gateup_alone():
    F = L.MOE_GU_F32
    assert L.moe_w4_gateup_silu(0, FAKE, 4, 64, 32, 8, 2, FAKE, None, 0, 0, FAKE, FAKE, FAKE, FAKE,
                                16, FAKE, FAKE, 1 << 30, F, stream=0, check=False) == L.MOE_E_DEVICE
    assert L.moe_w4_down_combine(0, FAKE, 4, 64, 32, 8, 2, FAKE, None, 0, 0, FAKE, FAKE, FAKE, FAKE,
                                 FAKE, FAKE, 16, FAKE, FAKE, 1 << 30, F, stream=0,
                                 check=False) == L.MOE_E_INVAL
    b = L.MxBankDesc(FAKE, FAKE)
    assert L.moe_mx4_gateup_silu(0, FAKE, 4, 64, 32, 8, 2, b, None, 0, 0, FAKE, FAKE, FAKE, FAKE,
                                 1 << 30, F, stream=0, check=False) == L.MOE_E_DEVICE
    assert L.moe_mx4_down_combine(0, FAKE, 4, 64, 32, 8, 2, b, None, 0, 0, FAKE, FAKE, FAKE, FAKE,
                                  FAKE, 1 << 30, F, stream=0, check=False) == L.MOE_E_INVAL


def test_python_refuses():
    torch = pytest.importorskip("torch")
    from packed_bit_grouped_amd import lora
    with pytest.raises(ValueError, match="max_rank"):
        lora.Adapters(2, 4, 64, 32, max_rank=12, device="cpu")
    ad = lora.Adapters(2, 4, 64, 32, 1, 96, max_rank=16, device="cpu")
    bf = dict(dtype=torch.bfloat16)
    a, b = torch.zeros(4, 16, 64, **bf), torch.zeros(4, 64, 8, **bf)
    for kw, match in ((dict(slot=2), "slot"), (dict(slot=0, b13=None), "a13"), (dict(slot=0, first=2), "first"),
                      (dict(slot=0, first=1), "sizes"), (dict(slot=0, a13=a[:, :12]), "rank"),
                      (dict(slot=0, a13=torch.zeros(4, 48, 64, **bf)), "rank"),
                      (dict(slot=0, b13=torch.zeros(4, 64, 16, **bf)), "b13"),
                      (dict(slot=0, a13=a[..., :32]), "a13")):
        with pytest.raises(ValueError, match=match):
            ad.load(**{**dict(a13=a, b13=b), **kw})
    with pytest.raises(TypeError, match="a13"):
        ad.load(0, a13=a.float(), b13=b)
    with pytest.raises(ValueError, match="aligned"):
        ad.load(0, a13=torch.zeros(4 * 16 * 64 + 8, **bf)[4:-4].view(4, 16, 64), b13=b)
    with pytest.raises(ValueError, match="GPU"):
        ad.load(1, a13=a, b13=b, scale=0.5)
    assert not ad.table["13"].any() and not ad._held


def test_tiling_refusals():
    def tile(**kw):
        a = dict(src=FAKE, n=2, rows=32, cols=64, is_b=0, dst=2 * FAKE)
        a.update(kw)
        return L.moe_lora_tile(*a.values(), stream=0, check=False)
    for kw in (dict(n=-1), dict(rows=0), dict(cols=0), dict(is_b=2), dict(src=None), dict(dst=None),
               dict(dst=FAKE), dict(src=FAKE + 8), dict(dst=FAKE + 8)):
        assert tile(**kw) == L.MOE_E_INVAL, kw
    for kw in (dict(rows=20), dict(cols=40), dict(is_b=1, rows=24), dict(is_b=1, cols=12),
               dict(rows=1 << 16, cols=1 << 15), dict(n=1 << 30, rows=64)):
        assert tile(**kw) == L.MOE_E_UNSUPPORTED, kw
    for kw in (dict(), dict(rows=8), dict(is_b=1), dict(is_b=1, cols=8)):
        assert tile(**kw) == L.MOE_E_DEVICE, kw
    assert tile(n=0, src=None, dst=None) == L.MOE_OK


def test_layer_buffers_are_all_there_from_the_start():
    """Nothing is made in a step: a step's stream is not the one that memory would come from."""
    torch = pytest.importorskip("torch")
    from packed_bit_grouped_amd import lora
    B = lora.LoraBuffers(5, 64, 32, 8, 2, 1, 96, device="cpu")
    held = {name: id(v) for name, v in vars(B).items() if isinstance(v, torch.Tensor)}
    assert {"h", "out", "ws", "gu", "base", "tiles", "n_tiles"} <= set(held)
    assert B.gu.shape == (15, 192) and B.base.shape == (5, 64)
    assert B.gu.dtype == B.base.dtype == torch.float32 and B.tiles.dtype == torch.int32
    assert len(B.tiles) == L.moe_permute_max_tiles(5, 2, 8, 4096)
    assert {name: id(getattr(B, name)) for name in held} == held
    assert lora.LoraBuffers(5, 64, 32, 8, 2, 1, 96, device="cpu", layer=False).gu is None


def test_how_a_call_runs():
    """One launch of few rows, three of many; as many tokens a block as leave a
    workgroup to each compute unit."""
    block = lambda T, H=2048, I=512, E=256, k=8, s=1, n=4, rank=16, down=1: L.moe_lora_block(
        T, H, I, E, k, s, I if s else 0, n, rank, down)
    assert block(0) == block(1) == block(64) == 0 and block(1, down=0) == block(64, down=0) == 0
    assert block(4096) == 512 and block(4096, down=0) == 256
    assert block(4096, H=1024) == 256 and block(1100, H=2080) == 128 and block(2000, H=96, E=8) == 64
    assert block(4096, n=0) == 0 and block(4096, E=1024, s=65) == 0      # more experts than a plan holds
    assert block(4096, E=1024, s=65, down=0) == 256
    assert block(4, H=48) == L.MOE_E_UNSUPPORTED and block(-1) == L.MOE_E_INVAL
    assert block(4, rank=12) == L.MOE_E_INVAL and block(4, down=2) == L.MOE_E_INVAL
