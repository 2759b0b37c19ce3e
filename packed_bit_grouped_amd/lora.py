"""Low-rank adapters of many requests beside the experts' projections: the
adapters' tables, per-step buffers and the calls (``moe_lora_*`` of
include/moe_w4.h, where the operators are defined).

The packed expert weights are shared by all requests and stay as they are; a
token may have an adapter, which holds for an expert's gate/up and down
projections a pair of low-rank matrices and a scale.

* ``Adapters`` holds the tables of up to n adapters of one layer; ``load`` and
  ``unload`` fill and empty a place while the others serve.
* ``LoraBuffers`` preallocates the per-step buffers of one layer shape.
* ``gateup_silu`` and ``down_combine`` run the adapters beside the two
  projections; ``run_layer`` runs a whole layer, routing included, on an int4/int2
  bank (layer.py) or an MXFP4 one (mx.py).

``stream`` as in mx.py: a torch stream, or a handle as a number, on which inputs,
tables and buffers have to be ready.  Outputs are the buffers' own tensors,
overwritten by the next call on them; calls that overlap in time need buffers
each.  ``Adapters`` keeps its own copies of the matrices until their place is
loaded anew or emptied: wait for the steps that still use them before doing so.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import _lib as L
from . import layer as _w4
from . import mx as _mx
from . import router as _router
from .mx import _BF16, _F32, _I32, _empty, _gate, _gpu, _launch, _side, _used_on, _want

_DESC = np.dtype([("a", np.uint64), ("b", np.uint64), ("rank", np.int32), ("scale", np.float32),
                  ("N", np.int32), ("K", np.int32)])   # struct moe_lora
assert _DESC.itemsize == ctypes.sizeof(L.LoraDesc)
_TILE_M = 4096   # of a sort whose tiles nobody reads: as few as there can be


class Adapters:
    """Tables of n adapters of a layer with E routed experts of H x I and
    n_shared shared ones of H x I_shared; ranks are multiples of 8 up to
    max_rank.  A place that nothing was loaded into has no effect."""

    def __init__(self, n, E, H, I, n_shared=0, I_shared=0, max_rank=16, device="cuda"):
        if n < 0 or max_rank <= 0 or max_rank % 8 or max_rank > 128:
            raise ValueError(f"n = {n}, max_rank = {max_rank}: expected n >= 0 and a multiple of 8 "
                             "up to 128")
        self.n, self.E, self.H, self.I = n, E, H, I
        self.n_shared, self.I_shared, self.max_rank = n_shared, I_shared, max_rank
        self.per = E + n_shared
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self._dev = dev.index if dev.type == "cuda" else -1
        size = ctypes.sizeof(L.LoraDesc)
        self._host = {tag: (L.LoraDesc * (n * self.per))() for tag in ("13", "2")}
        self.table = {tag: torch.zeros(max(n * self.per, 1) * size, dtype=torch.uint8, device=dev)
                      for tag in self._host}
        self._held = {}

    def _entries(self, tag, slot, first, count):
        lo = slot * self.per + first
        return np.frombuffer(self._host[tag], dtype=_DESC)[lo:lo + count]

    def _put(self, tag, slot, first, count, stream):
        size = ctypes.sizeof(L.LoraDesc)
        lo = (slot * self.per + first) * size
        src = torch.from_numpy(self._entries(tag, slot, first, count).copy().view(np.uint8))
        side = _side(self._dev, stream) if self._dev >= 0 else None
        if side is None:
            self.table[tag][lo:lo + count * size].copy_(src)
        else:
            with torch.cuda.stream(side):
                self.table[tag][lo:lo + count * size].copy_(src)

    def load(self, slot, a13=None, b13=None, a2=None, b2=None, scale=1.0, first=0, stream=None):
        """Adapter `slot` for the experts first, first + 1, ... (shared experts
        are numbers E, ...; one call holds experts of one size): a13 bf16
        [m][2*rank][H] (the gate's rows, then up's) with b13 [m][2I][rank], and a2
        [m][rank][I] with b2 [m][H][rank], or one of the pairs alone.  They are
        laid out anew (moe_lora_tile) and not needed any more."""
        if not 0 <= slot < self.n:
            raise ValueError(f"slot: {slot}, expected one of {self.n}")
        if (a13 is None) != (b13 is None) or (a2 is None) != (b2 is None) or (a13 is None and a2 is None):
            raise ValueError("expected a13 with b13, a2 with b2, or both pairs")
        m = (a13 if a13 is not None else a2).shape[0]
        if first < 0 or m < 1 or first + m > self.per:
            raise ValueError(f"first: experts {first} to {first + m - 1} of {self.per}")
        widths = {self.I if e < self.E else self.I_shared for e in (first, first + m - 1)}
        if len(widths) != 1:
            raise ValueError("first: routed and shared experts of different sizes in one call")
        width = widths.pop()
        todo = []
        for tag, a, b, halves, N, K in (("13", a13, b13, 2, 2 * width, self.H),
                                        ("2", a2, b2, 1, self.H, width)):
            if a is None:
                continue
            rank = a.shape[1] // halves if a.dim() == 3 else 0
            if rank <= 0 or rank % 8 or rank > self.max_rank:
                raise ValueError(f"a{tag}: shape {tuple(a.shape)}, expected [{m}][{halves} * rank][{K}] "
                                 f"with a rank of 8, 16, ... up to {self.max_rank}")
            pa = _want("a" + tag, a, _BF16, (m, halves * rank, K), self._dev)
            pb = _want("b" + tag, b, _BF16, (m, N, rank), self._dev)
            if (pa | pb) % 16:
                raise ValueError(f"a{tag}, b{tag}: expected 16-byte aligned matrices")
            todo.append((tag, a, b, rank, N, K))
        for tag, a, b, rank, N, K in todo:
            side = _side(_gpu(a), stream)
            rows = (a.shape[1] + 15) // 16 * 16
            ta = _empty((m, rows, K), torch.bfloat16, a.device, side)
            tb = _empty(b.shape, torch.bfloat16, b.device, side)
            _launch("moe_lora_tile", self._dev, stream, a.data_ptr(), m, a.shape[1], K, 0, ta.data_ptr())
            _launch("moe_lora_tile", self._dev, stream, b.data_ptr(), m, N, rank, 1, tb.data_ptr())
            _used_on(side, a, b)
            d = self._entries(tag, slot, first, m)
            i = np.arange(m, dtype=np.uint64)
            d["a"] = ta.data_ptr() + i * np.uint64(rows * K * 2)
            d["b"] = tb.data_ptr() + i * np.uint64(N * rank * 2)
            d["rank"], d["scale"], d["N"], d["K"] = rank, scale, N, K
            self._held.update({(tag, slot, first + i): (ta, tb) for i in range(m)})
            self._put(tag, slot, first, m, stream)

    def unload(self, slot, stream=None):
        """Empties a place."""
        if not 0 <= slot < self.n:
            raise ValueError(f"slot: {slot}, expected one of {self.n}")
        for tag in self._host:
            self._entries(tag, slot, 0, self.per)[:] = np.zeros((), _DESC)
            for e in range(self.per):
                self._held.pop((tag, slot, e), None)
            self._put(tag, slot, 0, self.per, stream)


class LoraBuffers:
    """Every per-step buffer of the adapters of one layer shape, allocated once,
    on the stream that is current then (other streams wait for it).
    h_f32: h in fp32 (layers with 8-bit activations), else bf16.  layer: with
    what run_layer keeps between the calls: the shared projections' sums gu fp32
    [R][2 * ld_h] and base fp32 [T][H], and the sort's tile list; False for
    callers of gateup_silu and down_combine that bring their own."""

    def __init__(self, T, H, I, E, k, n_shared=0, I_shared=0, max_rank=16, h_f32=False,
                 out_f32=False, device="cuda", layer=True):
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.n_shared, self.I_shared, self.max_rank = n_shared, I_shared, max_rank
        self.P = T * k
        self.R = self.P + n_shared * T
        self.ld_h = max(I, I_shared if n_shared else 0)
        self.ws_bytes = L.moe_lora_workspace_bytes(T, H, I, E, k, n_shared, I_shared, max_rank)
        if self.ws_bytes == 0:
            raise ValueError(f"unsupported sizes: T={T} H={H} I={I} E={E} k={k} n_shared={n_shared} "
                             f"I_shared={I_shared} max_rank={max_rank}")
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self._dev = dev.index if dev.type == "cuda" else -1
        self.h_flags = L.MOE_H_F32 if h_f32 else 0
        self.out_flags = L.MOE_OUT_F32 if out_f32 else 0
        # zeroed once: the columns past a shorter expert's I are never written
        self.h = torch.zeros((self.R, self.ld_h), device=dev,
                             dtype=torch.float32 if h_f32 else torch.bfloat16)
        self.out = torch.empty((T, H), device=dev, dtype=torch.float32 if out_f32 else torch.bfloat16)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)
        self.ws[:256].zero_()
        self.gu = self.base = self.tiles = self.n_tiles = None
        if layer:
            self.gu = torch.zeros((self.R, 2 * self.ld_h), dtype=torch.float32, device=dev)
            self.base = torch.empty((T, H), dtype=torch.float32, device=dev)
            # for projections that bring no tile list of their own
            m = max(L.moe_permute_max_tiles(T, k, E, _TILE_M), 1)
            self.tiles = torch.empty((m, 4), dtype=torch.int32, device=dev)
            self.n_tiles = torch.zeros(1, dtype=torch.int32, device=dev)

    def error_word(self) -> int:
        return int(self.ws[:4].view(torch.int32).item())


def _table(adapters, tag, B):
    for name in ("E", "H", "I", "n_shared"):
        if getattr(adapters, name) != getattr(B, name):
            raise ValueError(f"adapters: made for {name} = {getattr(adapters, name)}, the buffers "
                             f"for {getattr(B, name)}")
    if B.n_shared and adapters.I_shared != B.I_shared:
        raise ValueError(f"adapters: made for I_shared = {adapters.I_shared}, the buffers for "
                         f"{B.I_shared}")
    if adapters.max_rank > B.max_rank:
        raise ValueError(f"adapters: ranks up to {adapters.max_rank}, the buffers are for "
                         f"{B.max_rank}")
    if adapters._dev != B._dev:
        raise ValueError("adapters: on another device than the buffers")
    return adapters.table[tag].data_ptr() if adapters.n else None


def gateup_silu(adapters, x, adapter, gu, ids, offsets, sorted_pair, B, stream=None):
    """h (B.h) of x bf16 [T][H], the tokens' adapters int32 [T] (-1: none), the
    shared projection's sums gu fp32 [R][2 * ld_h] (mx.gateup_silu(gu=...), or
    MOE_GU_F32) and the routing's tables."""
    dev = B._dev
    px = _want("x", x, _BF16, (B.T, B.H), dev)
    pa = _want("adapter", adapter, _I32, (B.T,), dev)
    pg = _want("gu", gu, _F32, (B.R, 2 * B.ld_h), dev)
    pi = _want("ids", ids, _I32, (B.T, B.k), dev)
    _want("offsets", offsets, _I32, (B.E + 1,), dev)
    pp = _want("sorted_pair", sorted_pair, _I32, (B.P,), dev)
    pt = _table(adapters, "13", B)
    _launch("moe_lora_gateup_silu", dev, stream, px, B.T, B.H, B.I, B.E, B.k, B.n_shared,
            B.I_shared, pa, adapters.n, B.max_rank, pt, pi, pp, pg, B.h.data_ptr(),
            B.ws.data_ptr(), B.ws_bytes, B.h_flags)
    return B.h


def down_combine(adapters, h, base, adapter, w, ids, offsets, sorted_pair, pair_pos, B,
                 shared_gate=None, stream=None):
    """out [T][H] (B.out) of h (as from gateup_silu), the shared projection's
    weighted sum base fp32 [T][H], the tokens' adapters, the gate weights w fp32
    [T][k] and the routing's tables; shared_gate as in mx.down_combine."""
    dev = B._dev
    ph = _want("h", h, _F32 if B.h_flags else _BF16, (B.R, B.ld_h), dev)
    pb = _want("base", base, _F32, (B.T, B.H), dev)
    pa = _want("adapter", adapter, _I32, (B.T,), dev)
    pw = _want("w", w, _F32, (B.T, B.k), dev)
    pi = _want("ids", ids, _I32, (B.T, B.k), dev)
    po = _want("offsets", offsets, _I32, (B.E + 1,), dev)
    ps = _want("sorted_pair", sorted_pair, _I32, (B.P,), dev)
    pp = _want("pair_pos", pair_pos, _I32, (B.P,), dev)
    pt = _table(adapters, "2", B)
    _launch("moe_lora_down_combine", dev, stream, ph, B.T, B.H, B.I, B.E, B.k, B.n_shared,
            B.I_shared, pa, adapters.n, B.max_rank, pt, _gate(shared_gate, B), pw, pi, po, ps, pp,
            pb, B.out.data_ptr(), B.ws.data_ptr(), B.ws_bytes, B.h_flags | B.out_flags)
    return B.out


def run_layer(bank, M, adapters, B, x, adapter, logits, renormalize=1, routing=None,
              shared_gate=None, flags=0, stream=None):
    """One layer step with adapters: out [T][H] (B.out).  bank and M are the
    shared weights and their buffers, layer.Bank with layer.LayerBuffers or
    mx.MxBank with mx.MxBuffers; routing None: the softmax top-k of
    moe_route_topk (renormalize as there), else the keyword arguments of
    router.route_scored.  The routing's results are in M.ids, M.w and M's tables.
    flags: MOE_PATH_* (and MOE_QUANT_SEPARATE) of the int4/int2 projections.  What
    does not fit is refused before anything is launched."""
    T, H, I, E, k = M.T, M.H, M.I, M.E, M.k
    if (T, H, I, E, k, M.n_shared) != (B.T, B.H, B.I, B.E, B.k, B.n_shared) or M.ld_h != B.ld_h or (
            M.n_shared and M.I_shared != B.I_shared):
        raise ValueError("the shared projections' buffers and the adapters' are for different layers")
    packed = isinstance(M, _w4.LayerBuffers)
    wide = packed and M.act == L.MOE_A8
    if wide != bool(B.h_flags):
        raise ValueError("h_f32: fp32 h goes with 8-bit activations, bf16 h with the others")
    if not isinstance(bank, _w4.Bank if packed else _mx.MxBank):
        raise TypeError(f"bank: {type(bank).__name__} does not go with {type(M).__name__}")
    if flags & ~((L.MOE_PATH_MASK | L.MOE_QUANT_SEPARATE) if packed else 0):
        raise ValueError(f"flags: {flags:#x}, expected MOE_PATH_* of the int4/int2 projections")
    if M.ids.device != B.device:
        raise ValueError(f"the shared projections' buffers are on {M.ids.device}, the adapters' on {B.device}")
    if B.gu is None:
        raise ValueError("the adapters' buffers were made with layer=False")
    if T == 0:
        return B.out
    dev = B._dev
    if packed:
        w_flags = flags | (L.MOE_W_PREPACKED if bank.prepacked else 0)
        for tag, n in (("w13", E), ("w2", E), ("w13_sh", M.n_shared), ("w2_sh", M.n_shared)):
            table = getattr(bank, tag)
            held = 0 if table is None else table.numel() // ctypes.sizeof(L.QMatDesc)
            if held < n or (n and table.device != B.device):
                raise ValueError(f"{tag}: the bank holds {held} matrices, the buffers are for {n} on {B.device}")
        L.moe_w4_covers(M.act, T, H, I, E, k, M.n_shared, M.I_shared, M.tile_m, w_flags)
    else:
        for tag, shape in M.mats.items():
            bank.need(tag, shape, dev)
    _want("logits", logits, _F32, (T, E), dev)
    if _want("x", x, _BF16, (T, H), dev) % 16:
        raise ValueError("x: expected 16-byte aligned rows")
    _want("adapter", adapter, _I32, (T,), dev)
    _gate(shared_gate, B)
    _table(adapters, "13", B)
    if stream is not None and not isinstance(stream, int):
        stream = _mx._here(dev, stream).cuda_stream
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return run_layer(bank, M, adapters, B, x, adapter, logits, renormalize, routing,
                             shared_gate, flags, stream)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    if routing is None:
        L.moe_route_topk(logits, T, E, k, int(renormalize), M.ids, M.w, stream)
    else:
        _router.route_scored(logits, k, ids=M.ids, w=M.w, stream=stream, **routing)
    if packed:
        tile_m, tiles, n_tiles = M.tile_m, M.tiles, M.n_tiles
    else:
        tile_m, tiles, n_tiles = _TILE_M, B.tiles, B.n_tiles
    L.moe_permute(M.ids, T, k, E, tile_m, M.counts, M.offsets, M.sorted_pair, M.pair_pos, tiles,
                  n_tiles, stream)
    if not packed:
        _mx.gateup_silu(bank, x, M.offsets, M.sorted_pair, M, stream, gu=B.gu)
    else:
        L.moe_w4_gateup_silu(M.act, x, T, H, I, E, k, bank.w13, bank.w13_sh, M.n_shared,
                             M.I_shared, M.offsets, M.sorted_pair, tiles, n_tiles, tile_m, B.gu,
                             M.ws, M.ws_bytes, w_flags | L.MOE_GU_F32, stream)
    h = gateup_silu(adapters, x, adapter, B.gu, M.ids, M.offsets, M.sorted_pair, B, stream)
    if not packed:
        _mx.down_combine(bank, h, M.w, M.offsets, M.pair_pos, M, shared_gate, stream, out=B.base)
    else:
        L.moe_w4_down_combine(M.act, h, T, H, I, E, k, bank.w2, bank.w2_sh, M.n_shared,
                              M.I_shared, M.w, M.offsets, M.sorted_pair, M.pair_pos, tiles,
                              n_tiles, tile_m, B.base, M.ws, M.ws_bytes, w_flags | L.MOE_OUT_F32,
                              stream, shared_gate=shared_gate)
    return down_combine(adapters, h, B.base, adapter, M.w, M.ids, M.offsets, M.sorted_pair,
                        M.pair_pos, B, shared_gate, stream)
