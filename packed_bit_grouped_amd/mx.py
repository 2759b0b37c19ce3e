"""The MoE FFN layer on microscaled 4-bit (MXFP4) expert weights: rows to the
format and back, banks, per-step buffers and the layer's calls.

PyTorch serves only as the device allocator and stream provider; every step
runs in the HIP kernels behind the C ABI (include/moe_w4.h, the format and the
layer are defined there).

* ``quantize_rows`` / ``dequantize_rows``: bf16 or fp32 rows <-> codes, scales.
* ``MxBank`` lays the expert matrices of a layer out for the projections, once,
  from (codes, scales) pairs of stacked tensors: codes uint8 [n][N][K/2], scales
  uint8 [n][N][K/32].
* ``MxBuffers`` preallocates every per-step buffer of one layer shape.
* ``gateup_silu``, ``down_combine`` and ``run_layer`` issue the calls on the
  current stream of the tensors' device (or on ``stream``).  The outputs are
  the buffers' own tensors, overwritten by the next call on them; calls that
  overlap in time (other streams) need buffers each.

``stream`` (a torch stream, or a stream handle as a number, which has to live
as long as the tensors it was used with): inputs, a bank and buffers have to be
ready on it, and whoever reads the results elsewhere waits for it.  What a call
allocates or copies itself it does on that stream, and the new tensors belong
to it.  ``quantize_rows``, ``quantize_bank``, ``dequantize_rows`` and ``MxBank``
may be given tensors that are dropped at once; the step calls' tensors, bank
and buffers are kept until their work is done (``MxBuffers`` and ``MxBank`` fill
their tensors on the stream that they are made on: other streams wait for it).
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib as L

BLOCK = 32
ACTS = {"a16": L.MOE_A16, "a4": L.MOE_A4, L.MOE_A16: L.MOE_A16, L.MOE_A4: L.MOE_A4}


def _here(dev, stream):
    """The torch stream, which has to be one of the device with index dev."""
    if stream.device_index != dev:
        raise ValueError(f"stream: of device {stream.device_index}, the tensors are on device {dev}")
    return stream


def _launch(name, dev, stream, *args):
    """The C call on the device with index dev, on the stream (None: that
    device's current one)."""
    if stream is not None and not isinstance(stream, int):
        stream = _here(dev, stream).cuda_stream
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _launch(name, dev, stream, *args)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    st = getattr(L._lib or L.load(), name)(*args, stream)
    if st:
        raise L.MoeError(name, st, L.status_str(st))


def _side(dev, stream):
    """`stream` as a torch stream of the device with index dev; None: the
    current one there, on which torch allocates and copies anyway."""
    if stream is None:
        return None
    if not isinstance(stream, int):
        return _here(dev, stream)
    if stream == 0:
        return torch.cuda.default_stream(dev)
    return torch.cuda.ExternalStream(stream, device=dev)


def _empty(shape, dtype, device, side):
    """Memory of the stream `side`: what was freed there earlier is free there,
    while the current stream's pool may hand out what queued work still uses."""
    if side is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(side):
        return torch.empty(shape, dtype=dtype, device=device)


def _used_on(side, *tensors):
    """The tensors' memory is given to nothing else before the work that is
    queued on `side` by now is done, even if the caller drops them at once."""
    if side is not None:
        for t in tensors:
            t.record_stream(side)


def _want(name, t, dtypes, shape, dev=None):
    """t has one of the dtypes, the shape, no gaps, and lies on the device with
    index dev (None: any); returns its address."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape
            and t.is_contiguous() and (dev is None or t.get_device() == dev)):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise TypeError(f"{name}: expected a tensor of {' or '.join(map(str, dtypes))}, got "
                        f"{getattr(t, 'dtype', type(t))}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    raise ValueError(f"{name}: on {t.device}, expected it on the device of the other tensors")


_BF16 = (torch.bfloat16, torch.int16)   # int16: bf16 bit patterns
_F32 = (torch.float32,)
_I32 = (torch.int32,)
_U8 = (torch.uint8,)


def _gpu(t):
    if not t.is_cuda:
        raise ValueError(f"expected a tensor on the GPU, got one on {t.device}")
    return t.get_device()


def quantize_rows(src, codes=None, scales=None, stream=None):
    """bf16 or fp32 rows [R][C] (unit stride along C, any row stride) to MXFP4:
    (codes uint8 [R][C/2], scales uint8 [R][C/32]), new unless given."""
    f32 = src.dtype is torch.float32
    if not f32 and src.dtype is not torch.bfloat16:
        raise TypeError(f"src: expected bfloat16 or float32, got {src.dtype}")
    if src.dim() != 2:
        raise ValueError(f"src: expected rows [R][C], got shape {tuple(src.shape)}")
    R, C = src.shape
    if C == 0 or C % BLOCK:
        raise ValueError(f"src: rows of {C} values, expected a multiple of {BLOCK}")
    ld, unit = src.stride()
    if R <= 1:
        ld = C
    if R > 0 and unit != 1:
        raise ValueError("src: expected unit stride along C")
    if ld < C:
        raise ValueError("src: rows overlap")
    dev = _gpu(src)
    side = _side(dev, stream)
    if codes is None:
        codes = _empty((R, C // 2), torch.uint8, src.device, side)
    else:
        _want("codes", codes, _U8, (R, C // 2), dev)
    if scales is None:
        scales = _empty((R, C // BLOCK), torch.uint8, src.device, side)
    else:
        _want("scales", scales, _U8, (R, C // BLOCK), dev)
    _launch("moe_mx4_quant_rows", dev, stream, src.data_ptr(), f32, R, C, ld, codes.data_ptr(),
            scales.data_ptr())
    _used_on(side, src, codes, scales)
    return codes, scales


def dequantize_rows(codes, scales, dtype=torch.bfloat16, stream=None):
    """The values [R][C] (bf16 or fp32) of codes [R][C/2] and scales [R][C/32]."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"dtype: expected bfloat16 or float32, got {dtype}")
    if codes.dim() != 2:
        raise ValueError(f"codes: expected rows [R][C/2], got shape {tuple(codes.shape)}")
    R, C = codes.shape
    C *= 2
    if C == 0 or C % BLOCK:
        raise ValueError(f"codes: rows of {C} values, expected a multiple of {BLOCK}")
    pc = _want("codes", codes, _U8, (R, C // 2))
    ps = _want("scales", scales, _U8, (R, C // BLOCK), codes.get_device())
    dev = _gpu(codes)
    side = _side(dev, stream)
    dst = _empty((R, C), dtype, codes.device, side)
    _launch("moe_mx4_dequant_rows", dev, stream, pc, ps, R, C, dst.data_ptr(),
            dtype is torch.float32, C)
    _used_on(side, codes, scales)
    return dst


def quantize_bank(w, stream=None):
    """fp32 or bf16 matrices [n][N][K] to one (codes, scales) pair for MxBank."""
    n, N, K = w.shape
    side = _side(_gpu(w), stream)
    if side is None:
        rows = w.reshape(n * N, K)
    else:   # matrices that are not contiguous are copied: in front of the call that reads the copy
        with torch.cuda.stream(side):
            rows = w.reshape(n * N, K)
        _used_on(side, w)
    codes, scales = quantize_rows(rows, stream=stream)
    return codes.view(n, N, K // 2), scales.view(n, N, K // BLOCK)


class MxBank:
    """The matrices of one layer: w13 [E][2I][H] and w2 [E][H][I] of the routed
    experts, w13_shared [n_shared][2*I_shared][H] and w2_shared
    [n_shared][H][I_shared] of the shared ones, each given as a (codes, scales)
    pair of plain rows and kept tiled (moe_mx4_tile_bank): the pairs are not
    needed any more.  A bank for one of the projections alone is given that
    projection's pairs.  A later change of the weights needs a new bank."""

    def __init__(self, w13=None, w2=None, w13_shared=None, w2_shared=None, stream=None):
        self.tiles, self.desc, self.addr, self.shape = {}, {}, {}, {}
        self.device = None
        for tag, p in (("w13", w13), ("w2", w2), ("w13_shared", w13_shared),
                       ("w2_shared", w2_shared)):
            self.shape[tag] = None
            if p is None:
                continue
            codes, scales = p
            if codes.dim() != 3:
                raise ValueError(f"{tag}: expected codes [n][N][K/2], got {tuple(codes.shape)}")
            n, N, K = codes.shape[0], codes.shape[1], 2 * codes.shape[2]
            _want(tag + " codes", codes, _U8, (n, N, K // 2), self.device)
            self.device = codes.get_device()
            _want(tag + " scales", scales, _U8, (n, N, K // BLOCK), self.device)
            nc, ns = L.moe_mx4_bank_code_bytes(n, N, K), L.moe_mx4_bank_scale_bytes(n, N, K)
            if nc == 0:
                raise ValueError(f"{tag}: unsupported matrices (n, N, K) = {(n, N, K)}")
            side = _side(_gpu(codes), stream)
            tc = _empty(nc, torch.uint8, codes.device, side)
            ts = _empty(ns, torch.uint8, codes.device, side)
            _launch("moe_mx4_tile_bank", self.device, stream, codes.data_ptr(), scales.data_ptr(),
                    n, N, K, tc.data_ptr(), ts.data_ptr())
            _used_on(side, codes, scales)
            self.tiles[tag] = (tc, ts)
            self.desc[tag] = L.MxBankDesc(tc.data_ptr(), ts.data_ptr())
            self.addr[tag] = ctypes.addressof(self.desc[tag])
            self.shape[tag] = (n, N, K)

    def need(self, tag, shape, dev):
        """The address of the descriptor of `tag`, whose matrices have to be of
        that shape (n, N, K) and on the device with index dev."""
        if shape[0] == 0:
            return None
        if self.shape[tag] != shape:
            raise ValueError(f"{tag}: the bank holds {self.shape[tag]} (n, N, K), the buffers "
                             f"are for {shape}")
        if self.device != dev:
            raise ValueError(f"{tag}: the bank and the buffers are on different devices")
        return self.addr[tag]


class MxBuffers:
    """Every per-step buffer of one layer shape, allocated once."""

    def __init__(self, T, H, I, E, k, n_shared=0, I_shared=0, act="a16", device="cuda",
                 out_f32=False):
        if act not in ACTS:
            raise ValueError(f"act: expected 'a16' or 'a4', got {act!r}")
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.n_shared, self.I_shared, self.act = n_shared, I_shared, ACTS[act]
        P = T * k
        self.P, self.R = P, P + n_shared * T
        self.ld_h = max(I, I_shared if n_shared else 0)
        self.ws_bytes = L.moe_mx4_workspace_bytes(self.act, T, H, I, E, k, n_shared, I_shared)
        if self.ws_bytes == 0:
            raise ValueError(f"unsupported layer shape: T={T} H={H} I={I} E={E} k={k} "
                             f"n_shared={n_shared} I_shared={I_shared}")
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self._dev = dev.index if dev.type == "cuda" else -1
        # the matrices that a bank has to hold for these buffers
        self.mats = {"w13": (E, 2 * I, H), "w2": (E, H, I), "w13_shared": (n_shared, 2 * I_shared, H),
                     "w2_shared": (n_shared, H, I_shared)}
        i32 = dict(dtype=torch.int32, device=dev)
        self.ids = torch.empty((T, k), **i32)
        self.w = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.counts = torch.empty(E, **i32)
        self.offsets = torch.empty(E + 1, **i32)
        self.sorted_pair = torch.empty(P, **i32)
        self.pair_pos = torch.empty(P, **i32)
        # zeroed once: the columns past a shorter expert's I are never written
        self.h = torch.zeros((self.R, self.ld_h), dtype=torch.bfloat16, device=dev)
        self.out_flags = L.MOE_OUT_F32 if out_f32 else 0
        self.out = torch.empty((T, H), dtype=torch.float32 if out_f32 else torch.bfloat16,
                               device=dev)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)


def _gate(shared_gate, B):
    if shared_gate is None or not B.n_shared:
        return None
    return _want("shared_gate", shared_gate, _F32, (B.T, B.n_shared), B._dev)


def gateup_silu(bank, x, offsets, sorted_pair, B, stream=None, gu=None):
    """h [T*k + n_shared*T][max(I, I_shared)] in bf16 (B.h) of x bf16 [T][H] and
    the sort's tables (int32): rows in the order of the sort, then the shared
    experts' tokens.  With gu, fp32 [...][2*max(I, I_shared)], the gate and up
    sums go there as they are (MOE_GU_F32, see lora.py), and gu is returned."""
    dev = B._dev
    px = _want("x", x, _BF16, (B.T, B.H), dev)
    po = _want("offsets", offsets, _I32, (B.E + 1,), dev)
    pp = _want("sorted_pair", sorted_pair, _I32, (B.P,), dev)
    need, mats = bank.need, B.mats
    w13, sh = need("w13", mats["w13"], dev), need("w13_shared", mats["w13_shared"], dev)
    if gu is None:
        to, flags = B.h.data_ptr(), 0
    else:
        to, flags = _want("gu", gu, _F32, (B.R, 2 * B.ld_h), dev), L.MOE_GU_F32
    _launch("moe_mx4_gateup_silu", dev, stream, B.act, px, B.T, B.H, B.I, B.E, B.k, w13, sh,
            B.n_shared, B.I_shared, po, pp, to, B.ws.data_ptr(), B.ws_bytes, flags)
    return B.h if gu is None else gu


def down_combine(bank, h, w, offsets, pair_pos, B, shared_gate=None, stream=None, out=None):
    """out [T][H] (B.out, or `out` in fp32 if given) of h (as from gateup_silu),
    the gate weights w fp32 [T][k] and the sort's tables; shared_gate fp32
    [T][n_shared]: gate logits of the shared experts (sigmoid), None: weight 1."""
    dev = B._dev
    ph = _want("h", h, _BF16, (B.R, B.ld_h), dev)
    pw = _want("w", w, _F32, (B.T, B.k), dev)
    po = _want("offsets", offsets, _I32, (B.E + 1,), dev)
    pp = _want("pair_pos", pair_pos, _I32, (B.P,), dev)
    need, mats = bank.need, B.mats
    w2, sh = need("w2", mats["w2"], dev), need("w2_shared", mats["w2_shared"], dev)
    if out is None:
        to, flags = B.out.data_ptr(), B.out_flags
    else:
        to, flags = _want("out", out, _F32, (B.T, B.H), dev), L.MOE_OUT_F32
    _launch("moe_mx4_down_combine", dev, stream, B.act, ph, B.T, B.H, B.I, B.E, B.k, w2, sh,
            B.n_shared, B.I_shared, _gate(shared_gate, B), pw, po, pp, to, B.ws.data_ptr(),
            B.ws_bytes, flags)
    return B.out if out is None else out


def run_layer(bank, x, logits, B, renormalize=1, shared_gate=None, stream=None):
    """One layer step: out [T][H] (B.out) of x bf16 [T][H] and the router's
    logits fp32 [T][E]; the routing's results are in B.ids, B.w and the sort's
    tables of B."""
    dev = B._dev
    px = _want("x", x, _BF16, (B.T, B.H), dev)
    pl = _want("logits", logits, _F32, (B.T, B.E), dev)
    need, mats = bank.need, B.mats
    w13, w2 = need("w13", mats["w13"], dev), need("w2", mats["w2"], dev)
    s13, s2 = need("w13_shared", mats["w13_shared"], dev), need("w2_shared", mats["w2_shared"], dev)
    _launch("moe_mx4_layer", dev, stream, B.act, pl, px, B.T, B.H, B.I, B.E, B.k,
            int(renormalize), w13, w2, s13, s2, B.n_shared, B.I_shared, _gate(shared_gate, B),
            B.ids.data_ptr(), B.w.data_ptr(), B.counts.data_ptr(), B.offsets.data_ptr(),
            B.sorted_pair.data_ptr(), B.pair_pos.data_ptr(), B.h.data_ptr(), B.out.data_ptr(),
            B.ws.data_ptr(), B.ws_bytes, B.out_flags)
    return B.out
