"""The microscaled 4-bit (MXFP4) operators of the mixture-of-experts layer, as
cases to measure: each in a plain form of elementary torch operations and as
the calls a user makes of the library.

The format: a row of C values is cut into blocks of 32.  A block is held as 32
codes of 4 bits (sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2,
3, 4, 6 and their negatives, two codes a byte, the even index in the low
nibble) and one scale byte s that stands for 2**(s - 127); s = 255 marks a
block that held a value that is not finite.  A block is made from its largest
magnitude a: the scale is 2**(floor(log2 a) - 2), every value is divided by it
and rounded to the nearest code (a tie to the even mantissa), magnitudes above
6 become 6; a block of zeros has s = 0.

The operators ("op" of a case):
  quant   rows (bf16 or fp32) to codes and scales, and back to the values they
          stand for, in bf16
  gateup  h[r] = SiLU(x . Wg_e) * (x . Wu_e) of every (token, expert) pair in
          the order of the sort by expert, then of every shared expert, bf16
  down    out[t] = sum_j w[t, j] * (h . W2_e) + sum_s g[t, s] * (h_s . W2_s)
  layer   routing of the logits (the k largest, softmax over them), gate/up,
          down and the weighted sum
"act" says how activations meet the 4-bit weights: "a16" bf16 as they are,
"a4" quantised to the same format by the rule above (x before gate/up, h, in
bf16, before down).
"""
import math

import torch

own = False

BLOCK = 32


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # The hidden rows of 12 tokens (4 requests of 3 draft positions): the
        # smallest call, where the launch is what a caller pays.
        {"name": "quant_rows_12", "op": "quant", "src": "bf16", "R": 12, "C": 2048, "pad": 0},
        # The activations of one prefill chunk.
        {"name": "quant_rows_4096", "op": "quant", "src": "bf16", "R": 4096, "C": 4096, "pad": 0},
        # Packing a checkpoint's fp32 gate/up weights, 64 experts at a time.
        {"name": "quant_bank", "op": "quant", "src": "fp32", "R": 64 * 2 * 768, "C": 2048, "pad": 0},
        # One token of one request, with a shared expert: the first half of a decode step.
        {"name": "gateup_t1", "op": "gateup", "act": "a16", "T": 1, "H": 2048, "I": 768, "E": 128, "k": 8,
         "n_shared": 1, "skew": False},
        # A decode batch of 64 requests with 4-bit activations: about 4 rows an expert.
        {"name": "gateup_t64_a4", "op": "gateup", "act": "a4", "T": 64, "H": 2048, "I": 768, "E": 128, "k": 8,
         "n_shared": 0, "skew": False},
        # A prefill chunk over 256 experts: about 128 rows an expert.
        {"name": "gateup_t4096", "op": "gateup", "act": "a16", "T": 4096, "H": 4096, "I": 1536, "E": 256, "k": 8,
         "n_shared": 0, "skew": False},
        # Speculative decode of 12 positions with a few favoured experts and a gated shared one.
        {"name": "down_t12", "op": "down", "act": "a16", "T": 12, "H": 2048, "I": 768, "E": 128, "k": 8,
         "n_shared": 1, "skew": True},
        # The second half of the prefill chunk, 4-bit activations.
        {"name": "down_t4096_a4", "op": "down", "act": "a4", "T": 4096, "H": 4096, "I": 1536, "E": 256, "k": 8,
         "n_shared": 0, "skew": False},
        # A whole decode step of one token.
        {"name": "layer_t1", "op": "layer", "act": "a16", "T": 1, "H": 2048, "I": 768, "E": 128, "k": 8,
         "n_shared": 1, "skew": False},
        # A whole step of 12 draft positions, 4-bit activations, favoured experts.
        {"name": "layer_t12_a4", "op": "layer", "act": "a4", "T": 12, "H": 2048, "I": 768, "E": 128, "k": 8,
         "n_shared": 1, "skew": True},
        # A ragged batch on a layer whose sizes are odd numbers of blocks.
        {"name": "layer_odd", "op": "layer", "act": "a16", "T": 37, "H": 1056, "I": 352, "E": 12, "k": 3,
         "n_shared": 0, "skew": True},
        # A whole prefill chunk, 4-bit activations: the largest.
        {"name": "layer_t4096_a4", "op": "layer", "act": "a4", "T": 4096, "H": 4096, "I": 1536, "E": 256, "k": 8,
         "n_shared": 0, "skew": False},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["quant", "gateup", "down", "layer"])
    if op == "quant":
        C = BLOCK * _spread(rng, 1, 128)
        R = min(_spread(rng, 1, 1 << 17), (1 << 27) // C)
        return {"op": op, "src": rng.choice(["bf16", "fp32"]), "R": R, "C": C, "pad": rng.choice([0, 0, 8, 3])}
    E = _spread(rng, 4, 256)
    n_shared = rng.choice([0, 0, 1])
    return {"op": op, "act": rng.choice(["a16", "a4"]), "T": _spread(rng, 1, 4096), "H": BLOCK * _spread(rng, 8, 128),
            "I": BLOCK * _spread(rng, 4, 48), "E": E, "k": rng.randint(1, min(E, 8 - n_shared)), "n_shared": n_shared,
            "skew": rng.random() < 0.5}


def work(case):
    if case["op"] == "quant":
        n = case["R"] * case["C"]
        packed = n // 2 + n // BLOCK
        # the rows read, the packed form written and read, the values written
        return {"bytes": n * (2 if case["src"] == "bf16" else 4) + 2 * packed + 2 * n, "flops": 4 * n}
    T, H, I, E, k, s = (case[x] for x in ("T", "H", "I", "E", "k", "n_shared"))
    rows = T * (k + s)
    # experts that at least one of T tokens is expected to choose
    share = [(e + 1) ** -1.1 if case["skew"] else 1.0 for e in range(E)]
    touched = s + sum(1 - (1 - min(1.0, k * p / sum(share))) ** T for p in share)
    up, down = 2 * I * H, H * I
    packed = 0.5 + 1 / BLOCK
    x, h, out = T * H * 2, rows * I * 2, T * H * 2
    if case["op"] == "gateup":
        return {"bytes": touched * up * packed + x + h, "flops": 2 * rows * up}
    if case["op"] == "down":
        return {"bytes": touched * down * packed + h + out, "flops": 2 * rows * down}
    return {"bytes": touched * (up + down) * packed + T * E * 4 + x + out, "flops": 2 * rows * (up + down)}


# ---------------------------------------------------------------------------
# inputs


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _weights(gen, n, N, K):
    """n matrices [N][K] of N(0, 0.02), quantised: codes [n][N][K/2], scales [n][N][K/32]."""
    codes = torch.empty((n, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n, N, K // BLOCK), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (N * K))
    for i in range(0, n, step):
        m = min(step, n - i)
        _, e, q = _quantise(_normal(gen, m * N, K) * 0.02)
        nib = q.abs()  # 0, .5, 1, 1.5, 2, 3, 4, 6 are the codes 0..7
        nib = torch.where(nib < 2, nib * 2, torch.where(nib < 4, nib + 2, nib / 2 + 4)).to(torch.uint8)
        nib = (nib + 8 * torch.signbit(q)).to(torch.uint8).view(m, N, K)
        codes[i:i + m] = nib[..., 0::2] | (nib[..., 1::2] << 4)
        scales[i:i + m] = (e + 127).to(torch.uint8).view(m, N, K // BLOCK)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = {"case": case}
    if case["op"] == "quant":
        R, C = case["R"], case["C"]
        dtype = torch.bfloat16 if case["src"] == "bf16" else torch.float32
        # rows of a larger buffer where "pad" says so; a few channels are much
        # larger than the rest, as activations are, and a few blocks are zero
        full = _normal(gen, R, C + case["pad"])
        full *= torch.exp(1.5 * _normal(gen, C + case["pad"]))
        full[:, :BLOCK] *= (_normal(gen, R, 1) > -1).float()
        state["rows"] = full.to(dtype)[:, :C]
        return state
    T, H, I, E, k, s = (case[x] for x in ("T", "H", "I", "E", "k", "n_shared"))
    logits = _normal(gen, T, E) * (0.02 * math.sqrt(H))
    if case["skew"]:  # a Zipf(1.1) prior over the experts, in an order of its own
        rank = torch.randperm(E, generator=gen, device="cuda")
        logits -= 1.1 * torch.log(rank.float() + 1)
    ids, w = _route(logits, k)
    offsets, order = _sort(ids, E)
    state["most"] = int((offsets[1:] - offsets[:-1]).max())  # rows of the fullest expert
    if case["op"] != "down":
        state["x"] = _normal(gen, T, H).bfloat16()
        state["w13"] = _weights(gen, E, 2 * I, H)
        state["w13_shared"] = _weights(gen, s, 2 * I, H) if s else None
    if case["op"] != "gateup":
        state["w2"] = _weights(gen, E, H, I)
        state["w2_shared"] = _weights(gen, s, H, I) if s else None
        state["gate"] = _normal(gen, T, s) if s else None  # the shared experts' gate logits
    if case["op"] == "layer":
        state["logits"] = logits
    else:  # the tables that the routing call leaves behind
        state["offsets"], state["sorted_pair"] = offsets.int(), order.int()
    if case["op"] == "down":
        g, u = _normal(gen, T * (k + s), I) * 0.9, _normal(gen, T * (k + s), I) * 0.9
        state["h"] = (g * torch.sigmoid(g) * u).bfloat16()
        state["w"] = w
        pos = torch.empty_like(order)
        pos[order] = torch.arange(T * k, device="cuda")
        state["pair_pos"] = pos.int()
    if own:  # the per-step buffers that a program allocates once
        from packed_bit_grouped_amd import mx
        state["bank"] = mx.MxBank(state.get("w13"), state.get("w2"), state.get("w13_shared"), state.get("w2_shared"))
        state["buffers"] = mx.MxBuffers(T, H, I, E, k, s, I if s else 0, act=case["act"])
    return state


# ---------------------------------------------------------------------------
# one pass


def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    return {"quant": _plain_quant, "gateup": _plain_gateup, "down": _plain_down, "layer": _plain_layer}[case["op"]](case, state)


def _run_own(case, state):
    from packed_bit_grouped_amd import mx
    if case["op"] == "quant":
        codes, scales = mx.quantize_rows(state["rows"])
        return {"values": mx.dequantize_rows(codes, scales)}
    b = state["buffers"]
    if case["op"] == "gateup":
        return {"h": mx.gateup_silu(state["bank"], state["x"], state["offsets"], state["sorted_pair"], b)}
    if case["op"] == "down":
        return {"out": mx.down_combine(state["bank"], state["h"], state["w"], state["offsets"], state["pair_pos"], b,
                                       shared_gate=state["gate"])}
    out = mx.run_layer(state["bank"], state["x"], state["logits"], b, shared_gate=state["gate"])
    return {"out": out, "ids": b.ids, "w": b.w}


# ---------------------------------------------------------------------------
# the plain form


def _quantise(rows):
    """(values, scale exponents, codes as numbers) of fp32 rows [R][C]: [R][C], [R][C/32], [R][C]."""
    R, C = rows.shape
    v = rows.view(R, C // BLOCK, BLOCK)
    a = v.abs().amax(-1, keepdim=True)
    e = torch.where(a > 0, torch.frexp(a).exponent - 3, -127).clamp(min=-127)
    m = torch.ldexp(v, -e)
    step = torch.where(m.abs() < 2, 0.5, torch.where(m.abs() < 4, 1.0, 2.0))
    q = (torch.round(m / step) * step).clamp(-6, 6)  # round: half to even
    return torch.ldexp(q, e).view(R, C), e.view(R, C // BLOCK), q.view(R, C)


def _values(packed):
    """The fp32 values of (codes [..., N, K/2], scales [..., N, K/32]): [..., N, K]."""
    codes, scales = packed
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    grid = torch.cat([grid, -grid])
    pairs = torch.stack([grid.repeat(16), grid.repeat_interleave(16)], -1)  # of every byte
    v = pairs[codes.int()].view(*scales.shape, BLOCK)
    return (v * torch.exp2(scales.float() - 127).unsqueeze(-1)).flatten(-2)


def _plain_quant(case, state):
    return {"values": _quantise(state["rows"].float().contiguous())[0].bfloat16()}


def _route(logits, k):
    order = torch.sort(logits, dim=-1, descending=True, stable=True)  # ties: the lower index first
    top = order.values[:, :k]
    w = torch.exp(top - top[:, :1])
    return order.indices[:, :k].int(), w / w.sum(-1, keepdim=True)


def _sort(ids, E):
    order = torch.sort(ids.flatten().long(), stable=True)
    edges = torch.arange(E + 1, device=ids.device)
    return torch.searchsorted(order.values, edges), order.indices


def _grouped(rows, packed, offsets, most):
    """rows [P][K], in the order of their experts, times their experts' matrices [E][N][K]: [P][N], in fp32."""
    P, E = rows.shape[0], packed[0].shape[0]
    at = torch.arange(P, device=rows.device)
    expert = torch.searchsorted(offsets[1:].contiguous(), at.to(offsets.dtype), right=True)
    if P < E:  # fewer rows than experts: only the matrices that are used
        w = _values((packed[0][expert], packed[1][expert]))
        return torch.bmm(w, rows.unsqueeze(-1)).squeeze(-1)
    place = at - offsets[expert]
    padded = rows.new_zeros(E, most, rows.shape[1])
    padded[expert, place] = rows
    return torch.bmm(padded, _values(packed).transpose(1, 2))[expert, place]


def _plain_h(case, state, x, offsets, order):
    T, I, k, s = case["T"], case["I"], case["k"], case["n_shared"]
    x = x.float()
    if case["act"] == "a4":
        x = _quantise(x)[0]
    y = _grouped(x[order.long() // k], state["w13"], offsets, state["most"])
    if s:
        shared = torch.bmm(x.expand(s, T, -1), _values(state["w13_shared"]).transpose(1, 2))
        y = torch.cat([y, shared.reshape(s * T, 2 * I)])
    g, u = y[:, :I], y[:, I:]
    return (g / (1 + torch.exp(-g)) * u).bfloat16()


def _plain_out(case, state, h, w, offsets, pos):
    T, H, k, s = case["T"], case["H"], case["k"], case["n_shared"]
    h = h.float()
    if case["act"] == "a4":
        h = _quantise(h)[0]
    y = _grouped(h[:T * k], state["w2"], offsets, state["most"])
    out = (w.unsqueeze(-1) * y[pos.long()].view(T, k, H)).sum(1)
    if s:
        shared = torch.bmm(h[T * k:].view(s, T, -1), _values(state["w2_shared"]).transpose(1, 2))
        out = out + (torch.sigmoid(state["gate"]).t().unsqueeze(-1) * shared).sum(0)
    return out.bfloat16()


def _plain_gateup(case, state):
    return {"h": _plain_h(case, state, state["x"], state["offsets"], state["sorted_pair"])}


def _plain_down(case, state):
    return {"out": _plain_out(case, state, state["h"], state["w"], state["offsets"], state["pair_pos"])}


def _plain_layer(case, state):
    ids, w = _route(state["logits"], case["k"])
    offsets, order = _sort(ids, case["E"])
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=order.device)
    h = _plain_h(case, state, state["x"], offsets, order)
    return {"out": _plain_out(case, state, h, w, offsets, pos), "ids": ids, "w": w}


# ---------------------------------------------------------------------------
# the definition in 64 bits


def _to_grid(v):
    """Rows in 64 bits, each value replaced by the one that its block holds for it: the nearest of the 15, by distance."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=v.device)
    blocks = v.unflatten(-1, (-1, BLOCK))
    top = blocks.abs().amax(-1, keepdim=True)
    unit = torch.exp2((torch.floor(torch.log2(top.clamp(min=2.0 ** -149))) - 2).clamp(min=-127))
    ratio = blocks.abs() / unit
    middle = (grid[1:] + grid[:-1]) / 2
    # how many midpoints lie below; a midpoint itself goes to the neighbour with the even index
    low, high = torch.bucketize(ratio, middle), torch.bucketize(ratio, middle, right=True)
    place = torch.where(low == high, low, torch.where(low % 2 == 0, low, high))
    return (grid[place] * unit * torch.sign(blocks)).flatten(-2)


def _matrix(packed, i):
    """Matrix i in 64 bits, from sign, exponent and mantissa of every code."""
    codes, scales = packed[0][i], packed[1][i]
    nib = torch.stack([codes % 16, codes // 16], -1).flatten(-2)
    sign, ex, man = (nib // 8).double(), (nib // 2 % 4).double(), (nib % 2).double()
    mag = torch.where(ex == 0, man / 2, (1 + man / 2) * 2.0 ** (ex - 1))
    return (1 - 2 * sign) * mag * (2.0 ** (scales.double() - 127)).repeat_interleave(BLOCK, -1)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "quant":
        n = case["R"]
        step = max(1, (1 << 25) // case["C"])
        return {"values": torch.cat([_to_grid(state["rows"][i:i + step].double()) for i in range(0, n, step)])}
    T, H, I, E, k, s = (case[x] for x in ("T", "H", "I", "E", "k", "n_shared"))
    if case["op"] == "layer":
        logits = state["logits"].double()
        ids = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k]
        w = torch.softmax(torch.gather(logits, 1, ids), 1)
        flat = ids.flatten()
        sorted_pair = torch.argsort(flat, stable=True)
        counts = torch.bincount(flat, minlength=E).tolist()
    else:
        counts = (state["offsets"][1:] - state["offsets"][:-1]).tolist()
        sorted_pair = state["sorted_pair"].long()
    if case["op"] == "down":
        h, w = state["h"].double(), state["w"].double()
    else:
        x = state["x"].double()
        x = _to_grid(x) if case["act"] == "a4" else x
        h = torch.empty(T * (k + s), I, dtype=torch.float64, device="cuda")
        r = 0
        for e, n in enumerate(counts + [T] * s):
            if n:
                rows = x[sorted_pair[r:r + n] // k] if e < E else x
                y = rows @ (_matrix(state["w13"], e) if e < E else _matrix(state["w13_shared"], e - E)).t()
                h[r:r + n] = y[:, :I] * torch.sigmoid(y[:, :I]) * y[:, I:]
            r += n
        if case["op"] == "gateup":
            return {"h": h}
        h = h.bfloat16().double()  # the layer hands h on in bf16
    if case["act"] == "a4":
        h = _to_grid(h)
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    r = 0
    for e, n in enumerate(counts + [T] * s):
        if n:
            y = h[r:r + n] @ (_matrix(state["w2"], e) if e < E else _matrix(state["w2_shared"], e - E)).t()
            if e < E:
                pair = sorted_pair[r:r + n]
                out.index_add_(0, pair // k, y * w.flatten()[pair].unsqueeze(-1))
            else:
                out += y * torch.sigmoid(state["gate"][:, e - E].double()).unsqueeze(-1)
        r += n
    return {"out": out, "ids": ids, "w": w} if case["op"] == "layer" else {"out": out}
