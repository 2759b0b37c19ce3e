"""Routing by scores and low-rank adapters of the mixture-of-experts layer, as
cases to measure: each in a plain form of elementary torch operations and as
the calls a user makes of the library.

The operators ("op" of a case):
  route   a token's k experts and their weights from its logits: scores s are
          the softmax over all experts or each logit's sigmoid; choice values
          c = s + bias; of n_group equal groups of neighbouring experts only the
          topk_group best stay (a group counts the sum of its best one or two
          c); of those the k experts with the largest c are chosen (ties to the
          lower index), with weights s, divided by their sum where "renorm" says
          so, times a factor
  gateup  low-rank adapters of many requests beside the gate/up projection that
          all requests share: a row is a (token, expert) pair in the order of
          the sort by expert, or a shared expert's token; with g, u the shared
          projection's sums of the row and (A, B) the matrices that the token's
          adapter has for the row's expert,
          h = SiLU(g + scale Bg (Ag x)) * (u + scale Bu (Au x))
  down    the same beside down: out[t] = base[t] + sum over the token's rows of
          (gate weight) scale B (A h)
Tokens without an adapter (-1) have g, u and base alone.
"""
import math

import torch

own = False


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # One token of one request: the smallest call, where the launch is what a caller pays.
        {"name": "route_t1", "op": "route", "T": 1, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "n_group": 8,
         "topk_group": 4, "best": 2, "renorm": True, "scale": 2.5, "coarse": False},
        # A decode batch; softmax over all experts, neither groups nor bias; logits as a bf16 product leaves them (with ties).
        {"name": "route_t64", "op": "route", "T": 64, "E": 128, "k": 8, "score": "softmax", "bias": False, "n_group": 1,
         "topk_group": 1, "best": 1, "renorm": False, "scale": 1.0, "coarse": True},
        # A ragged batch over odd groups that count their best expert alone.
        {"name": "route_odd", "op": "route", "T": 777, "E": 159, "k": 6, "score": "softmax", "bias": True, "n_group": 3,
         "topk_group": 2, "best": 1, "renorm": True, "scale": 16.0, "coarse": True},
        # A prefill chunk.
        {"name": "route_t4096", "op": "route", "T": 4096, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "n_group": 8,
         "topk_group": 4, "best": 2, "renorm": True, "scale": 2.5, "coarse": False},
        # One token of one request in a server that holds four adapters, with a shared expert.
        {"name": "gateup_t1", "op": "gateup", "T": 1, "H": 2048, "I": 512, "E": 256, "k": 8, "n_shared": 1, "n": 4,
         "rank": 16, "mixed": False, "none": 0.0, "wide": False},
        # A decode batch of 64 requests over 32 adapters: hardly two rows share one.
        {"name": "gateup_t64", "op": "gateup", "T": 64, "H": 2048, "I": 512, "E": 256, "k": 8, "n_shared": 1, "n": 32,
         "rank": 16, "mixed": True, "none": 0.0, "wide": False},
        # A ragged batch on odd sizes, a quarter of the requests without an adapter, h in fp32 (8-bit activations follow).
        {"name": "gateup_odd", "op": "gateup", "T": 77, "H": 1056, "I": 352, "E": 12, "k": 3, "n_shared": 0, "n": 5,
         "rank": 24, "mixed": True, "none": 0.25, "wide": True},
        # A prefill chunk of four prompts, an adapter each.
        {"name": "gateup_t4096", "op": "gateup", "T": 4096, "H": 2048, "I": 512, "E": 256, "k": 8, "n_shared": 1, "n": 4,
         "rank": 16, "mixed": False, "none": 0.0, "wide": False},
        # The second half of the same steps.
        {"name": "down_t1", "op": "down", "T": 1, "H": 2048, "I": 512, "E": 256, "k": 8, "n_shared": 1, "n": 4,
         "rank": 16, "mixed": False, "none": 0.0, "wide": False},
        {"name": "down_t64", "op": "down", "T": 64, "H": 2048, "I": 512, "E": 256, "k": 8, "n_shared": 1, "n": 32,
         "rank": 16, "mixed": True, "none": 0.0, "wide": False},
        {"name": "down_odd", "op": "down", "T": 77, "H": 1056, "I": 352, "E": 12, "k": 3, "n_shared": 0, "n": 5,
         "rank": 24, "mixed": True, "none": 0.25, "wide": True},
        {"name": "down_t4096", "op": "down", "T": 4096, "H": 2048, "I": 512, "E": 256, "k": 8, "n_shared": 1, "n": 4,
         "rank": 16, "mixed": False, "none": 0.0, "wide": False},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["route", "gateup", "down"])
    if op == "route":
        n_group = rng.choice([1, 1, 2, 3, 4, 8])
        size = _spread(rng, 2, 512 // n_group)
        topk_group = rng.randint(1, n_group)
        return {"op": op, "T": min(_spread(rng, 1, 16384), (1 << 20) // (n_group * size)), "E": n_group * size,
                "k": rng.randint(1, min(16, topk_group * size)), "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "n_group": n_group, "topk_group": topk_group, "best": rng.choice([1, 2]),
                "renorm": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5]), "coarse": rng.random() < 0.5}
    most = work(next(c for c in listed() if c["name"] == op + "_t4096"))
    while True:
        E = _spread(rng, 4, 256)
        n_shared = rng.choice([0, 0, 1])
        case = {"op": op, "T": _spread(rng, 1, 4096), "H": 32 * _spread(rng, 8, 128), "I": 32 * _spread(rng, 4, 48), "E": E,
                "k": rng.randint(1, min(E, 8 - n_shared)), "n_shared": n_shared, "n": _spread(rng, 1, 64),
                "rank": 8 * _spread(rng, 1, 16), "mixed": rng.random() < 0.5, "none": rng.choice([0.0, 0.0, 0.25]),
                "wide": rng.random() < 0.3}
        cost = work(case)
        held = case["n"] * (E + n_shared) * case["rank"] * (3 * case["H"] + 3 * case["I"])
        if held < 1 << 30 and all(cost[x] <= most[x] for x in most):
            return case


def work(case):
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "route":
        # the logits and the bias read, ids and weights written; an exponential counted as ten operations
        return {"bytes": 4 * T * E + 4 * E * case["bias"] + 8 * T * k, "flops": 12 * T * E}
    H, I, s, n, rank = (case[x] for x in ("H", "I", "n_shared", "n", "rank"))
    rows = T * (k + s)
    tokens = T * (1 - case["none"])
    # (adapter, expert) pairs that at least one token is expected to need
    used = min(n, tokens)
    pairs = used * (s + E * (1 - (1 - k / E) ** (tokens / used)))
    if case["op"] == "gateup":
        matrices = 2 * rank * H + 2 * I * rank
        data = T * H * 2 + rows * 2 * I * 4 + rows * I * (4 if case["wide"] else 2)
    else:
        matrices = rank * I + H * rank
        data = rows * I * (4 if case["wide"] else 2) + T * H * 4 + T * H * (4 if case["wide"] else 2) + T * k * 4
    return {"bytes": int(pairs * matrices * 2 + data), "flops": int(2 * tokens * (k + s) * matrices)}


# ---------------------------------------------------------------------------
# inputs


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _matrices(gen, n, N, K, std):
    """n matrices [N][K] in bf16."""
    out = torch.empty((n, N, K), dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 27) // (N * K))
    for i in range(0, n, step):
        m = min(step, n - i)
        out[i:i + m] = _normal(gen, m, N, K) * std
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = {"case": case}
    T, E, k = case["T"], case["E"], case["k"]
    # activations of unit size against a router of standard deviation 0.02, 2048 long
    logits = _normal(gen, T, E) * (0.02 * math.sqrt(2048))
    if case["op"] == "route":
        state["logits"] = logits.bfloat16().float() if case["coarse"] else logits
        state["bias"] = _normal(gen, E) * 0.1 if case["bias"] else None
        if own:
            state["ids"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
            state["w"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
        return state
    H, I, s, n, rank = (case[x] for x in ("H", "I", "n_shared", "n", "rank"))
    rows = T * (k + s)
    # the routing's tables
    top = torch.topk(logits, k, dim=-1)
    flat = top.indices.flatten()
    order = torch.sort(flat, stable=True)
    edges = torch.arange(E + 1, device="cuda")
    pos = torch.empty_like(order.indices)
    pos[order.indices] = torch.arange(T * k, device="cuda")
    state["ids"] = top.indices.int()
    state["w"] = torch.softmax(top.values, -1)
    state["offsets"] = torch.searchsorted(order.values, edges).int()
    state["sorted_pair"], state["pair_pos"] = order.indices.int(), pos.int()
    # the tokens' adapters: of prompts that follow one another, or of requests of a token each
    if case["mixed"]:
        adapter = torch.randint(0, n, (T,), generator=gen, device="cuda")
    else:
        first = torch.randint(0, n, (1,), generator=gen, device="cuda")
        adapter = (first + torch.arange(T, device="cuda") * n // T) % n
    adapter[torch.rand(T, generator=gen, device="cuda") < case["none"]] = -1
    state["adapter"] = adapter.int()
    state["scale"] = [2.0 ** (i % 3) / 2 for i in range(n)]
    x_in = H if case["op"] == "gateup" else I
    out = 2 * I if case["op"] == "gateup" else H
    wide = case["op"] == "gateup"
    state["a"] = _matrices(gen, n * (E + s), (2 if wide else 1) * rank, x_in, x_in ** -0.5).unflatten(0, (n, E + s))
    state["b"] = _matrices(gen, n * (E + s), out, rank, 0.3 * rank ** -0.5).unflatten(0, (n, E + s))
    if wide:
        state["x"] = _normal(gen, T, H).bfloat16()
        state["gu"] = _normal(gen, rows, 2 * I) * 0.9
    else:
        g, u = _normal(gen, rows, I) * 0.9, _normal(gen, rows, I) * 0.9
        h = g * torch.sigmoid(g) * u
        state["h"] = h if case["wide"] else h.bfloat16()
        state["base"] = _normal(gen, T, H) * 0.3
        state["gate"] = _normal(gen, T, s) if s else None  # the shared experts' gate logits
    if own:  # the adapters' table and the per-step buffers that a program allocates once
        from packed_bit_grouped_amd import lora
        state["adapters"] = lora.Adapters(n, E, H, I, s, I if s else 0, max_rank=rank)
        for i in range(n):
            pair = {("a13" if wide else "a2"): state["a"][i], ("b13" if wide else "b2"): state["b"][i]}
            state["adapters"].load(i, scale=state["scale"][i], **pair)
        state["buffers"] = lora.LoraBuffers(T, H, I, E, k, s, I if s else 0, max_rank=rank, h_f32=case["wide"],
                                            out_f32=case["wide"])
    return state


# ---------------------------------------------------------------------------
# one pass


def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    return {"route": _plain_route, "gateup": _plain_gateup, "down": _plain_down}[case["op"]](case, state)


def _run_own(case, state):
    if case["op"] == "route":
        from packed_bit_grouped_amd import router
        ids, w = router.route_scored(state["logits"], case["k"], score=case["score"], bias=state["bias"],
                                     n_group=case["n_group"], topk_group=case["topk_group"], group_best=case["best"],
                                     renormalize=case["renorm"], scale=case["scale"], ids=state["ids"], w=state["w"])
        return {"ids": ids, "w": w}
    from packed_bit_grouped_amd import lora
    b = state["buffers"]
    if case["op"] == "gateup":
        return {"h": lora.gateup_silu(state["adapters"], state["x"], state["adapter"], state["gu"], state["ids"],
                                      state["offsets"], state["sorted_pair"], b)}
    return {"out": lora.down_combine(state["adapters"], state["h"], state["base"], state["adapter"], state["w"],
                                     state["ids"], state["offsets"], state["sorted_pair"], state["pair_pos"], b,
                                     shared_gate=state["gate"])}


# ---------------------------------------------------------------------------
# the plain form


def _plain_route(case, state):
    E, n_group = case["E"], case["n_group"]
    l = state["logits"].double()  # choices next to a border: 64 bits
    if case["score"] == "softmax":
        s = torch.exp(l - l.amax(-1, keepdim=True))
        s = s / s.sum(-1, keepdim=True)
    else:
        s = 1 / (1 + torch.exp(-l))
    c = s if state["bias"] is None else s + state["bias"].double()
    if n_group > 1:
        groups = c.unflatten(-1, (n_group, E // n_group))
        value = torch.sort(groups, -1, descending=True).values[..., :case["best"]].sum(-1)
        best = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, :case["topk_group"]]
        stays = torch.zeros_like(value, dtype=torch.bool)
        stays[torch.arange(best.shape[0], device=best.device).unsqueeze(-1), best] = True
        c = torch.where(stays.unsqueeze(-1), groups, -math.inf).flatten(-2)
    ids = torch.sort(c, dim=-1, descending=True, stable=True).indices[:, :case["k"]]
    w = s[torch.arange(ids.shape[0], device=ids.device).unsqueeze(-1), ids]
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return {"ids": ids.int(), "w": (w * case["scale"]).float()}


def _rows(case, state):
    """Token, and number of the adapter's pair of matrices (-1: none), of every row."""
    T, E, k, s = case["T"], case["E"], case["k"], case["n_shared"]
    pair = state["sorted_pair"].long()
    token = torch.cat([pair // k, torch.arange(T, device=pair.device).repeat(s)])
    expert = torch.cat([state["ids"].flatten().long()[pair], E + torch.arange(s, device=pair.device).repeat_interleave(T)])
    adapter = state["adapter"].long()[token]
    return token, torch.where(adapter < 0, -1, adapter * (E + s) + expert)


def _plain_products(case, state, rows, key, halves):
    """scale B (A row) of every row, in fp32: [R][N]; halves: gate and up have the rows of A and B by halves."""
    a, b = state["a"].flatten(0, 1), state["b"].flatten(0, 1)
    scale = torch.tensor(state["scale"], device=key.device).repeat_interleave(state["a"].shape[1])
    rank, N = case["rank"], b.shape[1]
    out = rows.new_zeros(rows.shape[0], N)
    step = max(1, (1 << 28) // (a.shape[1] * a.shape[2] + N * rank))
    for i in range(0, rows.shape[0], step):
        q = key[i:i + step]
        at = q.clamp(min=0)
        v = torch.bmm(a[at].float(), rows[i:i + step].unsqueeze(-1)).unflatten(1, (halves, rank))
        y = torch.matmul(b[at].float().unflatten(1, (halves, N // halves)), v).flatten(1)
        out[i:i + step] = torch.where(q.unsqueeze(-1) < 0, 0, y * scale[at].unsqueeze(-1))
    return out


def _plain_gateup(case, state):
    I = case["I"]
    token, key = _rows(case, state)
    y = state["gu"] + _plain_products(case, state, state["x"].float()[token], key, 2)
    g, u = y[:, :I], y[:, I:]
    h = g / (1 + torch.exp(-g)) * u
    return {"h": h if case["wide"] else h.bfloat16()}


def _plain_down(case, state):
    T, H, k, s = case["T"], case["H"], case["k"], case["n_shared"]
    _, key = _rows(case, state)
    y = _plain_products(case, state, state["h"].float(), key, 1)
    out = (state["w"].unsqueeze(-1) * y[state["pair_pos"].long()].view(T, k, H)).sum(1)
    if s:
        gate = 1 / (1 + torch.exp(-state["gate"]))
        out = out + (gate.t().unsqueeze(-1) * y[T * k:].view(s, T, H)).sum(0)
    out = state["base"] + out
    return {"out": out if case["wide"] else out.bfloat16()}


# ---------------------------------------------------------------------------
# the definition in 64 bits


def _exact_route(case, state):
    E, k, size = case["E"], case["k"], case["E"] // case["n_group"]
    l = state["logits"].double().cpu()
    s = torch.softmax(l, 1) if case["score"] == "softmax" else torch.sigmoid(l)
    c = s.clone() if state["bias"] is None else s + state["bias"].double().cpu()
    if case["n_group"] > 1:
        value = torch.stack([g.topk(min(case["best"], size), 1).values.sum(1) for g in c.split(size, 1)], 1)
        # a group stays if fewer than topk_group come before it
        before = (value.unsqueeze(1) > value.unsqueeze(2)).sum(2)
        same = (value.unsqueeze(1) == value.unsqueeze(2)).tril(-1).sum(2)
        c[(before + same >= case["topk_group"]).repeat_interleave(size, 1)] = -math.inf
    ids = torch.argsort(c, dim=1, descending=True, stable=True)[:, :k]
    w = torch.gather(s, 1, ids)
    if case["renorm"]:
        w /= w.sum(1, keepdim=True)
    return {"ids": ids.int().cuda(), "w": (w * case["scale"]).cuda()}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, state)
    T, H, I, E, k, s, rank = (case[x] for x in ("T", "H", "I", "E", "k", "n_shared", "rank"))
    R = T * (k + s)
    counts = (state["offsets"][1:] - state["offsets"][:-1]).tolist()
    pair = state["sorted_pair"].long()
    token = torch.cat([pair // k] + [torch.arange(T, device="cuda")] * s)
    adapter = state["adapter"].long()
    delta = torch.zeros(R, 2 * I if case["op"] == "gateup" else H, dtype=torch.float64, device="cuda")
    r = 0
    for e, m in enumerate(counts + [T] * s):
        of = adapter[token[r:r + m]]
        for d in torch.unique(of).tolist():
            if d < 0:
                continue
            at = r + (of == d).nonzero().flatten()
            A, B = state["a"][d, e].double(), state["b"][d, e].double()
            if case["op"] == "gateup":
                v = state["x"][token[at]].double() @ A.t()
                delta[at, :I] = state["scale"][d] * (v[:, :rank] @ B[:I].t())
                delta[at, I:] = state["scale"][d] * (v[:, rank:] @ B[I:].t())
            else:
                delta[at] = state["scale"][d] * ((state["h"][at].double() @ A.t()) @ B.t())
        r += m
    if case["op"] == "gateup":
        y = state["gu"].double() + delta
        return {"h": y[:, :I] * torch.sigmoid(y[:, :I]) * y[:, I:]}
    out = state["base"].double()
    out.index_add_(0, pair // k, delta[:T * k] * state["w"].double().flatten()[pair].unsqueeze(-1))
    for i in range(s):
        gate = torch.sigmoid(state["gate"][:, i].double())
        out += gate.unsqueeze(-1) * delta[T * k + i * T:T * k + (i + 1) * T]
    return {"out": out}
