"""Routing of tokens by scores on the device: softmax or sigmoid scores, a bias
for balance, groups of experts, top-k and renormalised weights
(``moe_route_scored`` of include/moe_w4.h, where each step is defined).

``route_scored`` hands out the (ids, w) that ``moe_permute`` and the projections
take.  ``stream`` as in mx.py: a torch stream, or a handle as a number, on which
the inputs have to be ready; what the call allocates belongs to that stream.
"""
from __future__ import annotations

from . import _lib as L
from .mx import _F32, _I32, _empty, _gpu, _launch, _side, _used_on, _want

import torch

SCORES = {"softmax": L.MOE_SCORE_SOFTMAX, "sigmoid": L.MOE_SCORE_SIGMOID}


def route_scored(logits, k, score="sigmoid", bias=None, n_group=1, topk_group=None, group_best=2,
                 renormalize=True, scale=1.0, ids=None, w=None, stream=None):
    """The k experts (int32 [T][k]) and gate weights (fp32 [T][k]) of every token
    from its logits fp32 [T][E], in new tensors unless given.  bias: fp32 [E],
    added to the scores for the choice alone; n_group, topk_group: groups of
    E / n_group neighbouring experts, of which the topk_group stay (None: all)
    whose group_best (1 or 2) best experts sum to most; renormalize: the chosen
    scores divided by their sum; scale: a factor on the weights."""
    if score not in SCORES:
        raise ValueError(f"score: expected 'softmax' or 'sigmoid', got {score!r}")
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits: expected a tensor [T][E]")
    T, E = logits.shape
    pl = _want("logits", logits, _F32, (T, E))
    dev = _gpu(logits)
    pb = None if bias is None else _want("bias", bias, _F32, (E,), dev)
    side = _side(dev, stream)
    if ids is None:
        ids = _empty((T, k), torch.int32, logits.device, side)
    else:
        _want("ids", ids, _I32, (T, k), dev)
    if w is None:
        w = _empty((T, k), torch.float32, logits.device, side)
    else:
        _want("w", w, _F32, (T, k), dev)
    _launch("moe_route_scored", dev, stream, pl, T, E, k, SCORES[score], pb, n_group,
            n_group if topk_group is None else topk_group, group_best, int(bool(renormalize)),
            scale, ids.data_ptr(), w.data_ptr())
    _used_on(side, logits, ids, w, *(() if bias is None else (bias,)))
    return ids, w
