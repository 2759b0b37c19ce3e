"""The adapters' calls where their other tests do not go: the sums of a block of
tokens over several segments of windows and more units than are taken at a time."""
import numpy as np
import pytest

from packed_bit_grouped_amd import _lib as L

torch = pytest.importorskip("torch")
from test_gpu_lora import check_down, make, run_down  # noqa: E402

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
