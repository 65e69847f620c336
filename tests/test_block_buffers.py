"""The calls around a layer with buffers longer than a batch needs: a slots (and weights) buffer made for the largest batch serves
every one of them, the gradients' call too.  No GPU: what the binding would launch is looked at, not launched."""
import pytest
import torch

import segmented_gather_matvec_amd as sg
from tests.test_block_host import on

N, K, W = 4, 2, 16


@pytest.fixture
def calls(monkeypatch):
    seen = []
    monkeypatch.setattr(sg, "_on_device", lambda index, call, stream, *args: seen.append((call, args)))
    return seen


def rows(n, dtype=torch.float16):
    return on(torch.zeros(n, W, dtype=dtype))


@pytest.mark.parametrize("longer", [0, 1, 3, N * K])
@pytest.mark.parametrize("weighted", [False, True])
def test_longer_slots_in_every_call(calls, longer, weighted):
    m = N * K
    slots, weights = on(torch.zeros(m + longer, dtype=torch.int32)), on(torch.zeros(m + longer)) if weighted else None
    ids = on(torch.zeros(N, K, dtype=torch.int32))
    sg.sgmv_route_rows(ids, 3, None, slots, None, None, None)
    sg.sgmv_dispatch_rows(rows(N), slots, rows(m))
    sg.sgmv_combine_rows(rows(m), slots, rows(N), weights=weights)
    sg.sgmv_combine_rows_backward(rows(N), None, slots, weights=weights, dYs=rows(m))
    sg.sgmv_combine_rows_backward(rows(N), rows(m), slots, weights=weights, dYs=rows(m), dweights=on(torch.zeros(m + longer)))
    sg.sgmv_combine_rows_backward(rows(N), rows(m), slots, weights=weights, dweights=on(torch.zeros(m)))
    assert [c for c, _ in calls] == ["sgmv_route_rows", "sgmv_dispatch_rows", "sgmv_combine_rows"] + ["sgmv_combine_rows_backward"] * 3
    assert all(a[1:3] == (N, K) for _, a in calls[1:])


def test_one_choice_a_row_in_a_buffer_for_two(calls):
    slots = on(torch.zeros(2 * N, dtype=torch.int32))
    sg.sgmv_combine_rows_backward(rows(N), rows(N), slots, dYs=rows(N), dweights=on(torch.zeros(N)))
    sg.sgmv_combine_rows_backward(rows(N), rows(N), slots, dweights=on(torch.zeros(N)))
    assert [a[1:3] for _, a in calls] == [(N, 1)] * 2


def test_what_is_too_short_or_does_not_agree(calls):
    m = N * K
    slots, short = on(torch.zeros(m, dtype=torch.int32)), on(torch.zeros(m - 1, dtype=torch.int32))
    f = lambda n: on(torch.zeros(n))  # noqa: E731
    for attempt, why in (
            (lambda: sg.sgmv_combine_rows_backward(rows(N), None, short, dYs=rows(m)), "slots must hold 8 entries, got 7"),
            (lambda: sg.sgmv_combine_rows_backward(rows(N), None, slots, dYs=rows(m + 1)), "dYs must have a whole number of rows"),
            (lambda: sg.sgmv_combine_rows_backward(rows(N), rows(N), slots, dYs=rows(m)), r"Ys must be \[8, 16\]"),
            (lambda: sg.sgmv_combine_rows_backward(rows(N), rows(m), slots, weights=f(m - 1), dYs=rows(m)), "weights must hold 8"),
            (lambda: sg.sgmv_combine_rows_backward(rows(N), rows(m), slots, dYs=rows(m), dweights=f(m - 1)), "dweights must hold 8"),
            (lambda: sg.sgmv_combine_rows_backward(rows(N), rows(m), short, dweights=f(m)), "slots must hold 8 entries, got 7"),
            (lambda: sg.sgmv_combine_rows_backward(rows(N), rows(m), slots, dweights=f(2 * m)), r"Ys must be \[16, 16\]"),
            (lambda: sg.sgmv_combine_rows_backward(rows(N), None, on(torch.zeros(m)), dYs=rows(m)), "slots must be torch.int32"),
            (lambda: sg.sgmv_combine_rows_backward(rows(N), None, slots, dYs=rows(m, torch.bfloat16)), "dYs must be torch.float16")):
        with pytest.raises(ValueError, match=why):
            attempt()
    assert not calls
