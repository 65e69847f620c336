"""Layer calls past what the other entry points take: more segments and longer ones, and gradients of so many LoRAs and
columns that they need several launches."""
import pytest
import torch

import segmented_gather_matvec_amd as sg
from tests import layer_reference as lr
from tests.test_gpu_layer import check_grads, i32, run_dense, run_dense_back

pytestmark = pytest.mark.gpu


def sorted_by_lora(c, rows_of):
    """The same layer with rows ordered by LoRA, one segment each: equal row by row, and equal gradients but for the order
    of the sums.  Returns it and the order."""
    order = torch.argsort(rows_of, stable=True)
    s = lr.Layer(1, "f16", 0, c.h_in, c.h_out, c.rank, c.P, "none", 0)
    s.dtype, s.n, s.proj, s.X, s.dY = c.dtype, c.n, c.proj, c.X[order], c.dY[order]
    ends = torch.searchsorted(rows_of[order].contiguous(), torch.arange(c.P, device="cuda"), right=True).tolist()
    s.seg, s.ids = [0] + ends, list(range(c.P))
    return s, order


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("layout", ["a_row_each", "one_segment"])
def test_more_rows_and_segments_than_other_entry_points_take(layout, dtype):
    n, P = (150_000, 3) if layout == "a_row_each" else (2_200_000, 1)
    c = lr.Layer(5, dtype, n, 16, 24, 8, P, "none", 1, None, True)
    if layout == "a_row_each":
        c.seg, c.ids = list(range(n + 1)), [i * 7 % P for i in range(n)]
    else:
        c.seg, c.ids = [0, n], [0]
    problem = sg.make_problem(dtype, n, 16, 24, 8, P, len(c.ids), n // len(c.ids))
    assert sg.sgmv_check_problem(problem) != sg.SGMV_OK
    rows_of = torch.tensor(c.ids, device="cuda").repeat_interleave(n // len(c.ids))
    s, order = sorted_by_lora(c, rows_of)
    lr.check(run_dense(c, dtype)[order], *lr.project(s, s.proj[0]), c.dtype, "Y")
    dX, grads = run_dense_back(c, dtype)
    d = s.dY.double()
    ref = lr.backward(s, s.proj[0], d, torch.zeros_like(d))
    lr.check(dX[order], *ref[0], c.dtype, "dX")
    check_grads(c, grads, [ref])


@pytest.mark.parametrize("accumulate", [False, True])
def test_gradients_in_several_launches(accumulate):
    """2^20 columns of X are 4096 column tiles, times 4200 LoRAs more workgroups than one launch holds."""
    n, h_in, h_out, rank, P = 5, 1 << 20, 8, 8, 4200
    c = lr.Layer(6, "bf16", n, h_in, h_out, rank, 3, "none", 1, None, False)
    used = [0, 4099, 4199]
    at = [0] * P
    for lora, rows in zip(used, (2, 1, 2)):
        at[lora] = rows
    seg = [0]
    for rows in at:
        seg.append(seg[-1] + rows)
    table = lambda ts: sg.pointer_list([ts[used.index(k)] if k in used else None for k in range(P)])  # noqa: E731
    p = c.proj[0]
    problem = sg.make_problem("bf16", n, h_in, h_out, rank, P, P, 2)
    ws = sg.new_layer_workspace(problem, sg.SGMV_DENSE_BACKWARD)
    dA, dB = ([torch.full_like(t, 2.0 if accumulate else float("nan")) for t in p[k]] for k in "AB")
    spare = torch.full_like(p["A"][0], 7.0)             # of a LoRA without rows, in another launch than the first
    grad = [dA[used.index(k)] if k in used else spare if k == 4150 else None for k in range(P)]
    sg.sgmv_dense_lora_backward(problem, c.X, p["W"], (table(p["A"]), table(p["B"])), c.dY, i32(seg), i32(list(range(P))), ws,
                                grad=(None, sg.pointer_list(grad), table(dB)), accumulate=accumulate)
    c.seg, c.ids = [0, 2, 3, 5], [0, 1, 2]
    d = c.dY.double()
    _, rA, rB, _ = lr.backward(c, p, d, torch.zeros_like(d), train_w=False)
    for k in range(3):
        for got, (ref, bound), what in ((dA[k], rA[k], "dA"), (dB[k], rB[k], "dB")):
            old = 2.0 if accumulate else 0.0
            lr.check(got, ref + old, bound + lr.U * (ref.abs() + old), c.dtype, f"{what}[{k}]")
    assert (spare == (7.0 if accumulate else 0.0)).all()
