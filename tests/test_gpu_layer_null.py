"""A null A_k or B_k of a LoRA with rows counts as rank 0 in every layer call: its rows get the shared projection alone,
whatever the other matrix holds, and neither of its gradients is written."""
import pytest
import torch

import segmented_gather_matvec_amd as sg
from tests import layer_reference as lr
from tests.test_gpu_layer import Call

pytestmark = pytest.mark.gpu


def without(c, k, lacks):
    """Tables of c in which LoRA k lacks A or B and the matrix it has is full of infinities."""
    call = {op: Call(c, op, "f16" if c.dtype == torch.float16 else "bf16") for op in range(4)}
    tables = []
    for p in c.proj:
        A, B = list(p["A"]), list(p["B"])
        if lacks == "A":
            A[k], B[k] = None, torch.full_like(B[k], float("inf"))
        else:
            A[k], B[k] = torch.full_like(A[k], float("inf")), None
        tables.append((sg.pointer_list(A), sg.pointer_list(B), A, B))
    return call, tables


# Terms added by the epilogue and by the tiles, gradients with and without row splits, by segment and by LoRA
SIZES = {"few": ("f16", 19, 136, 264, 16, 3), "tiles": ("bf16", 300, 264, 520, 64, 3), "splits": ("f16", 2000, 136, 264, 8, 2),
         "by_segment": ("bf16", 2000, 136, 264, 8, 7)}


@pytest.mark.parametrize("lacks", ["A", "B"])
@pytest.mark.parametrize("size", sorted(SIZES))
def test_a_lora_that_lacks_a_matrix(size, lacks):
    dtype, n, h_in, h_out, rank, P = SIZES[size]
    c = lr.Layer(17, dtype, n, h_in, h_out, rank, P, "none", 2, None, True)
    a, b = n // 3, n // 2
    c.seg, c.ids = [0, a, b, n], [0, 1, 0]
    call, tables = without(c, 1, lacks)
    W = [p["W"] for p in c.proj]

    ref = lr.Layer(17, dtype, n, h_in, h_out, rank, P, "none", 2, None, True)
    ref.seg, ref.ids = c.seg, c.ids
    for p in ref.proj:                  # the same by a pair of zeros
        p["A"][1].zero_()
        p["B"][1].zero_()

    def proj(i, Y):
        return (tables[i][0], tables[i][1], Y, None, c.proj[i]["scales"])

    Y = call[0].nan(n, h_out)
    sg.sgmv_dense_lora_apply(call[0].problem, c.X, W[0], proj(0, Y), call[0].seg, call[0].ids, call[0].ws)
    lr.check(Y, *lr.project(ref, ref.proj[0]), c.dtype, "Y")
    H, G, U = (call[2].nan(n, h_out) for _ in range(3))
    sg.sgmv_gated_lora_apply(call[2].problem, c.X, W[0], W[1], proj(0, G), proj(1, U), H, call[2].seg, call[2].ids, call[2].ws)
    for got, (want, bound), what in zip((H, G, U), lr.gate(ref, 0), "HGU"):
        lr.check(got, want, bound, c.dtype, what, rounded=True)

    for accumulate in (False, True):
        dX, grads = call[3].nan(n, h_in), call[3].grads(False, fill=3.0)
        sg.sgmv_gated_lora_backward(call[3].problem, c.X, W[0], W[1], proj(0, c.proj[0]["G"]), proj(1, c.proj[1]["G"]), c.dY,
                                    call[3].seg, call[3].ids, call[3].ws, dX=dX, gate_grad=grads[0][3],
                                    up_grad=grads[1][3], accumulate=accumulate)
        refs = [lr.backward(ref, p, *d, train_w=False) for p, d in zip(ref.proj, lr.gate_backward(ref, 0))]
        lr.check(dX, refs[0][0][0] + refs[1][0][0], refs[0][0][1] + refs[1][0][1], c.dtype, "dX")
        for i in range(2):
            for part in (1, 2):
                assert (grads[i][part][1] == 3.0).all(), "the gradient of a LoRA that lacks a matrix"
                want, bound = refs[i][part][0]
                if accumulate:
                    want, bound = want + 3.0, bound + lr.U * (want.abs() + 3.0)
                lr.check(grads[i][part][0], want, bound, c.dtype, f"{'AB'[part - 1]}[{i}]")
                for k in range(2, P):   # no rows: zeros, or left alone
                    assert (grads[i][part][k] == (3.0 if accumulate else 0.0)).all()
