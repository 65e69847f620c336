"""The backward pass of a layer with an activation from a stored Z that holds infinities (an fp16 Z beyond 65504 is stored as
one) and NaN: slopes of 0 and 1 at the infinities, a NaN in its own column of dbias and its own row of dX, every other row as
before, bit for bit.  Widths either side of those at which whole rows are one workgroup's, few rows (dZ in two halves) and many."""
import pytest
import torch

from tests import layer_reference as lr
from tests.test_gpu_act import ACTS, check_back, run_back

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,h_out", [(7, 264), (150, 264), (140, 4104), (9, 16392), (135, 16392)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", sorted(set(ACTS) - {"none"}))
def test_infinite_and_missing_values(act, dtype, n, h_out):
    c = lr.Layer(n + h_out, dtype, n, 72, h_out, 8, 1, "none", 1, None, False)
    Z = c.proj[0]["G"]
    before = run_back(c, dtype, act)[0]
    far = Z.clone()
    far[1, 5], far[1, h_out - 1] = float("inf"), float("-inf")
    far[3, ::2], far[3, 1::2] = float("-inf"), float("inf")
    # Slopes at the infinities are those of 2^10 and -2^10 (silu's and gelu's have long been 1 and 0 there).
    c.proj[0]["G"] = far.clamp(-1024.0, 1024.0)
    same = run_back(c, dtype, act)
    check_back(c, act, same)
    c.proj[0]["G"] = far
    dX, grads, db = run_back(c, dtype, act)
    assert torch.equal(dX, same[0]) and torch.equal(db, same[2]) and torch.equal(grads[0][0], same[1][0][0])
    rows = [i for i in range(n) if i not in (1, 3)]
    assert torch.equal(dX[rows], before[rows])
    far[2, 7], far[2, h_out - 3] = float("nan"), float("nan")
    dX, _, db = run_back(c, dtype, act)
    hit = torch.zeros(h_out, dtype=torch.bool, device="cuda")
    hit[7] = hit[h_out - 3] = True
    assert torch.equal(db.isnan(), hit) and torch.equal(db[~hit], same[2][~hit])
    assert dX[2].isnan().all()
    rows = [i for i in range(n) if i != 2]
    assert torch.equal(dX[rows], same[0][rows])
