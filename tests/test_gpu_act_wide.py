"""GPU parity of the layer with an activation at sizes whose outputs, or dX, are written by 128 x 256 tiles, with and without the LoRA
term in them, and at sizes whose splits share the term (tests/test_act_plans.py checks that they are)."""
import pytest

from tests import layer_reference as lr
from tests.test_gpu_act import Extra, check_back, ref, run, run_back

pytestmark = pytest.mark.gpu

# rows, h_in, h_out, rank, segments (0: no LoRAs)
FORWARD = [(600, 1032, 11008, 64, 4), (1300, 264, 5128, 16, 0), (300, 520, 11016, 32, 4), (1800, 136, 4104, 8, 4), (700, 136, 9000, 8, 4)]
# Few rows, whose contraction is split and whose splits share the LoRA term's segments (more splits than segments in the last).
SHARED = [(132, 6224, 11080, 64, 11), (132, 4104, 8200, 32, 11), (200, 4104, 5128, 16, 4), (130, 8200, 4104, 64, 1), (140, 4104, 20008, 64, 140)]
BACKWARD = [(1300, 5128, 1032, 64, 4), (1300, 5128, 264, 16, 0), (600, 11008, 520, 32, 4)]


def layer(case, dtype):
    n, h_in, h_out, rank, segs = case
    layout = "none" if segs == 0 else "uncovered"
    return lr.Layer(n + h_in, dtype, n, h_in, h_out, rank, 4, layout, 1, None, segs > 0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", FORWARD, ids=str)
def test_forward(case, dtype):
    c = layer(case, dtype)
    e = Extra(c)
    for g, r, what in zip(run(c, dtype, "gelu_tanh", e), ref(c, "gelu_tanh", e), "YZ"):
        lr.check(g, *r, c.dtype, what)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", SHARED, ids=str)
def test_shared_term(case, dtype):
    n, h_in, h_out, rank, segs = case
    c = lr.Layer(n + h_in, dtype, n, h_in, h_out, rank, 4, {11: "mixed", 4: "uncovered", 1: "one", 140: "distinct"}[segs], 1, None, True)
    assert len(c.ids) == segs
    e = Extra(c)
    for g, r, what in zip(run(c, dtype, "silu", e), ref(c, "silu", e), "YZ"):
        lr.check(g, *r, c.dtype, what)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", BACKWARD, ids=str)
def test_backward(case, dtype):
    c = layer(case, dtype)
    check_back(c, "silu", run_back(c, dtype, "silu"))
