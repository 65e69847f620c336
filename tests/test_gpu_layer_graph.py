"""What a layer call writes, seen by tests that would notice a call that wrote nothing, or too much: every output and both
workspaces are overwritten before each replay of a captured step, and the gradients of all LoRAs lie in one buffer of
sentinels of which the unwanted ones must keep theirs."""
import pytest
import torch

import segmented_gather_matvec_amd as sg
from tests.test_gpu_layer import Call, case, run_dense, run_gated, run_gated_back

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["one_row_r8", "distinct_r16", "several_tiles", "uncovered_r64"])
def test_every_replay_writes_every_output(name):
    c, dtype = case(name, 2)
    H, G, U = run_gated(c, dtype, 0)
    c.proj[0]["G"], c.proj[1]["G"] = G, U
    dX, grads = run_gated_back(c, dtype, 0)
    want = [H, G, U, dX] + [t for g in grads for t in [g[0]] + g[1] + g[2]]

    fwd, bwd = Call(c, sg.SGMV_GATED_FORWARD, dtype), Call(c, sg.SGMV_GATED_BACKWARD, dtype)
    H2, G2, U2, dX2 = (torch.empty_like(t) for t in (H, G, U, dX))
    new = bwd.grads()
    outputs = [H2, G2, U2, dX2] + [t for g in new for t in [g[0]] + g[1] + g[2]]
    W = [p["W"] for p in c.proj]

    def step():
        sg.sgmv_gated_lora_apply(fwd.problem, c.X, W[0], W[1], fwd.projection(0, G2), fwd.projection(1, U2), H2, fwd.seg,
                                 fwd.ids, fwd.ws)
        sg.sgmv_gated_lora_backward(bwd.problem, c.X, W[0], W[1], bwd.projection(0, G2), bwd.projection(1, U2), c.dY,
                                    bwd.seg, bwd.ids, bwd.ws, dX=dX2, gate_grad=new[0][3], up_grad=new[1][3])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        for t in outputs:
            t.fill_(float("nan"))
        for ws in (fwd.ws, bwd.ws):
            ws.fill_(0xFF)
        graph.replay()
        run_dense(c, dtype)             # the program's own eager work between replays
        torch.cuda.synchronize()
        for i, (got, ref) in enumerate(zip(outputs, want)):
            assert torch.equal(got, ref), f"output {i}"


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("name", ["mixed_r32", "uncovered", "several_tiles"])
def test_null_entries_and_neighbours_keep_their_values(name, accumulate):
    """Gradients of all LoRAs side by side in one buffer; the first LoRA with rows and the last one are not wanted."""
    c, dtype = case(name, 2)
    _, grads = run_gated_back(c, dtype, 0, accumulate=accumulate, fill=7.0)
    unwanted = {c.pieces[0][2], c.P - 1}
    call = Call(c, sg.SGMV_GATED_BACKWARD, dtype)
    for part, shape in ((1, (c.h_in, c.rank)), (2, (c.rank, c.h_out))):
        buffer = torch.full((c.P + 2, *shape), 7.0, dtype=c.dtype, device="cuda")     # one more at either end
        tables = sg.pointer_list([None if k in unwanted else buffer[k + 1] for k in range(c.P)])
        grad = (None, tables, None) if part == 1 else (None, None, tables)
        sg.sgmv_gated_lora_backward(call.problem, c.X, c.proj[0]["W"], c.proj[1]["W"], call.projection(0, c.proj[0]["G"]),
                                    call.projection(1, c.proj[1]["G"]), c.dY, call.seg, call.ids, call.ws,
                                    gate_grad=grad, accumulate=accumulate)
        assert (buffer[0] == 7.0).all() and (buffer[-1] == 7.0).all()
        for k in range(c.P):
            if k in unwanted:
                assert (buffer[k + 1] == 7.0).all(), f"LoRA {k} was not wanted"
            else:
                assert torch.equal(buffer[k + 1], grads[0][part][k])
