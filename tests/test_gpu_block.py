"""A block of a model as a user runs it on these calls, forward and backward: layer norm, the tokens sorted by the adapters that a
router chose, an up projection with bias and gelu, a down projection with bias, back to the tokens' order with the router's
weights and the residual.  Every stage is checked from the 16-bit values that the stage before it left, against 64 bits within the bounds of the
operators' own tests; the whole step is captured once and every replay equals the eager step bit for bit."""
import numpy as np
import pytest
import torch

import segmented_gather_matvec_amd as sg
from tests import layer_reference as lr
from tests import test_gpu_act as ta
from tests import test_gpu_norm as tn
from tests import test_gpu_route as tr

pytestmark = pytest.mark.gpu
u = 2.0 ** -24


class Block:
    """Weights, inputs and every buffer of one step."""

    def __init__(self, seed, dtype, n, k, h, f, rank, P):
        self.name, self.dtype = dtype, {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
        self.n, self.k, self.h, self.f, self.rank, self.P, self.m = n, k, h, f, rank, P, n * k
        self.norm = tn.Case(seed, dtype, n, h)
        rng = np.random.default_rng(seed)
        self.ids = torch.from_numpy(rng.integers(-1, P, size=(n, k)).astype(np.int32)).cuda()   # some choices have none
        self.weights = torch.from_numpy(rng.dirichlet(np.ones(k), size=n).astype(np.float32)).cuda()
        # Two layers' weights and adapters in the reference's form; rows, segments and gradients are filled in below.
        self.up = lr.Layer(seed + 1, dtype, self.m, h, f, rank, P, "none", 1, None, True)
        self.down = lr.Layer(seed + 2, dtype, self.m, f, h, rank, P, "none", 1, None, False)
        g = torch.Generator().manual_seed(seed + 3)
        self.bias = [torch.randn(w, generator=g).to(self.dtype).cuda() for w in (f, h)]
        self.dY = torch.randn(n, h, generator=g).to(self.dtype).cuda()
        e = lambda *s, t=self.dtype: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
        i = lambda s: torch.full((s,), -7, dtype=torch.int32, device="cuda")  # noqa: E731
        m, f32 = self.m, torch.float32
        self.buf = {"N": e(n, h), "mean": e(n, t=f32), "rstd": e(n, t=f32), "perm": i(m), "slots": i(m), "seg": i(P + 1), "idx": i(P),
                    "Xs": e(m, h), "Z": e(m, f), "H": e(m, f), "Ys": e(m, h), "Y": e(n, h),
                    "dYs": e(m, h), "dw": e(n, k, t=f32), "dH": e(m, f), "dXs": e(m, h), "dN": e(n, h), "dX": e(n, h),
                    "dgamma": e(h), "dbeta": e(h), "db0": e(f), "db1": e(h)}
        self.grads = []
        for i, c in enumerate((self.up, self.down)):
            p = c.proj[0]
            self.grads.append((e(*p["W"].shape), [torch.full_like(t, float("nan")) for t in p["A"]],
                               [torch.full_like(t, float("nan")) for t in p["B"]]))
        problem = lambda a, b: sg.make_problem(dtype, m, a, b, rank, P, P, m)  # noqa: E731
        self.problems = [problem(h, f), problem(f, h)]
        self.tables = [(sg.pointer_list(c.proj[0]["A"]), sg.pointer_list(c.proj[0]["B"])) for c in (self.up, self.down)]
        self.grad_args = [(W, sg.pointer_list(A), sg.pointer_list(B)) for W, A, B in self.grads]
        self.ws = {"route": sg.new_route_workspace(n, k, P), "norm": sg.new_layer_norm_workspace(n, h)}
        for i, p in enumerate(self.problems):
            self.ws[f"f{i}"] = sg.new_layer_workspace(p, sg.SGMV_DENSE_ACT_FORWARD)
            self.ws[f"b{i}"] = sg.new_layer_workspace(p, sg.SGMV_DENSE_ACT_BACKWARD)

    def outputs(self):
        return list(self.buf.values()) + [t for W, A, B in self.grads for t in [W] + A + B]

    def step(self):
        b, w, c = self.buf, self.ws, self.norm
        (Wu, Wd), (Au, Bu), (Ad, Bd) = [x.proj[0]["W"] for x in (self.up, self.down)], *self.tables
        su = self.up.proj[0]["scales"]
        sg.sgmv_layer_norm_apply(c.X, c.gamma, c.beta, b["N"], c.eps, mean=b["mean"], rstd=b["rstd"])
        sg.sgmv_route_rows(self.ids, self.P, b["perm"], b["slots"], b["seg"], b["idx"], w["route"])
        sg.sgmv_dispatch_rows(b["N"], b["slots"], b["Xs"])
        sg.sgmv_dense_act_lora_apply(self.problems[0], b["Xs"], Wu, (Au, Bu, b["H"], None, su), b["seg"], b["idx"], w["f0"],
                                     act=sg.SGMV_ACT_GELU_TANH, bias=self.bias[0], Z=b["Z"])
        sg.sgmv_dense_act_lora_apply(self.problems[1], b["H"], Wd, (Ad, Bd, b["Ys"]), b["seg"], b["idx"], w["f1"], bias=self.bias[1])
        sg.sgmv_combine_rows(b["Ys"], b["slots"], b["Y"], weights=self.weights, residual=c.X)

        sg.sgmv_combine_rows_backward(self.dY, b["Ys"], b["slots"], weights=self.weights, dYs=b["dYs"], dweights=b["dw"])
        sg.sgmv_dense_act_lora_backward(self.problems[1], b["H"], Wd, (Ad, Bd), b["dYs"], b["seg"], b["idx"], w["b1"], dX=b["dH"],
                                        grad=self.grad_args[1], dbias=b["db1"])
        sg.sgmv_dense_act_lora_backward(self.problems[0], b["Xs"], Wu, (Au, Bu, None, None, su), b["dH"], b["seg"], b["idx"], w["b0"],
                                        act=sg.SGMV_ACT_GELU_TANH, Z=b["Z"], dX=b["dXs"], grad=self.grad_args[0], dbias=b["db0"])
        sg.sgmv_combine_rows(b["dXs"], b["slots"], b["dN"])
        sg.sgmv_layer_norm_backward(c.X, c.gamma, b["mean"], b["rstd"], b["dN"], w["norm"], dX=b["dX"], beyond=self.dY,
                                    dgamma=b["dgamma"], dbeta=b["dbeta"])


SHAPES = [("bf16", 1, 2, 136, 264, 16, 3), ("f16", 37, 1, 264, 520, 32, 5), ("bf16", 150, 2, 520, 1032, 16, 6),
          ("f16", 700, 3, 264, 1032, 64, 40), ("bf16", 1500, 2, 1024, 1376, 8, 8)]


@pytest.mark.parametrize("dtype,n,k,h,f,rank,P", SHAPES)
def test_every_stage_of_a_step(dtype, n, k, h, f, rank, P):
    t = Block(n, dtype, n, k, h, f, rank, P)
    for w in t.ws.values():
        if w.numel():
            w.fill_(0xFF)
    t.step()
    b, c = t.buf, t.norm
    for key, (ref, bound) in zip(("N", "mean", "rstd"), c.ref_forward()):
        tn.check(b[key], ref, bound, key)
    perm, slots, seg = tr.expected(t.ids, P)
    assert np.array_equal(b["perm"].cpu().numpy(), perm) and np.array_equal(b["slots"].cpu().numpy(), slots)
    assert np.array_equal(b["seg"].cpu().numpy(), seg) and np.array_equal(b["idx"].cpu().numpy(), np.arange(P))
    at = b["slots"].long().reshape(n, k)
    assert torch.equal(b["Xs"][at.reshape(-1)], b["N"].repeat_interleave(k, 0))

    for i, (layer, x, z, y, act) in enumerate(((t.up, "Xs", "Z", "H", "gelu_tanh"), (t.down, "H", None, "Ys", "none"))):
        layer.X, layer.seg, layer.ids = b[x], seg.tolist(), list(range(P))
        e = ta.Extra(layer, bias=False, residual=False)
        e.bias = t.bias[i]
        (ry, ey), (rz, ez) = ta.ref(layer, act, e)
        lr.check(b[y], ry, ey, t.dtype, y)
        if z:
            lr.check(b[z], rz, ez, t.dtype, z)
    terms = t.weights.double()[:, :, None] * b["Ys"].double()[at]
    tr.check(b["Y"], terms.sum(1) + c.X.double(), (k + 1) * u * (terms.abs().sum(1) + c.X.double().abs()), "Y")

    dy = t.dY.double()
    want = (t.weights.double()[:, :, None] * dy[:, None, :]).reshape(-1, h)
    tr.check(b["dYs"][at.reshape(-1)], want, u * want.abs(), "dYs")
    products = dy[:, None, :] * b["Ys"].double()[at]
    tr.check(b["dw"], products.sum(2), (h // 64 + 32) * u * products.abs().sum(2), "dw")
    for i, (layer, d, x, db, act) in enumerate(((t.up, "dH", "dXs", "db0", "gelu_tanh"), (t.down, "dYs", "dH", "db1", "none"))):
        layer.dY, layer.proj[0]["G"] = b[d], b["Z"]
        W, A, B = t.grads[i]
        ta.check_back(layer, act, (b[x], [(W, A, B, None)], b[db]), name=d)
    dn = b["dXs"].double()[at]
    tr.check(b["dN"], dn.sum(1), (k + 1) * u * dn.abs().sum(1), "dN")
    c.dY, c.beyond = b["dN"], t.dY
    for key, (ref, bound) in zip(("dX", "dgamma", "dbeta"), c.ref_backward(b["mean"], b["rstd"])):
        tn.check(b[key], ref, bound, key)


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[2], SHAPES[3]], ids=str)
def test_a_captured_step_repeats(shape):
    dtype, n, k, h, f, rank, P = shape
    t = Block(7, dtype, n, k, h, f, rank, P)
    t.step()
    want = [x.clone() for x in t.outputs()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        t.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.step()
    for _ in range(3):
        for x in t.outputs():
            x.fill_(-7 if x.dtype == torch.int32 else float("nan"))
        for w in t.ws.values():
            if w.numel():
                w.fill_(0xFF)
        graph.replay()
        t.norm.forward()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(t.outputs(), want)):
            assert torch.equal(a, b), f"output {i}"
    # Another routing through the same graph.
    t.ids.copy_((t.ids + 1) % P)
    graph.replay()
    got = [x.clone() for x in t.outputs()]
    t.step()
    assert all(torch.equal(a, b) for a, b in zip(got, t.outputs()))
