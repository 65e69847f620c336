"""Host side of the layer entry points: struct layouts, refusals before any launch, workspace sizes, and the
binding's shape checks.  No GPU: every call here is refused, or has nothing to do."""
import ctypes
import os
import re

import pytest
import torch

import segmented_gather_matvec_amd as sg

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "sgmv.h")
FAKE = ctypes.c_void_p(0x10000)
OPS = (sg.SGMV_DENSE_FORWARD, sg.SGMV_DENSE_BACKWARD, sg.SGMV_GATED_FORWARD, sg.SGMV_GATED_BACKWARD)


def good(**kw):
    d = dict(dtype="f16", n_rows=40, h_in=128, h_out=256, rank=16, num_loras=4, num_segs=3, max_seg_len=20)
    d.update(kw)
    return sg.make_problem(**d)


def test_grad_struct_layout_matches_header():
    src = open(HEADER).read()
    body = re.search(r"typedef struct sgmv_projection_grad \{(.*?)\} sgmv_projection_grad_t;", src, re.S).group(1)
    fields = re.findall(r"(\w+);", re.sub(r"/\*.*?\*/", "", body, flags=re.S))
    assert fields == [n for n, _ in sg.sgmv_projection_grad_t._fields_]
    assert ctypes.sizeof(sg.sgmv_projection_grad_t) == 8 * len(fields)
    for enum, names in (("sgmv_act", ("SGMV_ACT_SILU", "SGMV_ACT_GELU_TANH")),
                        ("sgmv_layer_op", ("SGMV_DENSE_FORWARD", "SGMV_DENSE_BACKWARD", "SGMV_GATED_FORWARD",
                                           "SGMV_GATED_BACKWARD"))):
        body = re.search(r"typedef enum %s \{(.*?)\} %s_t;" % (enum, enum), src, re.S).group(1)
        found = dict(re.findall(r"(SGMV_\w+) = (\d+)", body))
        assert {n: int(found[n]) for n in names} == {n: getattr(sg, n) for n in names}


class Raw:
    """The four C calls with fake pointers: only refusals may come back."""

    def __init__(self, problem):
        self.p = problem

    def call(self, op, ws_bytes=None, **kw):
        lib = sg.load_library()
        a = dict(X=FAKE, W=FAKE, W2=FAKE, Y=0x10000, Y2=0x10000, A=0x10000, B=0x10000, ranks=None, scales=None, act=0,
                 H=FAKE, dY=FAKE, dX=FAKE, dW=None, dA=None, dB=None, acc=0, seg=FAKE, ids=FAKE, ws=FAKE)
        a.update(kw)
        pj = sg.sgmv_projection_t(a["A"], a["B"], a["Y"], a["ranks"], a["scales"])
        pk = sg.sgmv_projection_t(a["A"], a["B"], a["Y2"], a["ranks"], a["scales"])
        g = sg.sgmv_projection_grad_t(a["dW"], a["dA"], a["dB"])
        p = ctypes.byref(self.p)
        n = ws_bytes if ws_bytes is not None else 1 << 40
        tail = (a["seg"], a["ids"], a["ws"], n, None)
        if op == sg.SGMV_DENSE_FORWARD:
            return lib.sgmv_dense_lora_apply(p, a["X"], a["W"], ctypes.byref(pj), *tail)
        if op == sg.SGMV_GATED_FORWARD:
            return lib.sgmv_gated_lora_apply(p, a["X"], a["W"], a["W2"], ctypes.byref(pj), ctypes.byref(pk), a["act"],
                                             a["H"], *tail)
        if op == sg.SGMV_DENSE_BACKWARD:
            return lib.sgmv_dense_lora_backward(p, a["X"], a["W"], ctypes.byref(pj), a["dY"], a["dX"], ctypes.byref(g),
                                                a["acc"], *tail)
        return lib.sgmv_gated_lora_backward(p, a["X"], a["W"], a["W2"], ctypes.byref(pj), ctypes.byref(pk), a["act"],
                                            a["dY"], a["dX"], ctypes.byref(g), ctypes.byref(g), a["acc"], *tail)


ODD = ctypes.c_void_p(0x10004)
COMMON = [
    (dict(X=None), sg.SGMV_ERR_INVALID_ARG), (dict(W=None), sg.SGMV_ERR_INVALID_ARG),
    (dict(A=None), sg.SGMV_ERR_INVALID_ARG), (dict(B=None), sg.SGMV_ERR_INVALID_ARG),
    (dict(seg=None), sg.SGMV_ERR_INVALID_ARG), (dict(ids=None), sg.SGMV_ERR_INVALID_ARG),
    (dict(X=ODD), sg.SGMV_ERR_UNSUPPORTED), (dict(W=ODD), sg.SGMV_ERR_UNSUPPORTED),
    (dict(A=0x10004), sg.SGMV_ERR_UNSUPPORTED), (dict(B=0x10004), sg.SGMV_ERR_UNSUPPORTED),
    (dict(ranks=0x10002), sg.SGMV_ERR_UNSUPPORTED), (dict(scales=0x10001), sg.SGMV_ERR_UNSUPPORTED),
    (dict(seg=ctypes.c_void_p(0x10002)), sg.SGMV_ERR_UNSUPPORTED),
    (dict(ws=None), sg.SGMV_ERR_WORKSPACE), (dict(ws=ODD), sg.SGMV_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("kw,status", COMMON)
def test_refusals_of_every_entry_point(op, kw, status):
    assert Raw(good()).call(op, **kw) == status


@pytest.mark.parametrize("op,kw,status", [
    (sg.SGMV_DENSE_FORWARD, dict(Y=None), sg.SGMV_ERR_INVALID_ARG),
    (sg.SGMV_DENSE_FORWARD, dict(Y=0x10008), sg.SGMV_ERR_UNSUPPORTED),
    (sg.SGMV_GATED_FORWARD, dict(H=None), sg.SGMV_ERR_INVALID_ARG),
    (sg.SGMV_GATED_FORWARD, dict(H=ODD), sg.SGMV_ERR_UNSUPPORTED),
    (sg.SGMV_GATED_FORWARD, dict(W2=None), sg.SGMV_ERR_INVALID_ARG),
    (sg.SGMV_GATED_FORWARD, dict(act=2), sg.SGMV_ERR_INVALID_ARG),
    (sg.SGMV_GATED_FORWARD, dict(act=-1), sg.SGMV_ERR_INVALID_ARG),
    (sg.SGMV_DENSE_BACKWARD, dict(dY=None), sg.SGMV_ERR_INVALID_ARG),
    (sg.SGMV_DENSE_BACKWARD, dict(dY=ODD), sg.SGMV_ERR_UNSUPPORTED),
    (sg.SGMV_DENSE_BACKWARD, dict(dX=ODD), sg.SGMV_ERR_UNSUPPORTED),
    (sg.SGMV_DENSE_BACKWARD, dict(dW=0x10008), sg.SGMV_ERR_UNSUPPORTED),
    (sg.SGMV_DENSE_BACKWARD, dict(dA=0x10004), sg.SGMV_ERR_UNSUPPORTED),
    (sg.SGMV_DENSE_BACKWARD, dict(acc=2), sg.SGMV_ERR_INVALID_ARG),
    (sg.SGMV_GATED_BACKWARD, dict(Y=None), sg.SGMV_ERR_INVALID_ARG),
    (sg.SGMV_GATED_BACKWARD, dict(Y2=None), sg.SGMV_ERR_INVALID_ARG),
    (sg.SGMV_GATED_BACKWARD, dict(act=7), sg.SGMV_ERR_INVALID_ARG),
    (sg.SGMV_GATED_BACKWARD, dict(acc=-1), sg.SGMV_ERR_INVALID_ARG),
])
def test_refusals_of_one_entry_point(op, kw, status):
    assert Raw(good()).call(op, **kw) == status


@pytest.mark.parametrize("op", OPS)
def test_workspace_is_checked_to_the_byte(op):
    p = good()
    need = sg.sgmv_layer_workspace_bytes(p, op)
    assert need > 0
    assert Raw(p).call(op, ws_bytes=need - 1) == sg.SGMV_ERR_WORKSPACE


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("kw", [dict(rank=24), dict(h_in=4), dict(h_out=1 << 21), dict(n_rows=-1), dict(dtype=2)])
def test_bad_problems(op, kw):
    p = good(**kw)
    assert Raw(p).call(op) == sg.sgmv_check_problem(p) != sg.SGMV_OK
    with pytest.raises(sg.SgmvError):
        sg.sgmv_layer_workspace_bytes(p, op)


@pytest.mark.parametrize("op", OPS)
def test_rows_beyond_the_tiles_reach(op):
    most = int(re.search(r"#define SGMV_MAX_LAYER_ROWS \(1 << (\d+)\)", open(HEADER).read()).group(1))
    kw = dict(h_in=8, h_out=8, num_segs=0, max_seg_len=0)
    assert sg.sgmv_layer_workspace_bytes(good(n_rows=1 << most, **kw), op) >= 0
    p = good(n_rows=(1 << most) + 1, **kw)
    assert sg.sgmv_check_problem(p) == sg.SGMV_OK
    assert Raw(p).call(op) == sg.SGMV_ERR_UNSUPPORTED
    with pytest.raises(sg.SgmvError):
        sg.sgmv_layer_workspace_bytes(p, op)


def test_workspace_arguments():
    lib = sg.load_library()
    out = ctypes.c_size_t(0)
    assert lib.sgmv_layer_workspace_bytes(ctypes.byref(good()), 4, ctypes.byref(out)) == sg.SGMV_ERR_INVALID_ARG
    assert lib.sgmv_layer_workspace_bytes(ctypes.byref(good()), -1, ctypes.byref(out)) == sg.SGMV_ERR_INVALID_ARG
    assert lib.sgmv_layer_workspace_bytes(ctypes.byref(good()), 0, None) == sg.SGMV_ERR_INVALID_ARG


def test_no_rows_forward_does_nothing():
    p = good(n_rows=0, num_segs=0, max_seg_len=0)
    for op in (sg.SGMV_DENSE_FORWARD, sg.SGMV_GATED_FORWARD):
        assert Raw(p).call(op, X=None, ws=None, ws_bytes=0, seg=None, ids=None) == sg.SGMV_OK


@pytest.mark.parametrize("op", OPS)
def test_workspace_stays_sane_over_sizes(op):
    """Sizes never go negative or wild, and the largest problems' splits stay within a fixed memory budget."""
    for n in (0, 1, 31, 129, 4097, 1 << 20):
        for h_in, h_out in ((8, 8), (4096, 11008), (11008, 4096), (1 << 20, 8)):
            for P, S in ((1, 1), (64, 64), (5000, 300)):
                S = min(S, n)
                p = good(n_rows=n, h_in=h_in, h_out=h_out, rank=64, num_loras=P, num_segs=S, max_seg_len=-(-n // S) if S else 0)
                size = sg.sgmv_layer_workspace_bytes(p, op)
                planes = 16 * 2 * n * max(h_in, h_out) * 4
                assert 0 <= size <= planes + 4 * n * max(h_in, h_out) + 64 * n * 64 * 4 * 8 + (600 << 20)


def test_binding_checks_shapes_and_devices():
    p = good()
    X, W, Y = torch.zeros(40, 128).half(), torch.zeros(128, 256).half(), torch.zeros(40, 256).half()
    with pytest.raises(ValueError, match="device tensor"):
        sg.sgmv_dense_lora_apply(p, X, W, (None, None, Y), None, None, None)
    for t, kw, why in ((torch.zeros(40, 120), dict(shape=(40, 128)), r"must be \[40, 128\], got \[40, 120\]"),
                       (torch.zeros(3), dict(least=4), "must hold 4 entries, got 3"),
                       (torch.zeros(3).half(), dict(least=3), "must be torch.float32"),
                       (torch.zeros(4, 4).t()[:, :2], dict(shape=(4, 2)), "must be contiguous")):
        class OnDevice(torch.Tensor):
            is_cuda = True
            get_device = lambda self: 0  # noqa: E731
        with pytest.raises(ValueError, match="T " + why):
            sg._layer_ptr(t.as_subclass(OnDevice), "T", 0, torch.float32, **kw)


def test_binding_refuses_tensors_of_two_devices():
    class On:
        is_cuda = True

        def __init__(self, index):
            self.index, self.device = index, torch.device("cuda", index)

        def get_device(self):
            return self.index

    with pytest.raises(ValueError, match="W must be on X's device, is on cuda:0"):
        sg._layer_ptr(On(0), "W", 1, torch.float16)
