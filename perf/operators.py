"""Cases of the layer operators: a shared projection with the adapters of many requests, and the gated
feed-forward block made of two such projections, each with its backward pass.

    y_i  = x_i @ W + s_k (x_i @ A_k) @ B_k          k: the adapter of row i's segment (none: the first term alone)
    h_i  = act(g_i) * u_i                            g, u: two such projections of the same x

Rows are grouped into segments that share an adapter, as everywhere in this library.  Gradients come in the
inputs' format; the gradient of an adapter that no row uses is zero.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _case(name, op, dtype, n, h_in, h_out, rank, adapters, segs, cover=1.0, scales=False, train_w=False, act="silu"):
    return {"name": name, "op": op, "dtype": dtype, "n": n, "h_in": h_in, "h_out": h_out, "rank": rank,
            "adapters": adapters, "segs": segs, "cover": cover, "scales": scales, "train_w": train_w, "act": act}


def listed():
    return [
        # one request decoding one token through an attention projection: latency
        _case("dense_token", "dense", "f16", 1, 4096, 4096, 16, 32, 1),
        # prompts of 8 requests through an attention projection of width 5120, an odd number of rows, some without adapter
        _case("dense_prompts", "dense", "bf16", 2011, 5120, 5120, 64, 8, 8, cover=0.9),
        # long prompts through the up projection of a 4096-wide layer
        _case("dense_long", "dense", "bf16", 8192, 4096, 11008, 16, 16, 16),
        # fine-tuning small adapters of several tenants on a narrow layer, base frozen
        _case("dense_grad_small", "dense_grad", "f16", 203, 1024, 1376, 8, 6, 9, scales=True),
        # a training step of one attention projection, base trained too
        _case("dense_grad_full", "dense_grad", "bf16", 4096, 4096, 4096, 16, 4, 8, scales=True, train_w=True),
        # one request decoding one token through the feed-forward block: streams both weights
        _case("gated_token", "gated", "f16", 1, 4096, 11008, 16, 32, 1),
        # decode batch of 32 requests, each with its own adapter
        _case("gated_decode", "gated", "f16", 32, 4096, 11008, 16, 32, 32),
        # prompts of width 5120, odd rows, rank 64
        _case("gated_prompts", "gated", "bf16", 1777, 5120, 13824, 64, 8, 12, cover=0.95),
        # long prompts
        _case("gated_long", "gated", "bf16", 8192, 4096, 11008, 16, 16, 16),
        # a few short sequences of several tenants, ragged widths, tanh gelu
        _case("gated_grad_small", "gated_grad", "f16", 77, 520, 1048, 8, 5, 7, cover=0.9, scales=True, act="gelu_tanh"),
        # a micro-batch of adapter fine-tuning, base frozen
        _case("gated_grad_adapters", "gated_grad", "bf16", 2048, 4096, 11008, 16, 4, 8, scales=True),
        # the same with the base trained too
        _case("gated_grad_full", "gated_grad", "bf16", 4096, 4096, 11008, 64, 4, 4, train_w=True),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    most = max(_flops(c) for c in listed())
    while True:
        op = rng.choice(["dense", "dense_grad", "gated", "gated_grad"])
        n = _log(rng, 1, 8192)
        h_in, h_out = _log(rng, 256, 5120, 8), _log(rng, 256, 13824, 8)
        adapters = _log(rng, 1, 64)
        segs = min(n, _log(rng, 1, 64))
        c = _case("", op, rng.choice(["f16", "bf16"]), n, h_in, h_out, rng.choice([8, 16, 32, 64]), adapters, segs,
                  cover=rng.choice([1.0, 1.0, 0.9, 0.5]), scales=rng.random() < 0.5,
                  train_w="grad" in op and rng.random() < 0.4, act=rng.choice(["silu", "silu", "gelu_tanh"]))
        del c["name"]
        if _flops(c) <= most:
            return c


def _gated(case):
    return case["op"].startswith("gated")


def _grad(case):
    return case["op"].endswith("grad")


def _flops(case):
    n, k, f, r = case["n"], case["h_in"], case["h_out"], case["rank"]
    rows = int(n * case["cover"])
    per = 2 * n * k * f + 2 * rows * r * (k + f)  # one projection, forward
    if _grad(case):
        # dX and the adapters' four products (V again, dV, dA and dB beside the adapters' part of dX), dW on request
        per = 2 * n * k * f * (2 if case["train_w"] else 1) + 2 * rows * r * (3 * k + 2 * f)
    return per * (2 if _gated(case) else 1)


def work(case):
    n, k, f, r, e = case["n"], case["h_in"], case["h_out"], case["rank"], 2
    two = 2 if _gated(case) else 1
    used = min(case["segs"], case["adapters"])
    weights = two * k * f * e + two * used * r * (k + f) * e
    if not _grad(case):
        outs = n * f * e * (3 if _gated(case) and _keeps(case) else 1)
        return {"bytes": n * k * e + weights + outs, "flops": _flops(case)}
    reads = n * k * e + weights + n * f * e * (3 if _gated(case) else 1)
    writes = n * k * e + two * case["adapters"] * r * (k + f) * e + (two * k * f * e if case["train_w"] else 0)
    return {"bytes": reads + writes, "flops": _flops(case)}


def _keeps(case):
    """Whether the gated forward keeps g and u for a backward pass: prompts do, decoding does not."""
    return case["n"] > 128


def _layout(case, seed):
    """Segment bounds and adapter ids (host): random lengths over the covered rows, adapters in any order, some twice."""
    rng = np.random.default_rng(seed)
    rows = max(1, int(case["n"] * case["cover"]))
    cuts = np.sort(rng.integers(0, rows + 1, size=case["segs"] - 1)) if case["segs"] < rows else np.arange(1, case["segs"])
    indptr = np.concatenate([[0], np.minimum(cuts, rows), [rows]]).astype(np.int32)
    order = np.concatenate([rng.permutation(case["adapters"]) for _ in range(-(-case["segs"] // case["adapters"]))])
    return indptr, order[: case["segs"]].astype(np.int32)


def prepare(case, seed):
    dt, dev = DTYPES[case["dtype"]], "cuda"
    n, k, f, r, P = case["n"], case["h_in"], case["h_out"], case["rank"], case["adapters"]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev).mul_(std).to(dt)

    indptr, ids = _layout(case, seed)
    rows_of = torch.full((n,), -1, dtype=torch.int64)
    rows_of[: int(indptr[-1])] = torch.from_numpy(np.repeat(ids, np.diff(indptr)).astype(np.int64))
    st = {"case": case, "X": normal(n, k), "indptr": torch.from_numpy(indptr).to(dev), "ids": torch.from_numpy(ids).to(dev),
          "rows_of": rows_of.to(dev)}
    for p in ("g", "u") if _gated(case) else ("g",):
        st["W" + p] = normal(k, f, std=k ** -0.5)
        st["A" + p] = normal(P, k, r, std=k ** -0.5)
        st["B" + p] = normal(P, r, f, std=r ** -0.5)
        st["s" + p] = torch.rand(P, generator=gen, device=dev) + 0.5 if case["scales"] else None
        if _gated(case) and _grad(case):
            st["Y" + p] = normal(n, f, std=2 ** 0.5)
    if _grad(case):
        st["dY"] = normal(n, f)
    if own:
        _handles(st)
    return st


# ------------------------------------------------------------------ the plain form

def _mask(st):
    """[n, P * r]: true where column j belongs to the row's adapter."""
    c = st["case"]
    cols = torch.arange(c["adapters"], device="cuda").repeat_interleave(c["rank"])
    return st["rows_of"][:, None] == cols[None, :]


def _flat(st, p):
    """The adapters of projection p side by side, in 32 bits: A [h_in, P r], B [P r, h_out], scales [P r]."""
    c = st["case"]
    A = st["A" + p].float().permute(1, 0, 2).reshape(c["h_in"], -1)
    B = st["B" + p].float().reshape(-1, c["h_out"])
    s = st["s" + p].repeat_interleave(c["rank"]) if st["s" + p] is not None else torch.ones(A.shape[1], device="cuda")
    return A, B, s


def _project(st, p, x, mask):
    A, B, s = _flat(st, p)
    return x @ st["W" + p].float() + torch.where(mask, (x @ A) * s, 0.0) @ B


def _act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return g * sig, sig * (1 + g * (1 - sig))
    c, a = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(c * (g + a * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * a * g * g)


def _project_grads(st, p, x, dy, mask):
    """dX of projection p in 32 bits, and dA [P, h_in, r], dB [P, r, h_out], dW or None, rounded."""
    c = st["case"]
    dt, P, r = DTYPES[c["dtype"]], c["adapters"], c["rank"]
    A, B, s = _flat(st, p)
    v = torch.where(mask, (x @ A) * s, 0.0)
    dv = torch.where(mask, (dy @ B.t()) * s, 0.0)
    dx = dy @ st["W" + p].float().t() + dv @ A.t()
    dA = (x.t() @ dv).reshape(c["h_in"], P, r).permute(1, 0, 2).contiguous().to(dt)
    dB = (v.t() @ dy).reshape(P, r, c["h_out"]).to(dt)
    return dx, {"dA" + p: dA, "dB" + p: dB, **({"dW" + p: (x.t() @ dy).to(dt)} if c["train_w"] else {})}


def _plain(st):
    c = st["case"]
    dt, x, mask = DTYPES[c["dtype"]], st["X"].float(), _mask(st)
    if c["op"] == "dense":
        return {"Y": _project(st, "g", x, mask).to(dt)}
    if c["op"] == "gated":
        g, u = _project(st, "g", x, mask), _project(st, "u", x, mask)
        out = {"H": (_act(g, c["act"])[0] * u).to(dt)}
        return {**out, "G": g.to(dt), "U": u.to(dt)} if _keeps(c) else out
    dy = st["dY"].float()
    if c["op"] == "dense_grad":
        dx, grads = _project_grads(st, "g", x, dy, mask)
        return {"dX": dx.to(dt), **grads}
    value, slope = _act(st["Yg"].float(), c["act"])
    dxg, grads = _project_grads(st, "g", x, dy * st["Yu"].float() * slope, mask)
    dxu, more = _project_grads(st, "u", x, dy * value, mask)
    return {"dX": (dxg + dxu).to(dt), **grads, **more}


# ------------------------------------------------------------------ the framework's calls

def _handles(st):
    """What a program that uses the library keeps: the problem, tables of pointers, outputs, a workspace."""
    import segmented_gather_matvec_amd as sg

    c = st["case"]
    n, k, f = c["n"], c["h_in"], c["h_out"]
    dt = DTYPES[c["dtype"]]
    longest = int((st["indptr"][1:] - st["indptr"][:-1]).max())
    st["problem"] = sg.make_problem(c["dtype"], n, k, f, c["rank"], c["adapters"], c["segs"], longest)
    op = {"dense": sg.SGMV_DENSE_FORWARD, "dense_grad": sg.SGMV_DENSE_BACKWARD, "gated": sg.SGMV_GATED_FORWARD,
          "gated_grad": sg.SGMV_GATED_BACKWARD}[c["op"]]
    st["ws"] = sg.new_layer_workspace(st["problem"], op)
    st["act_code"] = {"silu": sg.SGMV_ACT_SILU, "gelu_tanh": sg.SGMV_ACT_GELU_TANH}[c["act"]]

    def empty(*shape):
        return torch.empty(*shape, dtype=dt, device="cuda")

    out = st["out"] = {}
    if c["op"] == "dense":
        out["Y"] = empty(n, f)
    elif c["op"] == "gated":
        out["H"] = empty(n, f)
        if _keeps(c):
            out["G"], out["U"] = empty(n, f), empty(n, f)
    else:
        out["dX"] = empty(n, k)
    for p in ("g", "u") if _gated(c) else ("g",):
        y = {"dense": out.get("Y"), "gated": out.get("G" if p == "g" else "U")}.get(c["op"], st.get("Y" + p))
        st["proj_" + p] = (sg.pointer_table(st["A" + p]), sg.pointer_table(st["B" + p]), y, None, st["s" + p])
        if _grad(c):
            out["dA" + p], out["dB" + p] = torch.empty_like(st["A" + p]), torch.empty_like(st["B" + p])
            if c["train_w"]:
                out["dW" + p] = empty(k, f)
            st["grad_" + p] = (out.get("dW" + p), sg.pointer_table(out["dA" + p]), sg.pointer_table(out["dB" + p]))


def _called(st):
    import segmented_gather_matvec_amd as sg

    op, out = st["case"]["op"], st["out"]
    if op == "dense":
        sg.sgmv_dense_lora_apply(st["problem"], st["X"], st["Wg"], st["proj_g"], st["indptr"], st["ids"], st["ws"])
    elif op == "gated":
        sg.sgmv_gated_lora_apply(st["problem"], st["X"], st["Wg"], st["Wu"], st["proj_g"], st["proj_u"], out["H"],
                                 st["indptr"], st["ids"], st["ws"], act=st["act_code"])
    elif op == "dense_grad":
        sg.sgmv_dense_lora_backward(st["problem"], st["X"], st["Wg"], st["proj_g"], st["dY"], st["indptr"], st["ids"],
                                    st["ws"], dX=out["dX"], grad=st["grad_g"])
    else:
        sg.sgmv_gated_lora_backward(st["problem"], st["X"], st["Wg"], st["Wu"], st["proj_g"], st["proj_u"], st["dY"],
                                    st["indptr"], st["ids"], st["ws"], dX=out["dX"], gate_grad=st["grad_g"],
                                    up_grad=st["grad_u"], act=st["act_code"])
    return out


def run(state):
    return _called(state) if own else _plain(state)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    """Segment by segment from the definition, in 64 bits; the backward pass by the chain rule on each segment."""
    st = prepare(case, seed)
    c, x = case, st["X"].double()
    bounds, ids = st["indptr"].tolist(), st["ids"].tolist()
    pieces = [(lo, hi, k) for lo, hi, k in zip(bounds[:-1], bounds[1:], ids) if hi > lo]
    names = ("g", "u") if _gated(c) else ("g",)
    W = {p: st["W" + p].double() for p in names}

    def adapter(p, k):
        scale = float(st["s" + p][k]) if st["s" + p] is not None else 1.0
        return st["A" + p][k].double(), st["B" + p][k].double(), scale

    def forward(p):
        y = x @ W[p]
        for lo, hi, k in pieces:
            A, B, s = adapter(p, k)
            y[lo:hi] += s * ((x[lo:hi] @ A) @ B)
        return y

    if c["op"] == "dense":
        return {"Y": forward("g")}
    if c["op"] == "gated":
        g, u = forward("g"), forward("u")
        if c["act"] == "silu":
            h = g * torch.sigmoid(g) * u
        else:
            h = torch.nn.functional.gelu(g, approximate="tanh") * u
        return {"H": h, "G": g, "U": u} if _keeps(c) else {"H": h}
    dy = st["dY"].double()
    if c["op"] == "dense_grad":
        d = {"g": dy}
    else:
        g, u = st["Yg"].double(), st["Yu"].double()
        if c["act"] == "silu":
            e = torch.sigmoid(g)
            value, slope = g * e, e + g * e * torch.sigmoid(-g)
        else:
            z = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
            value = g * torch.sigmoid(2 * z)  # (1 + tanh z) / 2 is the logistic function of 2 z
            slope = torch.sigmoid(2 * z) + g / (2 * torch.cosh(z) ** 2) * math.sqrt(2 / math.pi) * (1 + 0.134145 * g ** 2)
        d = {"g": dy * u * slope, "u": dy * value}
    dx = sum(d[p] @ W[p].t() for p in names)
    out = {}
    for p in names:
        dA, dB = torch.zeros_like(st["A" + p], dtype=torch.float64), torch.zeros_like(st["B" + p], dtype=torch.float64)
        for lo, hi, k in pieces:
            A, B, s = adapter(p, k)
            back = s * (d[p][lo:hi] @ B.t())
            dx[lo:hi] += back @ A.t()
            dA[k] += x[lo:hi].t() @ back
            dB[k] += s * ((x[lo:hi] @ A).t() @ d[p][lo:hi])
        out.update({"dA" + p: dA, "dB" + p: dB})
        if c["train_w"]:
            out["dW" + p] = x.t() @ d[p]
    return {"dX": dx, **out}
