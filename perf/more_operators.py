"""Cases of what stands around a layer of many adapters: the projection with bias, activation and residual, the
sorting of rows by adapter and back, and the layer norm, each with its backward pass.

    proj       z_i = x_i @ W + b + s_k (x_i @ A_k) @ B_k,  y_i = act(z_i) + r_i     k: the adapter of row i's segment
    proj_grad  dz = dy * act'(z) from the stored z; gradients of x, b, A_k, B_k and, on request, W
    sort       the choices (token i, its j-th adapter) sorted by adapter, stable, those without an adapter last: the order,
               its inverse and the segments, and every choice's row of X at its sorted place
    back       y_i = r_i + sum_j w_ij ys_(place of i, j)
    back_grad  dys and dw from dy, and dx_i = sum_j dxs_(place of i, j), the gradient of the sorting
    norm       y = (x - mean) / sqrt(var + eps) * gamma + beta, with mean and 1 / sqrt(var + eps) of every row
    norm_grad  gradients of x (plus the gradient that passes the norm by), gamma and beta

Gradients come in the inputs' format, those of the weights w_ij in 32 bits; the gradient of an adapter that no row uses is zero.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


def _proj(name, op, dtype, n, h_in, h_out, rank, adapters, segs, cover=1.0, scales=False, bias=True, act="gelu_tanh",
          residual=False, keep=False, train_w=False):
    return {"name": name, "op": op, "dtype": dtype, "n": n, "h_in": h_in, "h_out": h_out, "rank": rank, "adapters": adapters,
            "segs": segs, "cover": cover, "scales": scales, "bias": bias, "act": act, "residual": residual, "keep": keep,
            "train_w": train_w}


def _rows(name, op, dtype, n, h, top_k, adapters, cover=1.0, residual=False):
    return {"name": name, "op": op, "dtype": dtype, "n": n, "h": h, "top_k": top_k, "adapters": adapters, "cover": cover,
            "residual": residual}


def _norm(name, op, dtype, n, h, beyond=False):
    return {"name": name, "op": op, "dtype": dtype, "n": n, "h": h, "beyond": beyond}


def listed():
    return [
        # one request decoding one token through the up projection of a feed-forward block without a gate
        _proj("proj_token", "proj", "f16", 1, 4096, 11008, 16, 32, 1),
        # prompts of 8 requests through the down projection, whose output joins the residual stream; odd rows, some without adapter
        _proj("proj_prompts", "proj", "bf16", 2011, 11008, 4096, 64, 8, 8, cover=0.9, act="none", residual=True),
        # a training micro-batch through the up projection; z is kept for the backward pass
        _proj("proj_long", "proj", "bf16", 8192, 4096, 11008, 16, 16, 16, keep=True),
        # fine-tuning small adapters of several tenants on a narrow layer, base frozen
        _proj("proj_grad_small", "proj_grad", "f16", 203, 1024, 1376, 8, 6, 9, scales=True, act="relu"),
        # a training step of the up projection, base trained too
        _proj("proj_grad_full", "proj_grad", "bf16", 4096, 4096, 11008, 16, 4, 8, scales=True, train_w=True),
        # a decode batch of 32 requests, two adapters each, sorted before the adapters' products
        _rows("sort_decode", "sort", "f16", 32, 4096, 2, 32),
        # prompts of many requests, two of 16 adapters a token
        _rows("sort_long", "sort", "bf16", 8192, 4096, 2, 16),
        # prompts of width 5120, odd rows, four adapters a token, some choices without one; the sum joins the base's output
        _rows("back_prompts", "back", "bf16", 2011, 5120, 4, 64, cover=0.9, residual=True),
        # the backward pass of a training micro-batch with two adapters a token
        _rows("back_grad_long", "back_grad", "bf16", 4096, 4096, 2, 8),
        # a decode batch in front of a projection
        _norm("norm_decode", "norm", "f16", 32, 4096),
        # long prompts of width 5120
        _norm("norm_long", "norm", "bf16", 8192, 5120),
        # a training micro-batch; the residual stream's gradient joins
        _norm("norm_grad_long", "norm_grad", "bf16", 4096, 4096, beyond=True),
    ]


ACTS = ["none", "relu", "silu", "gelu_tanh", "gelu"]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    kind = rng.choice(["proj", "proj", "proj_grad", "proj_grad", "sort", "back", "back_grad", "norm", "norm_grad"])
    while True:
        dtype = rng.choice(["f16", "bf16"])
        if kind.startswith("proj"):
            n, adapters = _log(rng, 1, 8192), _log(rng, 1, 64)
            c = _proj("", kind, dtype, n, _log(rng, 256, 11008, 8), _log(rng, 256, 13824, 8), rng.choice([8, 16, 32, 64]),
                      adapters, min(n, _log(rng, 1, 64)), cover=rng.choice([1.0, 1.0, 0.9, 0.5]),
                      scales=rng.random() < 0.5, bias=rng.random() < 0.8, act=rng.choice(ACTS),
                      residual=kind == "proj" and rng.random() < 0.5, keep=kind == "proj" and rng.random() < 0.4,
                      train_w=kind == "proj_grad" and rng.random() < 0.4)
        elif kind.startswith("norm"):
            c = _norm("", kind, dtype, _log(rng, 1, 16384), _log(rng, 64, 16384, 8),
                      beyond=kind == "norm_grad" and rng.random() < 0.5)
        else:
            c = _rows("", kind, dtype, _log(rng, 1, 16384), _log(rng, 64, 8192, 8), rng.choice([1, 2, 2, 4, 6, 8]),
                      _log(rng, 1, 512), cover=rng.choice([1.0, 1.0, 0.9, 0.5]),
                      residual=kind == "back" and rng.random() < 0.5)
        del c["name"]
        if _cost(c) <= max(_cost(x) for x in listed() if x["op"] == kind):
            return c


def _cost(case):
    w = work(case)
    return w["bytes"] / 4e12 + w["flops"] / 1e15


def work(case):
    op, n, e = case["op"], case["n"], 2
    if op == "norm":
        return {"bytes": 2 * n * case["h"] * e + 2 * case["h"] * e + 8 * n, "flops": 8 * n * case["h"]}
    if op == "norm_grad":
        return {"bytes": (4 if case["beyond"] else 3) * n * case["h"] * e + 3 * case["h"] * e + 8 * n,
                "flops": 14 * n * case["h"]}
    if not op.startswith("proj"):
        m, h = n * case["top_k"], case["h"]
        if op == "sort":
            return {"bytes": (n + m) * h * e + 12 * m + 8 * case["adapters"], "flops": m}
        if op == "back":
            return {"bytes": (m + (2 if case["residual"] else 1) * n) * h * e + 8 * m, "flops": 2 * m * h}
        # dy, ys and dxs read, dys and dx written
        return {"bytes": (2 * n + 3 * m) * h * e + 12 * m, "flops": 4 * m * h}
    k, f, r = case["h_in"], case["h_out"], case["rank"]
    rows, used = int(n * case["cover"]), min(case["segs"], case["adapters"])
    weights = k * f * e + used * r * (k + f) * e
    if op == "proj":
        return {"bytes": n * k * e + weights + f * e * case["bias"] + n * f * e * (1 + case["residual"] + case["keep"]),
                "flops": 2 * n * k * f + 2 * rows * r * (k + f)}
    # z is not read where there is no activation
    reads = n * k * e + weights + n * f * e * (1 if case["act"] == "none" else 2)
    writes = n * k * e + case["adapters"] * r * (k + f) * e + f * e * case["bias"] + (k * f * e if case["train_w"] else 0)
    return {"bytes": reads + writes, "flops": 2 * n * k * f * (2 if case["train_w"] else 1) + 2 * rows * r * (3 * k + 2 * f)}


# ------------------------------------------------------------------ inputs

def _segments(case, seed):
    """Segment bounds and adapter ids (host): random lengths over the covered rows, adapters in any order, some twice."""
    rng = np.random.default_rng(seed)
    rows = max(1, int(case["n"] * case["cover"]))
    cuts = np.sort(rng.integers(0, rows + 1, size=case["segs"] - 1)) if case["segs"] < rows else np.arange(1, case["segs"])
    indptr = np.concatenate([[0], np.minimum(cuts, rows), [rows]]).astype(np.int32)
    order = np.concatenate([rng.permutation(case["adapters"]) for _ in range(-(-case["segs"] // case["adapters"]))])
    return indptr, order[: case["segs"]].astype(np.int32)


def _choices(case, gen):
    """What a router gives: per token its top_k adapters (some more popular) and weights that sum to one.  Choices past
    the adapters there are, and some more where not all are covered, have no adapter (-1)."""
    n, k, P = case["n"], case["top_k"], case["adapters"]
    logits = torch.randn(n, max(k, P), generator=gen, device="cuda")
    logits[:, :P] += torch.linspace(1.5, 0, P, device="cuda")
    logits[:, P:] = -1e4
    top, ids = torch.topk(logits, k, dim=1)
    ids = torch.where(ids < P, ids, -1)
    if case["cover"] < 1:
        ids = torch.where(torch.rand(n, k, generator=gen, device="cuda") < case["cover"], ids, -1)
    w = torch.exp(top - top[:, :1])
    return ids.to(torch.int32).contiguous(), (w / w.sum(1, keepdim=True)).contiguous()


def prepare(case, seed):
    dt, dev, op, n = DTYPES[case["dtype"]], "cuda", case["op"], case["n"]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev).mul_(std).to(dt)

    st = {"case": case}
    if op.startswith("proj"):
        k, f, r, P = case["h_in"], case["h_out"], case["rank"], case["adapters"]
        indptr, ids = _segments(case, seed)
        rows_of = torch.full((n,), -1, dtype=torch.int64)
        rows_of[: int(indptr[-1])] = torch.from_numpy(np.repeat(ids, np.diff(indptr)).astype(np.int64))
        st.update(X=normal(n, k), W=normal(k, f, std=k ** -0.5), A=normal(P, k, r, std=k ** -0.5),
                  B=normal(P, r, f, std=r ** -0.5), indptr=torch.from_numpy(indptr).to(dev),
                  ids=torch.from_numpy(ids).to(dev), rows_of=rows_of.to(dev),
                  s=torch.rand(P, generator=gen, device=dev) + 0.5 if case["scales"] else None,
                  b=normal(f, std=0.5) if case["bias"] else None, R=normal(n, f) if case["residual"] else None)
        if op == "proj_grad":
            st.update(Z=normal(n, f, std=2 ** 0.5) if case["act"] != "none" else None, dY=normal(n, f))
    elif op.startswith("norm"):
        h = case["h"]
        # a residual stream: some channels much larger than the others, rows off zero
        big = 1 + 15 * (torch.rand(h, generator=gen, device=dev) < 0.01)
        x = torch.randn(n, h, generator=gen, device=dev) * big + 0.3 * torch.randn(n, 1, generator=gen, device=dev)
        st.update(X=x.to(dt), gamma=(1 + 0.2 * torch.randn(h, generator=gen, device=dev)).to(dt), beta=normal(h, std=0.2))
        if op == "norm_grad":
            mean, rstd = _moments(st["X"].double())
            st.update(mean=mean.float(), rstd=rstd.float(), dY=normal(n, h), beyond=normal(n, h) if case["beyond"] else None)
    else:
        m, h = n * case["top_k"], case["h"]
        st["ids"], st["w"] = _choices(case, gen)
        if op == "sort":
            st["X"] = normal(n, h)
        else:
            _, slots, _, _ = _sorted(st)
            st.update(slots=slots, Ys=normal(m, h))
            if op == "back":
                st["R"] = normal(n, h) if case["residual"] else None
            else:
                st.update(dY=normal(n, h), dXs=normal(m, h))
    if own:
        _handles(st)
    return st


# ------------------------------------------------------------------ the plain form

def _act(z, kind):
    """The activation and its derivative."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        return torch.where(z > 0, z, 0.0), (z > 0).to(z.dtype)
    if kind == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return z * sig, sig * (1 + z * (1 - sig))
    if kind == "gelu":
        phi = 0.5 * torch.erfc(z * -math.sqrt(0.5))
        return z * phi, phi + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    c, a = math.sqrt(2 / math.pi), 0.044715
    sig = 1 / (1 + torch.exp(-2 * c * (z + a * z * z * z)))  # (1 + tanh) / 2
    return z * sig, sig + 2 * z * sig * (1 - sig) * c * (1 + 3 * a * z * z)


def _moments(x):
    mean = x.mean(1)
    d = x - mean[:, None]
    return mean, 1 / torch.sqrt((d * d).mean(1) + EPS)


def _sorted(st):
    """Order of the choices, its inverse, segment bounds and their adapters."""
    P = st["case"]["adapters"]
    ids = st["ids"].reshape(-1).long()
    key = torch.where((ids >= 0) & (ids < P), ids, P)
    perm = torch.argsort(key, stable=True)
    slots = torch.empty_like(perm)
    slots[perm] = torch.arange(perm.numel(), device="cuda")
    counts = torch.zeros(P + 1, dtype=torch.int64, device="cuda").index_add_(0, key, torch.ones_like(key))
    bounds = torch.cat([counts.new_zeros(1), torch.cumsum(counts[:P], 0)])
    return perm.int(), slots.int(), bounds.int(), torch.arange(P, device="cuda", dtype=torch.int32)


def _flat(st):
    """All adapters side by side, in 32 bits, and which columns are each row's."""
    c = st["case"]
    A = st["A"].float().permute(1, 0, 2).reshape(c["h_in"], -1)
    B = st["B"].float().reshape(-1, c["h_out"])
    s = st["s"].repeat_interleave(c["rank"]) if st["s"] is not None else torch.ones(A.shape[1], device="cuda")
    cols = torch.arange(c["adapters"], device="cuda").repeat_interleave(c["rank"])
    return A, B, s, st["rows_of"][:, None] == cols[None, :]


def _plain_proj(st):
    c = st["case"]
    dt, x = DTYPES[c["dtype"]], st["X"].float()
    A, B, s, mask = _flat(st)
    z = x @ st["W"].float() + torch.where(mask, (x @ A) * s, 0.0) @ B
    if c["bias"]:
        z = z + st["b"].float()
    y = _act(z, c["act"])[0]
    if c["residual"]:
        y = y + st["R"].float()
    return {"Y": y.to(dt), **({"Z": z.to(dt)} if c["keep"] else {})}


def _plain_proj_grad(st):
    c = st["case"]
    dt, P, r, x, dy = DTYPES[c["dtype"]], c["adapters"], c["rank"], st["X"].float(), st["dY"].float()
    A, B, s, mask = _flat(st)
    dz = dy if c["act"] == "none" else dy * _act(st["Z"].float(), c["act"])[1]
    v, dv = torch.where(mask, (x @ A) * s, 0.0), torch.where(mask, (dz @ B.t()) * s, 0.0)
    out = {"dX": (dz @ st["W"].float().t() + dv @ A.t()).to(dt),
           "dA": (x.t() @ dv).reshape(c["h_in"], P, r).permute(1, 0, 2).contiguous().to(dt),
           "dB": (v.t() @ dz).reshape(P, r, c["h_out"]).to(dt)}
    if c["bias"]:
        out["db"] = dz.sum(0).to(dt)
    if c["train_w"]:
        out["dW"] = (x.t() @ dz).to(dt)
    return out


def _plain_rows(st):
    c = st["case"]
    dt, k, h = DTYPES[c["dtype"]], c["top_k"], c["h"]
    if c["op"] == "sort":
        perm, slots, bounds, adapters = _sorted(st)
        return {"perm": perm, "slots": slots, "bounds": bounds, "adapters": adapters, "Xs": st["X"][perm.long() // k]}
    slots = st["slots"].long()
    if c["op"] == "back":
        y = (st["w"][:, :, None] * st["Ys"][slots].float().reshape(-1, k, h)).sum(1)
        if c["residual"]:
            y = y + st["R"].float()
        return {"Y": y.to(dt)}
    dy = st["dY"].float()
    dys = torch.empty_like(st["Ys"])
    dys[slots] = (st["w"][:, :, None] * dy[:, None, :]).reshape(-1, h).to(dt)
    dw = (dy[:, None, :] * st["Ys"][slots].float().reshape(-1, k, h)).sum(2)
    return {"dYs": dys, "dw": dw, "dX": st["dXs"][slots].float().reshape(-1, k, h).sum(1).to(dt)}


def _plain_norm(st):
    c = st["case"]
    dt, x, g = DTYPES[c["dtype"]], st["X"].float(), st["gamma"].float()
    if c["op"] == "norm":
        mean, rstd = _moments(x)
        return {"Y": ((x - mean[:, None]) * rstd[:, None] * g + st["beta"].float()).to(dt), "mean": mean, "rstd": rstd}
    dy, r = st["dY"].float(), st["rstd"][:, None]
    xh, q = (x - st["mean"][:, None]) * r, dy * g
    dx = r * (q - q.mean(1, keepdim=True) - xh * (q * xh).mean(1, keepdim=True))
    if c["beyond"]:
        dx = dx + st["beyond"].float()
    return {"dX": dx.to(dt), "dgamma": (dy * xh).sum(0).to(dt), "dbeta": dy.sum(0).to(dt)}


def _plain(st):
    op = st["case"]["op"]
    if op.startswith("proj"):
        return _plain_proj(st) if op == "proj" else _plain_proj_grad(st)
    return _plain_norm(st) if op.startswith("norm") else _plain_rows(st)


# ------------------------------------------------------------------ the framework's calls

def _handles(st):
    """What a program that uses the library keeps: the problem, tables of pointers, outputs, a workspace."""
    import segmented_gather_matvec_amd as sg

    c = st["case"]
    op, n, dt = c["op"], c["n"], DTYPES[c["dtype"]]

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    out = st["out"] = {}
    if op.startswith("proj"):
        k, f = c["h_in"], c["h_out"]
        longest = int((st["indptr"][1:] - st["indptr"][:-1]).max())
        st["problem"] = sg.make_problem(c["dtype"], n, k, f, c["rank"], c["adapters"], c["segs"], longest)
        st["act"] = {"none": sg.SGMV_ACT_NONE, "relu": sg.SGMV_ACT_RELU, "silu": sg.SGMV_ACT_SILU,
                     "gelu_tanh": sg.SGMV_ACT_GELU_TANH, "gelu": sg.SGMV_ACT_GELU}[c["act"]]
        st["ws"] = sg.new_layer_workspace(st["problem"], sg.SGMV_DENSE_ACT_FORWARD if op == "proj" else
                                          sg.SGMV_DENSE_ACT_BACKWARD)
        if op == "proj":
            out["Y"] = empty(n, f)
            if c["keep"]:
                out["Z"] = empty(n, f)
        else:
            out.update(dX=empty(n, k), dA=torch.empty_like(st["A"]), dB=torch.empty_like(st["B"]))
            if c["bias"]:
                out["db"] = empty(f)
            if c["train_w"]:
                out["dW"] = empty(k, f)
            st["grad"] = (out.get("dW"), sg.pointer_table(out["dA"]), sg.pointer_table(out["dB"]))
        st["proj"] = (sg.pointer_table(st["A"]), sg.pointer_table(st["B"]), out.get("Y"), None, st["s"])
    elif op == "norm":
        out.update(Y=empty(n, c["h"]), mean=empty(n, dtype=torch.float32), rstd=empty(n, dtype=torch.float32))
    elif op == "norm_grad":
        out.update(dX=empty(n, c["h"]), dgamma=empty(c["h"]), dbeta=empty(c["h"]))
        st["ws"] = sg.new_layer_norm_workspace(n, c["h"])
    elif op == "sort":
        m, P = n * c["top_k"], c["adapters"]
        i32 = torch.int32
        out.update(perm=empty(m, dtype=i32), slots=empty(m, dtype=i32), bounds=empty(P + 1, dtype=i32),
                   adapters=empty(P, dtype=i32), Xs=empty(m, c["h"]))
        st["ws"] = sg.new_route_workspace(n, c["top_k"], P)
    elif op == "back":
        out["Y"] = empty(n, c["h"])
    else:
        out.update(dYs=torch.empty_like(st["Ys"]), dw=torch.empty_like(st["w"]), dX=empty(n, c["h"]))


def _called(st):
    import segmented_gather_matvec_amd as sg

    c, out = st["case"], st["out"]
    op = c["op"]
    if op == "proj":
        sg.sgmv_dense_act_lora_apply(st["problem"], st["X"], st["W"], st["proj"], st["indptr"], st["ids"], st["ws"],
                                     act=st["act"], bias=st["b"], residual=st["R"], Z=out.get("Z"))
    elif op == "proj_grad":
        sg.sgmv_dense_act_lora_backward(st["problem"], st["X"], st["W"], st["proj"], st["dY"], st["indptr"], st["ids"],
                                        st["ws"], act=st["act"], Z=st["Z"], dX=out["dX"], grad=st["grad"],
                                        dbias=out.get("db"))
    elif op == "norm":
        sg.sgmv_layer_norm_apply(st["X"], st["gamma"], st["beta"], out["Y"], EPS, mean=out["mean"], rstd=out["rstd"])
    elif op == "norm_grad":
        sg.sgmv_layer_norm_backward(st["X"], st["gamma"], st["mean"], st["rstd"], st["dY"], st["ws"], dX=out["dX"],
                                    beyond=st["beyond"], dgamma=out["dgamma"], dbeta=out["dbeta"])
    elif op == "sort":
        sg.sgmv_route_rows(st["ids"], c["adapters"], out["perm"], out["slots"], out["bounds"], out["adapters"], st["ws"])
        sg.sgmv_dispatch_rows(st["X"], out["slots"], out["Xs"])
    elif op == "back":
        sg.sgmv_combine_rows(st["Ys"], st["slots"], out["Y"], weights=st["w"], residual=st["R"])
    else:
        sg.sgmv_combine_rows_backward(st["dY"], st["Ys"], st["slots"], weights=st["w"], dYs=out["dYs"], dweights=out["dw"])
        sg.sgmv_combine_rows(st["dXs"], st["slots"], out["dX"])
    return out


def run(state):
    return _called(state) if own else _plain(state)


# ------------------------------------------------------------------ the definition in 64 bits

def _slope64(z, kind):
    """The activation and its derivative in 64 bits."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        return z.clamp(min=0), (z > 0).double()
    if kind == "silu":
        e = torch.sigmoid(z)
        return z * e, e + z * e * torch.sigmoid(-z)
    if kind == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    e = torch.sigmoid(2 * u)
    return z * e, e + z / (2 * torch.cosh(u) ** 2) * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)


def _exact_proj(st):
    """Segment by segment from the definition."""
    c, x, W = st["case"], st["X"].double(), st["W"].double()
    bounds, ids = st["indptr"].tolist(), st["ids"].tolist()
    pieces = [(lo, hi, st["A"][k].double(), st["B"][k].double(), float(st["s"][k]) if st["s"] is not None else 1.0, k)
              for lo, hi, k in zip(bounds[:-1], bounds[1:], ids) if hi > lo]
    if c["op"] == "proj":
        z = x @ W
        for lo, hi, A, B, s, _ in pieces:
            z[lo:hi] += s * ((x[lo:hi] @ A) @ B)
        if st["b"] is not None:
            z += st["b"].double()
        y = _slope64(z, c["act"])[0]
        if st["R"] is not None:
            y = y + st["R"].double()
        return {"Y": y, "Z": z} if c["keep"] else {"Y": y}
    dz = st["dY"].double()
    if c["act"] != "none":
        dz = dz * _slope64(st["Z"].double(), c["act"])[1]
    dx = dz @ W.t()
    dA, dB = torch.zeros_like(st["A"], dtype=torch.float64), torch.zeros_like(st["B"], dtype=torch.float64)
    for lo, hi, A, B, s, k in pieces:
        back = s * (dz[lo:hi] @ B.t())
        dx[lo:hi] += back @ A.t()
        dA[k] += x[lo:hi].t() @ back
        dB[k] += s * ((x[lo:hi] @ A).t() @ dz[lo:hi])
    out = {"dX": dx, "dA": dA, "dB": dB}
    if c["bias"]:
        out["db"] = dz.sum(0)
    if c["train_w"]:
        out["dW"] = x.t() @ dz
    return out


def _exact_rows(st):
    """Choice by choice on the host for the order; rows one choice of all tokens at a time."""
    c = st["case"]
    k, P = c["top_k"], c["adapters"]
    if c["op"] == "sort":
        ids = st["ids"].cpu().numpy().reshape(-1)
        groups = [np.flatnonzero(ids == a) for a in range(P)] + [np.flatnonzero((ids < 0) | (ids >= P))]
        perm = np.concatenate(groups).astype(np.int32)
        slots = np.empty_like(perm)
        for place, e in enumerate(perm.tolist()):
            slots[e] = place
        bounds = np.cumsum([0] + [len(g) for g in groups[:-1]]).astype(np.int32)
        token = torch.from_numpy((perm // k).astype(np.int64)).cuda()
        dev = [torch.from_numpy(a).cuda() for a in (perm, slots, bounds, np.arange(P, dtype=np.int32))]
        return {"perm": dev[0], "slots": dev[1], "bounds": dev[2], "adapters": dev[3], "Xs": st["X"].double()[token]}
    at = st["slots"].long().reshape(-1, k)
    if c["op"] == "back":
        y = st["R"].double() if c["residual"] else torch.zeros(c["n"], c["h"], dtype=torch.float64, device="cuda")
        for j in range(k):
            y = y + st["w"][:, j, None].double() * st["Ys"].double()[at[:, j]]
        return {"Y": y}
    dy, ys, dxs = st["dY"].double(), st["Ys"].double(), st["dXs"].double()
    dys, dw, dx = torch.empty_like(ys), torch.empty_like(st["w"], dtype=torch.float64), torch.zeros_like(dy)
    for j in range(k):
        dys[at[:, j]] = st["w"][:, j, None].double() * dy
        dw[:, j] = torch.linalg.vecdot(dy, ys[at[:, j]])
        dx += dxs[at[:, j]]
    return {"dYs": dys, "dw": dw, "dX": dx}


def _exact_norm(st):
    c, x, g = st["case"], st["X"].double(), st["gamma"].double()
    if c["op"] == "norm":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + EPS).rsqrt()
        return {"Y": torch.addcmul(st["beta"].double(), (x - mean[:, None]) * rstd[:, None], g), "mean": mean, "rstd": rstd}
    dy, r = st["dY"].double(), st["rstd"].double()[:, None]
    xh = (x - st["mean"].double()[:, None]) * r
    q = dy * g
    along = (q @ torch.ones(c["h"], 1, dtype=torch.float64, device="cuda") + xh * (q * xh).sum(1, keepdim=True)) / c["h"]
    dx = (q - along) * r
    if c["beyond"]:
        dx = dx + st["beyond"].double()
    return {"dX": dx, "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}


def exact(case, seed):
    global own
    mine, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = mine
    op = case["op"]
    return _exact_proj(st) if op.startswith("proj") else _exact_norm(st) if op.startswith("norm") else _exact_rows(st)
