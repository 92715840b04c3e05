"""The training operators of the expert layer: cases, plain forms and exact values.

Four operators, each in a plain torch form and as the package's own call:

* grouped:  products of ragged row groups with their expert's matrix, the
            groups' rows given by the dispatch's offsets: forward
            y = x W_g^T, input gradient dx = dy W_g, weight gradient
            dW_g = dy_g^T x_g
* norm:     layer norm over the model width, forward and backward with the
            gradients of its weight and bias
* swiglu:   SiLU(gate) * up on the packed gate/up columns (blocks of 64 gate,
            64 up), forward and backward
* ortho:    Newton-Schulz orthogonalisation of a stack of update matrices

Sizes are those of the benchmark workloads (tiny, small, 16b, large) and
generic odd ones.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
NS_COEF = (3.4445, -4.7750, 2.0315)
NS_STEPS = 5
LN_EPS = 1e-5


def listed():
    return [
        # the fp32 correctness layer's gate/up product with its gradients
        {"name": "grouped_all_tiny_f32", "op": "grouped", "dir": "all", "T": 64, "top_k": 4, "groups": 16,
         "n": 128, "k": 128, "skew": 0.0, "dtype": "f32"},
        # one decode step of 8 tokens: the activated experts' gate/up weights are streamed
        {"name": "grouped_fwd_decode8", "op": "grouped", "dir": "fwd", "T": 8, "top_k": 6, "groups": 64,
         "n": 2816, "k": 2048, "skew": 0.05, "dtype": "bf16"},
        # training forward of the small-model-shaped layer, skewed loads
        {"name": "grouped_fwd_small", "op": "grouped", "dir": "fwd", "T": 8192, "top_k": 7, "groups": 63,
         "n": 1792, "k": 1280, "skew": 0.3, "dtype": "bf16"},
        # input gradient of the 16B-shaped layer's gate/up product
        {"name": "grouped_dx_16b", "op": "grouped", "dir": "dx", "T": 16384, "top_k": 6, "groups": 64,
         "n": 2816, "k": 2048, "skew": 0.05, "dtype": "bf16"},
        # weight gradient at the small model's size, with sizes that fill no tile
        {"name": "grouped_dw_odd", "op": "grouped", "dir": "dw", "T": 8191, "top_k": 7, "groups": 63,
         "n": 1784, "k": 1288, "skew": 0.1, "dtype": "bf16"},
        # the norm before the layer, a decode step of 32 tokens
        {"name": "norm_fwd_decode32", "op": "norm", "dir": "fwd", "T": 32, "d": 2048, "dtype": "bf16"},
        # an odd width in fp32, forward and backward
        {"name": "norm_all_odd_f32", "op": "norm", "dir": "all", "T": 4099, "d": 1283, "dtype": "f32"},
        # the large layer's tokens, forward and backward
        {"name": "norm_all_large", "op": "norm", "dir": "all", "T": 32768, "d": 4096, "dtype": "bf16"},
        # activations of the small layer's routed rows
        {"name": "swiglu_fwd_small", "op": "swiglu", "dir": "fwd", "rows": 57344, "inter": 896, "dtype": "bf16"},
        # and their gradient at the 16B shape
        {"name": "swiglu_bwd_16b", "op": "swiglu", "dir": "bwd", "rows": 98304, "inter": 1408, "dtype": "bf16"},
        # the router matrix's update, from a float32 momentum
        {"name": "ortho_router", "op": "ortho", "mats": 1, "rows": 64, "cols": 2048, "dtype": "f32"},
        # the down projections of the 16B-shaped layer, all experts at once
        {"name": "ortho_down_16b", "op": "ortho", "mats": 64, "rows": 2048, "cols": 1408, "dtype": "bf16"},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "grouped", "norm", "swiglu", "ortho"])
    if op == "grouped":
        f32 = rng.random() < 0.2
        groups = _logint(rng, 1, 64)
        top_k = rng.randint(1, min(groups, 8))
        n, k = 8 * _logint(rng, 8, 352), 8 * _logint(rng, 8, 256)
        T = _logint(rng, 1, 1024 if f32 else 16384)
        return {"op": "grouped", "dir": rng.choice(["fwd", "dx", "dw", "all"]), "T": T, "top_k": top_k,
                "groups": groups, "n": n, "k": k, "skew": rng.choice([0.0, 0.1, 0.3]),
                "dtype": "f32" if f32 else "bf16"}
    if op == "norm":
        d = _logint(rng, 64, 4096)
        return {"op": "norm", "dir": rng.choice(["fwd", "all"]), "T": _logint(rng, 1, 32768), "d": d,
                "dtype": rng.choice(["f32", "bf16"])}
    if op == "swiglu":
        return {"op": "swiglu", "dir": rng.choice(["fwd", "bwd"]), "rows": _logint(rng, 1, 98304),
                "inter": 64 * _logint(rng, 1, 22), "dtype": rng.choice(["f32", "bf16"])}
    rows, cols = _logint(rng, 16, 2048), _logint(rng, 16, 2048)
    most = max(1, 64 * 2048 * 1408 * 1408 // (rows * cols * min(rows, cols)))
    return {"op": "ortho", "mats": _logint(rng, 1, min(64, most)), "rows": rows, "cols": cols,
            "dtype": rng.choice(["f32", "bf16"])}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def rand(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)

    def out(*shape, dtype=dt):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    s = {"case": case}
    if case["op"] == "grouped":
        T, K, G, n, k, d = case["T"], case["top_k"], case["groups"], case["n"], case["k"], case["dir"]
        # the rows of each expert under top-K routing with per-expert biases
        scores = rand(T, G, dtype=torch.float32) + rand(G, std=math.sqrt(case["skew"]), dtype=torch.float32)
        counts = torch.bincount(scores.topk(K, dim=1).indices.reshape(-1), minlength=G)
        offsets = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = counts.cumsum(0)
        rows = T * K
        s |= {"offsets": offsets, "capacity": int(counts.max())}
        s |= {"x": rand(rows, k)} if d != "dx" else {}
        s |= {"w": rand(G, n, k, std=k ** -0.5)} if d != "dw" else {}
        s |= {"dy": rand(rows, n, std=0.1)} if d != "fwd" else {}
        s |= {"y": out(rows, n)} if d in ("fwd", "all") else {}
        s |= {"dx": out(rows, k)} if d in ("dx", "all") else {}
        s |= {"dw": out(G, n, k)} if d in ("dw", "all") else {}
    elif case["op"] == "norm":
        T, d = case["T"], case["d"]
        # a residual stream: a few channels carry large offsets
        x = rand(T, d, dtype=torch.float32) + 4.0 * (rand(d, dtype=torch.float32) > 2.0)
        s |= {"x": x.to(dt), "gamma": 1 + 0.1 * rand(d, dtype=torch.float32),
              "beta": 0.1 * rand(d, dtype=torch.float32), "y": out(T, d),
              "mean": out(T, dtype=torch.float32), "rstd": out(T, dtype=torch.float32)}
        if case["dir"] == "all":
            s |= {"dy": rand(T, d), "dx": out(T, d), "dgamma": out(d, dtype=torch.float32),
                  "dbeta": out(d, dtype=torch.float32)}
    elif case["op"] == "swiglu":
        rows, inter = case["rows"], case["inter"]
        s["gu"] = rand(rows, 2 * inter)
        if case["dir"] == "fwd":
            s["a"] = out(rows, inter)
        else:
            s |= {"da": rand(rows, inter, std=0.1), "dgu": out(rows, 2 * inter)}
    else:
        m, r, c = case["mats"], case["rows"], case["cols"]
        # a momentum: a few strong directions over noise
        rank = min(16, r, c)
        signal = rand(m, r, rank, dtype=torch.float32) @ rand(m, rank, c, dtype=torch.float32)
        s |= {"m": (signal * rank ** -0.5 + rand(m, r, c, std=0.5, dtype=torch.float32)).to(dt),
              "o": out(m, r, c, dtype=torch.bfloat16)}
    return s


# ------------------------------------------------------------- plain forms
def _grouped_plain(s):
    off, cap = s["offsets"].long(), s["capacity"]
    G, rows = off.numel() - 1, (s["x"] if "x" in s else s["dy"]).shape[0]
    at = torch.arange(rows, device=off.device)
    gid = torch.searchsorted(off[1:].contiguous(), at, right=True)
    slot = gid * cap + at - off[gid]

    def padded(t):
        p = torch.zeros(G * cap, t.shape[1], device=t.device)
        p[slot] = t.float()
        return p.view(G, cap, -1)

    got = {}
    w = s["w"].float() if "w" in s else None
    x = padded(s["x"]) if "x" in s else None
    dy = padded(s["dy"]) if "dy" in s else None
    if "y" in s:
        got["y"] = (x @ w.transpose(1, 2)).reshape(G * cap, -1)[slot].to(s["y"].dtype)
    if "dx" in s:
        got["dx"] = (dy @ w).reshape(G * cap, -1)[slot].to(s["dx"].dtype)
    if "dw" in s:
        got["dw"] = (dy.transpose(1, 2) @ x).to(s["dw"].dtype)
    return got


def _norm_plain(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    rstd = torch.rsqrt((x - mean).square().mean(1, keepdim=True) + LN_EPS)
    xh = (x - mean) * rstd
    got = {"y": (xh * s["gamma"] + s["beta"]).to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if "dy" in s:
        dy = s["dy"].float()
        t = dy * s["gamma"]
        dx = rstd * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
        got |= {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}
    return got


def _swiglu_plain(s):
    b = s["gu"].float().view(s["gu"].shape[0], -1, 2, 64)
    gate, up = b[:, :, 0], b[:, :, 1]
    sig = 1 / (1 + torch.exp(-gate))
    if "a" in s:
        return {"a": (gate * sig * up).reshape(s["a"].shape).to(s["a"].dtype)}
    da = s["da"].float().view(gate.shape)
    dgate = da * up * sig * (1 + gate * (1 - sig))
    dup = da * gate * sig
    return {"dgu": torch.stack([dgate, dup], 2).reshape(s["gu"].shape).to(s["gu"].dtype)}


def _ortho_plain(s):
    a, b, c = NS_COEF
    x = s["m"].float()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + 1e-7)
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    for _ in range(NS_STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return {"o": (x.transpose(1, 2) if tall else x).to(torch.bfloat16)}


# ------------------------------------------------------- the package's calls
def _lib():
    from mixture_experts_layer_56_b200 import _lib as L
    return L


def _dtype_of(L, case):
    return L.MOE_DTYPE_F32 if case["dtype"] == "f32" else L.MOE_DTYPE_BF16


def _scratch(nbytes):
    return torch.empty(max(1, nbytes), dtype=torch.uint8, device="cuda")


def _grouped_own(s):
    if "shape" not in s:
        L, c = _lib(), s["case"]
        s["L"] = L
        s["shape"] = L.make_grouped_shape(c["T"] * c["top_k"], c["groups"], c["n"], c["k"], _dtype_of(L, c))
        s["ws"] = _scratch(L.moe_grouped_workspace_size(s["shape"]))
    L, got = s["L"], {}
    if "y" in s:
        L.moe_grouped_matmul(s["shape"], s["x"], s["offsets"], s["w"], s["y"], s["ws"])
        got["y"] = s["y"]
    if "dx" in s:
        L.moe_grouped_matmul_dx(s["shape"], s["dy"], s["offsets"], s["w"], s["dx"], s["ws"])
        got["dx"] = s["dx"]
    if "dw" in s:
        L.moe_grouped_matmul_dw(s["shape"], s["dy"], s["x"], s["offsets"], s["dw"], s["ws"])
        got["dw"] = s["dw"]
    return got


def _norm_own(s):
    if "shape" not in s:
        L, c = _lib(), s["case"]
        s["L"] = L
        s["shape"] = L.make_norm_shape(c["T"], c["d"], _dtype_of(L, c), LN_EPS)
        s["ws"] = _scratch(L.moe_layer_norm_workspace_size(s["shape"]))
    L = s["L"]
    L.moe_layer_norm(s["shape"], s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"])
    got = {k: s[k] for k in ("y", "mean", "rstd")}
    if "dy" in s:
        L.moe_layer_norm_backward(s["shape"], s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"],
                                  s["dx"], s["dgamma"], s["dbeta"], s["ws"])
        got |= {k: s[k] for k in ("dx", "dgamma", "dbeta")}
    return got


def _swiglu_own(s):
    if "shape" not in s:
        L, c = _lib(), s["case"]
        s["L"] = L
        s["shape"] = L.make_swiglu_shape(c["rows"], c["inter"], _dtype_of(L, c))
    if "a" in s:
        s["L"].moe_swiglu(s["shape"], s["gu"], s["a"])
        return {"a": s["a"]}
    s["L"].moe_swiglu_backward(s["shape"], s["gu"], s["da"], s["dgu"])
    return {"dgu": s["dgu"]}


def _ortho_own(s):
    if "shape" not in s:
        L, c = _lib(), s["case"]
        s["L"] = L
        s["shape"] = L.make_ortho_shape(c["mats"], c["rows"], c["cols"], NS_STEPS, _dtype_of(L, c))
        s["ws"] = _scratch(L.moe_orthogonalize_workspace_size(s["shape"]))
    s["L"].moe_orthogonalize(s["shape"], s["m"], s["o"], s["ws"])
    return {"o": s["o"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"grouped": _grouped_own, "norm": _norm_own, "swiglu": _swiglu_own, "ortho": _ortho_own}[op](state)
    return {"grouped": _grouped_plain, "norm": _norm_plain, "swiglu": _swiglu_plain, "ortho": _ortho_plain}[op](state)


# ------------------------------------------------------------ work and exact
def work(case):
    el = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "grouped":
        T, K, G, n, k = case["T"], case["top_k"], case["groups"], case["n"], case["k"]
        rows = T * K
        used = G * (1 - (1 - K / G) ** T)  # experts with at least one row, expected under uniform routing
        times = 3 if case["dir"] == "all" else 1
        x, y, w = rows * k * el, rows * n * el, used * n * k * el
        nbytes = {"fwd": x + w + y, "dx": y + w + x, "dw": x + y + G * n * k * el,
                  "all": 2 * x + 2 * y + w + G * n * k * el}[case["dir"]]
        return {"bytes": nbytes, "flops": times * 2.0 * rows * n * k}
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        if case["dir"] == "fwd":
            return {"bytes": 2 * T * d * el + 8 * d + 8 * T, "flops": 8.0 * T * d}
        return {"bytes": 5 * T * d * el + 20 * d + 16 * T, "flops": 24.0 * T * d}
    if case["op"] == "swiglu":
        e = case["rows"] * case["inter"]
        return {"bytes": (3 if case["dir"] == "fwd" else 5) * e * el, "flops": (5.0 if case["dir"] == "fwd" else 12.0) * e}
    m, r, c = case["mats"], case["rows"], case["cols"]
    lo, hi = min(r, c), max(r, c)
    # per step: the two symmetric products by one triangle each, the third in full
    return {"bytes": m * r * c * (el + 2), "flops": m * NS_STEPS * (3.0 * lo * lo * hi + lo ** 3)}


def exact(case, seed):
    """What run() returns for these inputs, from the definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "grouped":
        off = s["offsets"].tolist()
        spans = list(zip(off[:-1], off[1:]))
        x, w, dy = (s[t].double() if t in s else None for t in ("x", "w", "dy"))
        got = {}
        if "y" in s:
            got["y"] = torch.cat([torch.einsum("rk,nk->rn", x[a:b], w[e]) for e, (a, b) in enumerate(spans)])
        if "dx" in s:
            got["dx"] = torch.cat([torch.einsum("rn,nk->rk", dy[a:b], w[e]) for e, (a, b) in enumerate(spans)])
        if "dw" in s:
            got["dw"] = torch.stack([torch.einsum("rn,rk->nk", dy[a:b], x[a:b]) for a, b in spans])
        return got
    if case["op"] == "norm":
        x = s["x"].double()
        mean = x.sum(1) / x.shape[1]
        var = ((x - mean[:, None]) ** 2).sum(1) / x.shape[1]
        rstd = 1 / torch.sqrt(var + LN_EPS)
        gamma, beta = s["gamma"].double(), s["beta"].double()
        got = {"y": (x - mean[:, None]) * rstd[:, None] * gamma + beta, "mean": mean, "rstd": rstd}
        if "dy" in s:
            # the Jacobian of the normalised row applied to dy * gamma
            dy, d = s["dy"].double(), x.shape[1]
            h = (x - mean[:, None]) * rstd[:, None]
            v = dy * gamma
            got |= {"dx": (v - (v.sum(1)[:, None] + h * (h * v).sum(1)[:, None]) / d) * rstd[:, None],
                    "dgamma": torch.einsum("td,td->d", dy, h), "dbeta": dy.sum(0)}
        return got
    if case["op"] == "swiglu":
        gu = s["gu"].double().view(case["rows"], -1, 128)
        gate, up = gu[:, :, :64], gu[:, :, 64:]
        if case["dir"] == "fwd":
            return {"a": (torch.sigmoid(gate) * gate * up).reshape(case["rows"], -1)}
        da = s["da"].double().view(gate.shape)
        p = torch.sigmoid(gate)
        return {"dgu": torch.cat([da * up * (p + gate * p * (1 - p)), da * gate * p], 2).reshape(case["rows"], -1)}
    a, b, c = NS_COEF
    outs = []
    for mat in s["m"].double():
        z = mat / (torch.linalg.norm(mat) + 1e-7)
        for _ in range(NS_STEPS):
            if z.shape[0] <= z.shape[1]:
                q = z @ z.T
                z = a * z + b * (q @ z) + c * (q @ (q @ z))
            else:
                q = z.T @ z
                z = a * z + b * (z @ q) + c * ((z @ q) @ q)
        outs.append(z)
    return {"o": torch.stack(outs)}
