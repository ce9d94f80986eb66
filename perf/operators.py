"""The MLP block's operators as they are measured: the cases, their inputs, the plain forms and the
framework's calls.

Operators: the matrix product with bias, activation and residual in its epilogue (forward, and the
gradients for its input, weight and bias), the layer norm (forward and backward) and the AdamW step over
many tensors (states in 32 or in 8 bits).

Sizes are those of the layers this repository computes elsewhere: h=4096 (Megatron-SP, sequence 4096,
fc1 shards of 2048 columns), h=12288 (GPT-3, sequence 2048, QKV shards of 4608 columns) and h=8192,
ffn=28672 (the MLP sweep, 3584 columns a rank of eight).
"""

import math

import torch

own = False   # False: run() computes the plain forms; True: it calls the framework's operators

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
QBLOCK = 256   # elements that share a scale of the 8-bit optimizer states
E4M3_MAX = 448.0
LARGEST_PRODUCT = 8192 * 8192 * 28672   # M*K*n of the largest listed matrix product


# ---- cases ------------------------------------------------------------------------------------------
def listed():
    return [
        # one token through one rank's fc1 shard: the shortest call of a decoding loop
        {"name": "linear_fc1_1tok", "op": "linear", "M": 1, "K": 4096, "n": 2048, "act": "gelu_tanh", "bias": "bf16",
         "residual": False, "preact": False, "layout": "nk", "out": "bf16"},
        # one token through the whole fc2 of the MLP: the weights' bytes are all there is
        {"name": "linear_fc2_1tok", "op": "linear", "M": 1, "K": 28672, "n": 8192, "act": "none", "bias": "bf16",
         "residual": True, "preact": False, "layout": "nk", "out": "bf16"},
        # a ragged batch of decoding sequences, inner and output extents that are no multiple of a tile
        {"name": "linear_ragged_45tok", "op": "linear", "M": 45, "K": 8190, "n": 3579, "act": "silu", "bias": "f32",
         "residual": True, "preact": False, "layout": "nk", "out": "bf16"},
        # a prompt of ordinary length through a rank's QKV columns, weights stored [K][n]
        {"name": "linear_prompt_1000tok", "op": "linear", "M": 1000, "K": 12288, "n": 4608, "act": "none",
         "bias": "bf16", "residual": False, "preact": False, "layout": "kn", "out": "bf16"},
        # fc1 of the MLP over the training sequence, pre-activation kept for the backward pass
        {"name": "linear_fc1_train", "op": "linear", "M": 8192, "K": 8192, "n": 28672, "act": "gelu_tanh",
         "bias": "bf16", "residual": False, "preact": True, "layout": "nk", "out": "bf16"},
        # all gradients of an fc2: dx through the activation in front of it, dW, db
        {"name": "linear_grad_train", "op": "linear_grad", "M": 4096, "K": 16384, "n": 4096, "act": "gelu",
         "residual": False, "layout": "nk", "out": "bf16"},
        # the same for a short, odd batch (fine-tuning on one short sample)
        {"name": "linear_grad_77tok", "op": "linear_grad", "M": 77, "K": 4096, "n": 2044, "act": "silu",
         "residual": True, "layout": "nk", "out": "bf16"},
        # layer norm in front of a decoding step
        {"name": "norm_3tok", "op": "norm", "rows": 3, "h": 12288, "x": "bf16", "out": "bf16", "params": "bf16"},
        # layer norm over the training sequence, forward and backward
        {"name": "norm_train", "op": "norm", "rows": 8192, "h": 8192, "x": "bf16", "out": "bf16", "params": "bf16"},
        {"name": "norm_grad_train", "op": "norm_grad", "rows": 8192, "h": 8192, "x": "bf16", "out": "bf16",
         "params": "bf16", "residual": True},
        # one rank's MLP block: two matrices, their biases and the norm's vectors, fp32 states and master weights
        {"name": "adamw_rank_f32", "op": "adamw", "matrices": 2, "rows": 3584, "h": 8192, "vectors": 4, "bits": 32,
         "grad": "bf16", "master": True},
        # the matrices of the h=4096 block, 8-bit states, fp32 main gradients, and many short vectors
        {"name": "adamw_many_8bit", "op": "adamw", "matrices": 6, "rows": 2048, "h": 4096, "vectors": 60, "bits": 8,
         "grad": "f32", "master": True},
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_grad", "norm", "norm_grad", "adamw"))
    if op in ("linear", "linear_grad"):
        while True:
            M, K, n = _logint(rng, 1, 8192), _logint(rng, 96, 28672), _logint(rng, 64, 28672)
            if M * K * n * (2 if op == "linear_grad" else 1) <= LARGEST_PRODUCT:
                break
        if rng.random() < 0.5:   # the usual extents; the others stay ragged
            K, n = -(-K // 64) * 64, -(-n // 64) * 64
            if M * K * n * (2 if op == "linear_grad" else 1) > LARGEST_PRODUCT:
                M = max(1, M // 2)
        act = rng.choice(ACTS)
        c = {"op": op, "M": M, "K": K, "n": n, "act": act, "residual": rng.random() < 0.5,
             "layout": rng.choice(("nk", "nk", "kn")), "out": "bf16"}
        if op == "linear":
            c["bias"] = rng.choice(("none", "bf16", "f32"))
            c["preact"] = act != "none" and rng.random() < 0.5
        return c
    if op in ("norm", "norm_grad"):
        while True:
            rows, h = _logint(rng, 1, 65536), _logint(rng, 64, 28672)
            if rows * h <= 8192 * 8192:
                break
        if rng.random() < 0.5:
            h = -(-h // 64) * 64
        c = {"op": op, "rows": rows, "h": h, "x": rng.choice(("bf16", "bf16", "f32")),
             "out": rng.choice(("bf16", "bf16", "f32")), "params": rng.choice(("bf16", "f32"))}
        if op == "norm_grad":
            c["residual"] = rng.random() < 0.5
        return c
    while True:
        c = {"op": "adamw", "matrices": rng.randint(1, 12), "rows": _logint(rng, 1, 8192), "h": _logint(rng, 64, 12288),
             "vectors": rng.randint(0, 200), "bits": rng.choice((8, 32)), "grad": rng.choice(("bf16", "f32")),
             "master": rng.random() < 0.6}
        if c["matrices"] * c["rows"] * c["h"] <= 100_000_000:
            return c


# ---- inputs -----------------------------------------------------------------------------------------
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _rows(r, c, dtype=torch.bfloat16):
    """[r][c] with rows that start on 16 bytes: a view of a wider buffer where c is ragged."""
    return torch.zeros(r, -(-c // 8) * 8, dtype=dtype, device="cuda")[:, :c]


def _normal(g, shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
    t = _rows(shape[0], shape[1], dtype) if len(shape) == 2 else torch.empty(shape, dtype=dtype, device="cuda")
    t.copy_(torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean))
    return t


def _adamw_numels(case):
    """Matrices, then vectors of the lengths that biases and norms have, some of them odd."""
    many = [case["rows"] * case["h"]] * case["matrices"]
    return many + [(case["h"], case["rows"], case["h"] + 1, 1 + case["h"] // 3)[i % 4] for i in range(case["vectors"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op in ("linear", "linear_grad"):
        M, K, n = case["M"], case["K"], case["n"]
        s["w"] = _normal(g, (n, K) if case["layout"] == "nk" else (K, n), 0.02)
        if op == "linear":
            s["x_"] = _normal(g, (M, K))
            s["b"] = None if case["bias"] == "none" else _normal(g, (n,), 0.1, dtype=_dtype(case["bias"]))
            s["r"] = _normal(g, (M, n)) if case["residual"] else None
            s["z"] = _rows(M, n) if case["preact"] else None
            s["y"] = _rows(M, n, _dtype(case["out"]))
        else:
            s["z"] = _normal(g, (M, K), 1.2)             # what the layer in front kept
            s["x_"] = _rows(M, K)
            s["x_"].copy_(_act32(s["z"].float(), case["act"]))
            s["dy"] = _normal(g, (M, n), 0.01)
            s["r"] = _normal(g, (M, K), 0.01) if case["residual"] else None
            s["dx"] = _rows(M, K, _dtype(case["out"]))
            s["dw"] = _rows(n if case["layout"] == "nk" else K, K if case["layout"] == "nk" else n, _dtype(case["out"]))
            s["db"] = torch.empty(n, dtype=torch.float32, device="cuda")
            if own:
                from collective_matmul_decomposition_gb300 import cm
                s["ws"] = torch.empty(cm.linear_wgrad_workspace_size(M, K, n), dtype=torch.uint8, device="cuda")
    elif op in ("norm", "norm_grad"):
        rows, h = case["rows"], case["h"]
        xd, yd, pd = _dtype(case["x"]), _dtype(case["out"]), _dtype(case["params"])
        s["x_"] = _normal(g, (rows, h), 1.5, 0.25, dtype=xd)
        s["gamma"] = _normal(g, (h,), 0.1, 1.0, dtype=pd)
        s["beta"] = _normal(g, (h,), 0.1, dtype=pd)
        s["eps"] = 1e-5
        if op == "norm":
            s["y"] = _rows(rows, h, yd)
            s["mean"] = torch.empty(rows, dtype=torch.float32, device="cuda")
            s["rstd"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        else:
            x = s["x_"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = (x - s["mean"][:, None]).square().mean(1).add(s["eps"]).rsqrt()
            s["dy"] = _normal(g, (rows, h), 0.02, dtype=yd)
            s["r"] = _normal(g, (rows, h), 0.02, dtype=xd) if case["residual"] else None
            s["dx"] = _rows(rows, h, xd)
            s["dgamma"] = torch.empty(h, dtype=torch.float32, device="cuda")
            s["dbeta"] = torch.empty(h, dtype=torch.float32, device="cuda")
            if own:
                from collective_matmul_decomposition_gb300 import cm
                s["ws"] = torch.empty(cm.layer_norm_backward_workspace_size(rows, h), dtype=torch.uint8, device="cuda")
    else:
        # every tensor is a view of a flat buffer, each starting on a block of its own, as trainers keep them
        numels = _adamw_numels(case)
        starts, total = [], 0
        for k in numels:
            starts.append(total)
            total += -(-k // QBLOCK) * QBLOCK
        blocks = total // QBLOCK
        s["numels"], s["starts"], s["total"] = numels, starts, total
        # the padding behind a tensor's end holds zeros, and a step leaves it so
        live = torch.zeros(total, device="cuda")
        for k, o in zip(numels, starts):
            live[o:o + k] = 1
        master = torch.randn(total, generator=g, device="cuda").mul_(0.02).mul_(live)
        s["param"] = master.bfloat16()
        s["master"] = master if case["master"] else None
        s["grad"] = torch.randn(total, generator=g, device="cuda").mul_(1e-3).mul_(live).to(_dtype(case["grad"]))
        m = torch.randn(total, generator=g, device="cuda").mul_(3e-4).mul_(live)
        v = torch.randn(total, generator=g, device="cuda").square_().mul_(1e-6).mul_(live)
        s["ms"] = s["vs"] = None
        if case["bits"] == 32:
            s["m"], s["v"] = m, v
        else:
            s["m"], s["ms"] = _quantise(m.view(blocks, QBLOCK), False)
            s["v"], s["vs"] = _quantise(v.sqrt_().view(blocks, QBLOCK), True)
        s["lr"], s["beta1"], s["beta2"], s["eps"], s["step"] = 3e-4, 0.9, 0.95, 1e-8, 100
        s["wd"] = [0.1] * case["matrices"] + [0.0] * case["vectors"]
        s["scale"] = torch.full((), 0.8, dtype=torch.float32, device="cuda")   # the gradient clip's factor
        if own:
            # the optimizer's list of tensors, which a training loop makes once
            from collective_matmul_decomposition_gb300 import cm
            tensors = cm.AdamWTensors()
            for k, o, wd in zip(numels, starts, s["wd"]):
                sl, bl = slice(o, o + k), slice(o // QBLOCK, o // QBLOCK + -(-k // QBLOCK))
                tensors.add(s["param"][sl], s["grad"][sl], s["m"][sl], s["v"][sl],
                            exp_avg_scale=None if s["ms"] is None else s["ms"][bl],
                            exp_avg_sq_scale=None if s["vs"] is None else s["vs"][bl],
                            master=None if s["master"] is None else s["master"][sl], weight_decay=wd)
            s["tensors"] = tensors
    return s


# ---- the plain forms: elementary operations in 32 bits ----------------------------------------------
def _act32(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _dact32(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    return torch.ones_like(z)


def _quantise(t, root):
    """Blocks of QBLOCK values (one row each) as e4m3 codes times a scale; a positive root keeps a code above zero."""
    amax = torch.where(torch.isfinite(t), t.abs(), torch.zeros_like(t)).amax(1)
    live = amax >= 2.0 ** -100
    inv = torch.where(live, E4M3_MAX / amax, torch.zeros_like(amax))
    q = (t * inv[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).float()
    if root:
        q = torch.where((q == 0) & (t > 0) & live[:, None], torch.full_like(q, 2.0 ** -9), q)
    q = torch.where(torch.isfinite(t), q, torch.full_like(q, float("nan")))
    scale = torch.where(live, amax / E4M3_MAX, torch.zeros_like(amax))
    return q.to(torch.float8_e4m3fn).reshape(-1), scale


def _plain(s):
    op = s["op"]
    if op == "linear":
        w = s["w"].float()
        z = s["x_"].float() @ (w.t() if s["layout"] == "nk" else w)
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act32(z, s["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return {"y": y.to(s["y"].dtype), "z": None if s["z"] is None else z.bfloat16()}
    if op == "linear_grad":
        w, dy, x = s["w"].float(), s["dy"].float(), s["x_"].float()
        dx = dy @ (w if s["layout"] == "nk" else w.t())
        if s["act"] != "none":
            dx = dx * _dact32(s["z"].float(), s["act"])
        if s["r"] is not None:
            dx = dx + s["r"].float()
        dw = dy.t() @ x if s["layout"] == "nk" else x.t() @ dy
        return {"dx": dx.to(s["dx"].dtype), "dw": dw.to(s["dw"].dtype), "db": dy.sum(0)}
    if op == "norm":
        x = s["x_"].float()
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = 1 / torch.sqrt(d.square().mean(1) + s["eps"])
        y = d * rstd[:, None] * s["gamma"].float() + s["beta"].float()
        return {"y": y.to(s["y"].dtype), "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        x, dy = s["x_"].float(), s["dy"].float()
        xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
        t = dy * s["gamma"].float()
        dx = (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
        if s["r"] is not None:
            dx = dx + s["r"].float()
        return {"dx": dx.to(s["dx"].dtype), "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}
    # AdamW: the flat buffers at once; the matrices decay, the vectors behind them do not
    c1, c2 = 1 - s["beta1"] ** s["step"], 1 - s["beta2"] ** s["step"]
    g = s["grad"].float() * s["scale"]
    if s["bits"] == 8:
        m = (s["m"].float().view(-1, QBLOCK) * s["ms"][:, None]).view(-1)
        v = (s["v"].float().view(-1, QBLOCK) * s["vs"][:, None]).view(-1).square()
    else:
        m, v = s["m"], s["v"]
    m = s["beta1"] * m + (1 - s["beta1"]) * g
    v = s["beta2"] * v + (1 - s["beta2"]) * g * g
    root = torch.sqrt(v)
    p = s["param"].float() if s["master"] is None else s["master"].clone()
    cut = s["starts"][s["matrices"]] if s["vectors"] else s["total"]
    p[:cut] *= 1 - s["lr"] * s["wd"][0]
    p -= (s["lr"] / c1) * m / (root * (1 / math.sqrt(c2)) + s["eps"])
    s["param"].copy_(p)
    if s["master"] is not None:
        s["master"].copy_(p)
    if s["bits"] == 8:
        for_m, for_v = _quantise(m.view(-1, QBLOCK), False), _quantise(root.view(-1, QBLOCK), True)
        s["m"].copy_(for_m[0])
        s["ms"].copy_(for_m[1])
        s["v"].copy_(for_v[0])
        s["vs"].copy_(for_v[1])
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    return {k: s[k] for k in ("param", "master", "m", "v", "ms", "vs")}


# ---- the framework's operators ----------------------------------------------------------------------
def _own(s):
    from collective_matmul_decomposition_gb300 import cm
    op = s["op"]
    if op == "linear":
        cm.cm_linear(s["x_"], s["w"], s["y"], bias=s["b"], act=s["act"], residual=s["r"], preact=s["z"],
                     w_layout=s["layout"])
        return {"y": s["y"], "z": s["z"]}
    if op == "linear_grad":
        cm.cm_linear_dgrad(s["dy"], s["w"], s["dx"], preact=s["z"], act=s["act"], residual=s["r"],
                           w_layout=s["layout"])
        cm.cm_linear_wgrad(s["x_"], s["dy"], s["dw"], s["ws"], db=s["db"], w_layout=s["layout"])
        return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    if op == "norm":
        cm.cm_layer_norm(s["x_"], s["y"], s["gamma"], s["beta"], eps=s["eps"], mean=s["mean"], rstd=s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "norm_grad":
        cm.cm_layer_norm_backward(s["x_"], s["dy"], s["gamma"], s["mean"], s["rstd"], s["dx"], s["ws"],
                                  dgamma=s["dgamma"], dbeta=s["dbeta"], residual=s["r"])
        return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    cm.cm_adamw(s["tensors"], lr=s["lr"], beta1=s["beta1"], beta2=s["beta2"], eps=s["eps"], step=s["step"],
                grad_scale=s["scale"])
    return _adamw_outputs(s)


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "linear":
        M, K, n = case["M"], case["K"], case["n"]
        elems = M * K + K * n + M * n * (1 + case["residual"] + case["preact"])
        return {"bytes": 2 * elems + n * {"none": 0, "bf16": 2, "f32": 4}[case["bias"]], "flops": 2 * M * K * n}
    if op == "linear_grad":
        M, K, n = case["M"], case["K"], case["n"]
        elems = M * n + K * n + M * K * (1 + case["residual"] + (case["act"] != "none")) + M * K + K * n
        return {"bytes": 2 * elems + 4 * n, "flops": 4 * M * K * n}
    if op in ("norm", "norm_grad"):
        rows, h = case["rows"], case["h"]
        xs, ys, ps = (2 if case[k] == "bf16" else 4 for k in ("x", "out", "params"))
        if op == "norm":
            return {"bytes": rows * h * (xs + ys) + 2 * h * ps + 8 * rows, "flops": 8 * rows * h}
        return {"bytes": rows * h * (xs * (2 + case["residual"]) + ys) + h * (ps + 8) + 8 * rows, "flops": 14 * rows * h}
    total = sum(_adamw_numels(case))
    state = 16 if case["bits"] == 32 else 4 + 16 / QBLOCK
    each = (2 if case["grad"] == "bf16" else 4) + state + (8 + 2 if case["master"] else 4)
    return {"bytes": int(total * each), "flops": 16 * total}


# ---- the definitions in 64 bits ---------------------------------------------------------------------
def _act64(z, act):
    """(act(z), act'(z)) in float64."""
    one = torch.ones_like(z)
    if act == "none":
        return z, one
    if act == "relu":
        return torch.maximum(z, torch.zeros_like(z)), torch.where(z > 0, one, torch.zeros_like(z))
    if act == "silu":
        sg = torch.sigmoid(z)
        return z * sg, sg + z * sg * (1 - sg)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    sg = torch.sigmoid(2 * u)   # (1 + tanh u) / 2
    return z * sg, sg + 2 * z * sg * (1 - sg) * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)


def exact(case, seed):
    s = prepare({**case}, seed)
    op = case["op"]
    if op == "linear":
        w = s["w"].double()
        z = torch.mm(s["x_"].double(), w.T if case["layout"] == "nk" else w)
        del w
        if s["b"] is not None:
            z += s["b"].double()
        keep = z.clone() if case["preact"] else None
        y = _act64(z, case["act"])[0]
        if s["r"] is not None:
            y = y + s["r"].double()
        return {"y": y, "z": keep}
    if op == "linear_grad":
        dy = s["dy"].double()
        w = s["w"].double()
        dx = torch.mm(dy, w if case["layout"] == "nk" else w.T)
        del w
        dx *= _act64(s["z"].double(), case["act"])[1]
        if s["r"] is not None:
            dx += s["r"].double()
        x = s["x_"].double()
        dw = torch.mm(dy.T, x) if case["layout"] == "nk" else torch.mm(x.T, dy)
        return {"dx": dx, "dw": dw, "db": dy.sum(dim=0)}
    if op == "norm":
        x = s["x_"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + s["eps"]) ** -0.5
        y = (x - mean.unsqueeze(1)) * (rstd.unsqueeze(1) * s["gamma"].double()) + s["beta"].double()
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        rstd = s["rstd"].double().unsqueeze(1)
        xh = (s["x_"].double() - s["mean"].double().unsqueeze(1)) * rstd
        dy = s["dy"].double()
        t = dy * s["gamma"].double()
        h = case["h"]
        dx = rstd * (t - t.sum(1, keepdim=True) / h - xh * ((t * xh).sum(1, keepdim=True) / h))
        if s["r"] is not None:
            dx += s["r"].double()
        return {"dx": dx, "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}
    # tensor by tensor; codes and scales of 8-bit states have no 64-bit value of their own
    out = {k: None for k in ("param", "master", "m", "v", "ms", "vs")}
    src = s["master"] if s["master"] is not None else s["param"]
    p = src.double()
    m = s["m"].double()
    v = s["v"].double()
    if case["bits"] == 8:
        m *= s["ms"].double().repeat_interleave(QBLOCK)
        v = (v * s["vs"].double().repeat_interleave(QBLOCK)) ** 2
    for k, o, wd in zip(s["numels"], s["starts"], s["wd"]):
        at = slice(o, o + k)
        g = s["grad"][at].double() * float(s["scale"])
        m[at] = s["beta1"] * m[at] + (1 - s["beta1"]) * g
        v[at] = s["beta2"] * v[at] + (1 - s["beta2"]) * g ** 2
        mh, vh = m[at] / (1 - s["beta1"] ** s["step"]), v[at] / (1 - s["beta2"] ** s["step"])
        p[at] = p[at] - s["lr"] * wd * p[at] - s["lr"] * mh / (vh.sqrt() + s["eps"])
    out["param"] = p
    if s["master"] is not None:
        out["master"] = p
    if case["bits"] == 32:
        out["m"], out["v"] = m, v
    return out
