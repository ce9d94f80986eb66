"""The ends of a language model and the gated MLP between them as they are measured: the cases, their inputs, the
plain forms and the framework's calls.

Operators: the gated product act(x Wg^T + bg) * (x Wu^T + bu) and its data gradient; the cross entropy of x W^T over a
vocabulary, of which no logits are kept, and its gradients; the embedding lookup and its gradient.

Sizes are those of the layers this repository computes elsewhere (h=4096 with fc1 shards of 2048 columns, h=8192 with
ffn=28672 and shards of 3584 columns, h=12288) with vocabularies of 2^15 to 2^17 tokens, whole, odd or a slice of one.
"""

import math

import torch

own = False   # False: run() computes the plain forms; True: it calls the framework's operators

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
LARGEST_GATED = 4096 * 8192 * 28672   # M*K*n of the largest listed gated product
LARGEST_HEAD = 8192 * 4096 * 131072   # M*K*V of the largest listed loss; the gradients take three times the products


# ---- cases ------------------------------------------------------------------------------------------
def listed():
    return [
        # one token through one rank's gated columns: the shortest call of a decoding loop
        {"name": "gated_1tok", "op": "gated", "M": 1, "K": 4096, "n": 2048, "act": "silu", "bias": "none",
         "keep": False, "layout": "nk"},
        # the gated MLP over a training sequence, both pre-activations kept for the backward pass
        {"name": "gated_train", "op": "gated", "M": 4096, "K": 8192, "n": 28672, "act": "silu", "bias": "none",
         "keep": True, "layout": "nk"},
        # back through the down projection and the gate: a short odd batch (fine-tuning on one sample), and a sequence
        {"name": "gated_grad_77tok", "op": "gated_grad", "M": 77, "f": 4093, "n": 2044, "act": "gelu", "layout": "nk"},
        {"name": "gated_grad_train", "op": "gated_grad", "M": 4096, "f": 16384, "n": 4096, "act": "gelu_tanh",
         "layout": "nk"},
        # scoring one token against a small vocabulary
        {"name": "loss_1tok", "op": "loss", "M": 1, "K": 4096, "V": 32768, "first": 0, "total": 32768, "ignored": 0,
         "ids": 64, "layout": "nk"},
        # the loss of a training sequence over a large vocabulary
        {"name": "loss_train", "op": "loss", "M": 8192, "K": 4096, "V": 131072, "first": 0, "total": 131072,
         "ignored": 0, "ids": 64, "layout": "nk"},
        # its gradients for a fine-tuning batch: odd sizes, the prompt's tokens carry no loss, a slice of the vocabulary
        {"name": "loss_grad_ragged", "op": "loss_grad", "M": 1003, "K": 4101, "V": 16381, "first": 16384,
         "total": 50001, "ignored": 350, "ids": 64, "layout": "nk"},
        {"name": "loss_grad_train", "op": "loss_grad", "M": 4096, "K": 4096, "V": 131072, "first": 0, "total": 131072,
         "ignored": 0, "ids": 64, "layout": "nk"},
        # the rows of a small decoding batch, and of a training sequence
        {"name": "embed_3tok", "op": "embed", "T": 3, "h": 12288, "V": 32768, "first": 0, "total": 32768, "pad": 0,
         "spread": "uniform", "ids": 64, "w": "bf16", "out": "bf16"},
        {"name": "embed_train", "op": "embed", "T": 16384, "h": 8192, "V": 131072, "first": 0, "total": 131072, "pad": 0,
         "spread": "zipf", "ids": 64, "w": "bf16", "out": "bf16"},
        # the whole gradient of the matrix, rows of absent tokens as zeros
        {"name": "embed_grad_train", "op": "embed_grad", "T": 16384, "h": 4096, "V": 131072, "first": 0, "total": 131072,
         "pad": 0, "spread": "zipf", "ids": 64, "dy": "bf16", "out": "f32", "accumulate": False},
        # added to the gradient that the loss has left in the tied matrix: a slice of the vocabulary, odd rows, padding
        {"name": "embed_grad_tied", "op": "embed_grad", "T": 10007, "h": 4100, "V": 16384, "first": 16384, "total": 65536,
         "pad": 900, "spread": "zipf", "ids": 32, "dy": "bf16", "out": "f32", "accumulate": True},
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("gated", "gated_grad", "loss", "loss_grad", "embed", "embed_grad"))
    layout = rng.choice(("nk", "nk", "kn"))
    even = rng.random() < 0.5   # the usual extents; the others stay ragged
    if op in ("gated", "gated_grad"):
        while True:
            M, K, n = _logint(rng, 1, 8192), _logint(rng, 64, 16384), _logint(rng, 64, 28672)
            if even:
                K, n = -(-K // 64) * 64, -(-n // 64) * 64
            if M * K * n <= LARGEST_GATED:
                break
        act = rng.choice(ACTS)
        if op == "gated_grad":
            return {"op": op, "M": M, "f": n, "n": K, "act": act, "layout": layout}
        return {"op": op, "M": M, "K": K, "n": n, "act": act, "bias": rng.choice(("none", "none", "bf16", "f32")),
                "keep": rng.random() < 0.5, "layout": layout}
    if op in ("loss", "loss_grad"):
        while True:
            M, K, V = _logint(rng, 1, 8192), _logint(rng, 64, 12288), _logint(rng, 512, 131072)
            if even:
                K, V = -(-K // 64) * 64, -(-V // 64) * 64
            if M * V <= 1 << 30 and M * K * V * (3 if op == "loss_grad" else 1) <= LARGEST_HEAD * 1.5:
                break
        first = rng.choice((0, 0, V, 3 * V))
        return {"op": op, "M": M, "K": K, "V": V, "first": first, "total": V if not first else first + rng.choice((1, 2)) * V,
                "ignored": rng.choice((0, M // 10, M // 2, M - 1)), "ids": rng.choice((32, 64)), "layout": layout}
    while True:
        T, h, V = _logint(rng, 1, 65536), _logint(rng, 64, 12288), _logint(rng, 256, 131072)
        if even:
            h = -(-h // 64) * 64
        if T * h <= 1 << 27 and V * h <= 1 << 29:
            break
    first = rng.choice((0, 0, V))
    c = {"op": op, "T": T, "h": h, "V": V, "first": first, "total": V if not first else 3 * V, "pad": rng.choice((0, T // 8)),
         "spread": rng.choice(("uniform", "zipf")), "ids": rng.choice((32, 64))}
    if op == "embed":
        return {**c, "w": rng.choice(("bf16", "bf16", "f32")), "out": rng.choice(("bf16", "bf16", "f32"))}
    return {**c, "dy": rng.choice(("bf16", "bf16", "f32")), "out": rng.choice(("f32", "f32", "bf16")),
            "accumulate": rng.random() < 0.5}


# ---- inputs -----------------------------------------------------------------------------------------
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _rows(r, c, dtype=torch.bfloat16):
    """[r][c] with rows that start on 16 bytes: a view of a wider buffer where c is ragged."""
    return torch.zeros(r, -(-c // 8) * 8, dtype=dtype, device="cuda")[:, :c]


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    t = _rows(shape[0], shape[1], dtype) if len(shape) == 2 else torch.empty(shape, dtype=dtype, device="cuda")
    t.copy_(torch.randn(shape, generator=g, device="cuda").mul_(std))
    return t


def _ids(g, count, case, none, spread="zipf"):
    """Token ids below case["total"], the frequent ones scattered over it; `none` of them, at random places, are -100."""
    u = torch.rand(count, generator=g, device="cuda", dtype=torch.float64)
    total = case["total"]
    if spread == "zipf":   # the k-th most frequent id with probability 1/k
        t = (torch.exp(u * math.log(total + 1)).long() - 1).clamp_(0, total - 1)
        t = (t * 1000003 + 12345) % total
    else:
        t = (u * total).long().clamp_(0, total - 1)
    t[torch.randperm(count, generator=g, device="cuda")[:none]] = -100
    return t if case["ids"] == 64 else t.int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op in ("gated", "gated_grad"):
        M = case["M"]
        if op == "gated":
            K, n = case["K"], case["n"]
            s["x_"] = _normal(g, (M, K))
            shape = (n, K) if case["layout"] == "nk" else (K, n)
            s["wg"], s["wu"] = _normal(g, shape, 0.02), _normal(g, shape, 0.02)
            s["bg"] = s["bu"] = s["zg"] = s["zu"] = None
            if case["bias"] != "none":
                s["bg"], s["bu"] = (_normal(g, (n,), 0.1, _dtype(case["bias"])) for _ in range(2))
            if case["keep"]:
                s["zg"], s["zu"] = _rows(M, n), _rows(M, n)
            s["y"] = _rows(M, n)
        else:
            f, n = case["f"], case["n"]
            s["dy"] = _normal(g, (M, n), 0.01)
            s["w_"] = _normal(g, (n, f) if case["layout"] == "nk" else (f, n), 0.02)
            s["zg"], s["zu"] = _normal(g, (M, f), 1.2), _normal(g, (M, f), 1.2)
            s["dzg"], s["dzu"] = _rows(M, f), _rows(M, f)
    elif op in ("loss", "loss_grad"):
        M, K, V = case["M"], case["K"], case["V"]
        s["x_"] = _normal(g, (M, K))
        s["w_"] = _normal(g, (V, K) if case["layout"] == "nk" else (K, V), 1.5 * K ** -0.5)
        s["t"] = _ids(g, M, case, case["ignored"])
        if op == "loss":
            s["loss"], s["lse"] = (torch.empty(M, dtype=torch.float32, device="cuda") for _ in range(2))
        else:
            # what the forward pass left: over the whole vocabulary, of which this may be a slice
            s["lse"] = (math.log(case["total"]) + 1.125 + 0.1 * torch.randn(M, generator=g, device="cuda"))
            s["lse"][s["t"] < 0] = 0
            s["dloss"] = torch.full((M,), 1.0 / max(1, M - case["ignored"]), dtype=torch.float32, device="cuda")
            s["dx"] = _rows(M, K)
            s["dw"] = _rows(V if case["layout"] == "nk" else K, K if case["layout"] == "nk" else V)
        if own:
            from collective_matmul_decomposition_gb300 import cm
            size = cm.linear_cross_entropy_workspace_size if op == "loss" else cm.linear_cross_entropy_backward_workspace_size
            s["ws"] = torch.empty(size(M, K, V), dtype=torch.uint8, device="cuda")
    else:
        T, h, V = case["T"], case["h"], case["V"]
        s["t"] = _ids(g, T, case, case["pad"], case["spread"])
        s["scale"] = math.sqrt(h) if op == "embed" else 0.5
        if op == "embed":
            s["w_"] = _normal(g, (V, h), 0.02, _dtype(case["w"]))
            s["y"] = _rows(T, h, _dtype(case["out"]))
        else:
            s["dy"] = _normal(g, (T, h), 0.01, _dtype(case["dy"]))
            s["dw"] = _rows(V, h, _dtype(case["out"]))
            if case["accumulate"]:   # small, so that passes over one state add up to nothing large
                s["dw"].copy_(torch.randn(V, h, generator=g, device="cuda").mul_(0.01))
            if own:
                from collective_matmul_decomposition_gb300 import cm
                s["ws"] = torch.empty(cm.embedding_backward_workspace_size(T, h), dtype=torch.uint8, device="cuda")
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


def _plain(s):
    op = s["op"]
    nk = s.get("layout") == "nk"
    if op == "gated":
        x = s["x_"].float()
        zg, zu = (x @ (s[k].float().t() if nk else s[k].float()) for k in ("wg", "wu"))
        if s["bg"] is not None:
            zg, zu = zg + s["bg"].float(), zu + s["bu"].float()
        keep = s["zg"] is not None
        return {"y": (_act32(zg, s["act"]) * zu).bfloat16(), "zg": zg.bfloat16() if keep else None,
                "zu": zu.bfloat16() if keep else None}
    if op == "gated_grad":
        w = s["w_"].float()
        da = s["dy"].float() @ (w if nk else w.t())
        zg, zu = s["zg"].float(), s["zu"].float()
        return {"dzg": (da * zu * _dact32(zg, s["act"])).bfloat16(), "dzu": (da * _act32(zg, s["act"])).bfloat16()}
    if op in ("loss", "loss_grad"):
        x, w, t = s["x_"].float(), s["w_"].float(), s["t"].long()
        z = x @ (w.t() if nk else w)
        at = t - s["first"]
        here = (t >= 0) & (at >= 0) & (at < s["V"])
        at = at.clamp(0, s["V"] - 1)[:, None]
        if op == "loss":
            top = z.amax(1, keepdim=True)
            lse = torch.log(torch.exp(z - top).sum(1)) + top[:, 0]
            picked = torch.where(here, z.gather(1, at)[:, 0], torch.zeros_like(lse))
            counts = t >= 0
            return {"loss": torch.where(counts, lse - picked, torch.zeros_like(lse)),
                    "lse": torch.where(counts, lse, torch.zeros_like(lse))}
        scale = torch.where(t >= 0, s["dloss"], torch.zeros_like(s["dloss"]))
        p = torch.exp(z - s["lse"][:, None]) * scale[:, None]
        p.scatter_add_(1, at, torch.where(here, -scale, torch.zeros_like(scale))[:, None])
        return {"dx": (p @ (w if nk else w.t())).bfloat16(), "dw": (p.t() @ x if nk else x.t() @ p).bfloat16()}
    t = s["t"].long()
    at = t - s["first"]
    here = (t >= 0) & (at >= 0) & (at < s["V"])
    at = at.clamp(0, s["V"] - 1)
    if op == "embed":
        y = s["w_"][at].float() * s["scale"]
        return {"y": torch.where(here[:, None], y, torch.zeros_like(y)).to(s["y"].dtype)}
    dy = torch.where(here[:, None], s["dy"].float(), torch.zeros((), device="cuda"))
    dw = torch.zeros(s["dw"].shape, dtype=torch.float32, device="cuda").index_add_(0, at, dy) * s["scale"]
    s["dw"].copy_(dw + s["dw"].float() if s["accumulate"] else dw)
    return {"dw": s["dw"]}


# ---- the framework's operators ----------------------------------------------------------------------
def _own(s):
    from collective_matmul_decomposition_gb300 import cm
    op = s["op"]
    if op == "gated":
        cm.cm_linear_gated(s["x_"], s["wg"], s["wu"], s["y"], act=s["act"], bias_gate=s["bg"], bias_up=s["bu"],
                           z_gate=s["zg"], z_up=s["zu"], w_layout=s["layout"])
        return {"y": s["y"], "zg": s["zg"], "zu": s["zu"]}
    if op == "gated_grad":
        cm.cm_linear_gated_dgrad(s["dy"], s["w_"], s["dzg"], s["dzu"], s["zg"], s["zu"], act=s["act"], w_layout=s["layout"])
        return {"dzg": s["dzg"], "dzu": s["dzu"]}
    if op == "loss":
        cm.cm_linear_cross_entropy(s["x_"], s["w_"], s["t"], s["loss"], s["lse"], s["ws"], first=s["first"],
                                   vocab=s["total"], w_layout=s["layout"])
        return {"loss": s["loss"], "lse": s["lse"]}
    if op == "loss_grad":
        cm.cm_linear_cross_entropy_backward(s["x_"], s["w_"], s["t"], s["lse"], s["dloss"], s["ws"], dx=s["dx"], dw=s["dw"],
                                            first=s["first"], vocab=s["total"], w_layout=s["layout"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "embed":
        cm.cm_embedding(s["t"], s["w_"], s["y"], scale=s["scale"], first=s["first"])
        return {"y": s["y"]}
    cm.cm_embedding_backward(s["dy"], s["t"], s["dw"], s["ws"], scale=s["scale"], first=s["first"],
                             accumulate=s["accumulate"])
    return {"dw": s["dw"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "gated":
        M, K, n = case["M"], case["K"], case["n"]
        bias = {"none": 0, "bf16": 2, "f32": 4}[case["bias"]]
        return {"bytes": 2 * (M * K + 2 * K * n + M * n * (3 if case["keep"] else 1)) + 2 * n * bias, "flops": 4 * M * K * n}
    if op == "gated_grad":
        M, f, n = case["M"], case["f"], case["n"]
        return {"bytes": 2 * (M * n + n * f + 4 * M * f), "flops": 2 * M * f * n}
    if op in ("loss", "loss_grad"):
        M, K, V = case["M"], case["K"], case["V"]
        rows = M - case["ignored"]   # ignored rows need no product
        each = M * case["ids"] // 8
        if op == "loss":
            return {"bytes": 2 * (rows * K + K * V) + each + 8 * M, "flops": 2 * rows * K * V}
        return {"bytes": 2 * (rows * K + M * K + 2 * K * V) + each + 8 * M, "flops": 6 * rows * K * V}
    T, h, V = case["T"], case["h"], case["V"]
    share = case["V"] / case["total"] * (T - case["pad"])   # tokens whose row lies in the slice, in the mean
    each = T * case["ids"] // 8
    if op == "embed":
        # a row that several tokens share is read once: how many there are goes by the spread
        return {"bytes": int(min(V, _distinct(case)) * h * (2 if case["w"] == "bf16" else 4)
                             + T * h * (2 if case["out"] == "bf16" else 4)) + each, "flops": T * h}
    es = 2 if case["out"] == "bf16" else 4
    written = 2 * min(V, _distinct(case)) if case["accumulate"] else V
    return {"bytes": int(share * h * (2 if case["dy"] == "bf16" else 4) + written * h * es) + each, "flops": int(share * h)}


def _distinct(case):
    """Expected number of different rows of the slice among the tokens."""
    T, total = case["T"] - case["pad"], case["total"]
    if case["spread"] == "uniform":
        return case["V"] * -math.expm1(T * math.log1p(-1.0 / total)) if total > 1 else 1.0
    c, n = math.log(total + 1), 0.0
    lo = 1
    while lo <= total:   # ids of about one frequency together
        hi = min(total, lo + lo // 8)
        p = math.log((hi + 1) / lo) / c / (hi - lo + 1)
        n += (hi - lo + 1) * (-math.expm1(T * math.log1p(-p)) if p < 1 else 1.0)
        lo = hi + 1
    return n * case["V"] / total


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
    nk = case.get("layout") == "nk"
    if op == "gated":
        x = s["x_"].double()
        z = []
        for w, b in ((s["wg"], s["bg"]), (s["wu"], s["bu"])):
            z.append(torch.mm(x, w.double().T if nk else w.double()))
            if b is not None:
                z[-1] += b.double()
        y = _act64(z[0], case["act"])[0].mul_(z[1])
        return {"y": y, "zg": z[0] if case["keep"] else None, "zu": z[1] if case["keep"] else None}
    if op == "gated_grad":
        da = torch.mm(s["dy"].double(), s["w_"].double() if nk else s["w_"].double().T)
        a, da_dz = _act64(s["zg"].double(), case["act"])
        return {"dzg": da * s["zu"].double() * da_dz, "dzu": da * a}
    if op in ("loss", "loss_grad"):
        # the rows that count alone, by pieces of the vocabulary
        rows = torch.nonzero(s["t"] >= 0)[:, 0]
        x, t = s["x_"][rows].double(), s["t"][rows].long()
        w = s["w_"] if nk else s["w_"].T
        M, K, V, piece = len(rows), case["K"], case["V"], 16384
        zero = torch.zeros(case["M"], dtype=torch.float64, device="cuda")
        lse, picked = torch.full((M,), -math.inf, dtype=torch.float64, device="cuda"), zero[:M].clone()
        dx = torch.zeros(M, K, dtype=torch.float64, device="cuda")
        dw = []
        for lo in range(0, V, piece):
            part = w[lo:lo + piece].double()
            z = torch.mm(x, part.T)
            at = t - case["first"] - lo
            mine = torch.nonzero((at >= 0) & (at < len(part)))[:, 0]
            if op == "loss":
                lse = torch.logaddexp(lse, torch.logsumexp(z, dim=1))
                picked[mine] = z[mine, at[mine]]
                continue
            z.sub_(s["lse"][rows].double().unsqueeze(1)).exp_()
            z[mine, at[mine]] -= 1
            z *= s["dloss"][rows].double().unsqueeze(1)
            dx += torch.mm(z, part)
            dw.append(torch.mm(z.T, x))
        if op == "loss":
            loss, whole = zero.clone(), zero.clone()
            loss[rows], whole[rows] = lse - picked, lse
            return {"loss": loss, "lse": whole}
        full = torch.zeros(case["M"], K, dtype=torch.float64, device="cuda")
        full[rows] = dx
        dw = torch.cat(dw)
        return {"dx": full, "dw": dw if nk else dw.T}
    t = s["t"].long() - s["first"]
    rows = torch.nonzero((s["t"] >= 0) & (t >= 0) & (t < case["V"]))[:, 0]
    if op == "embed":
        y = torch.zeros(case["T"], case["h"], dtype=torch.float64, device="cuda")
        y[rows] = s["w_"][t[rows]].double() * s["scale"]
        return {"y": y}
    dw = s["dw"].double() if case["accumulate"] else torch.zeros(case["V"], case["h"], dtype=torch.float64, device="cuda")
    dw.index_add_(0, t[rows], s["dy"][rows].double() * s["scale"])
    return {"dw": dw}
