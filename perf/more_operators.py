"""Timed cases of the operators around a stage's block: linear maps with their
epilogue, layer norm, embedding.

A case is a dict of plain values; ``prepare`` makes what a user's program has
in hand before the call, ``run`` makes one pass through one operator and
returns its outputs, ``work`` gives the bytes and operations the pass cannot
do without, ``exact`` the same outputs from the definition in 64 bits.  With
``own`` false ``run`` computes the operator in its plain form (elementary
torch operations in 32 bits, rounded once at the end); with ``own`` true it
calls the library.

Operators (``op`` of a case); ``bits`` is the type of the residual stream
  linear      D = X W (or X W^T).  store: D + b + R;  gelu: GeLU(D + b) + R,
              with D + b kept where ``save``;  grad: D GeLU'(H) + R
  norm        layer norm.  part fwd: y with the rows' mean and 1/deviation;
              bwd: dx (with the residual's gradient added, and a bf16 copy of
              an fp32 one), then the sums over rows dgamma and dbeta
  embedding   part lookup: rows of the table times a scale;  grad: the tokens'
              order by id, then the table's gradient
"""

import math
import random

import numpy as np
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
INV_SQRT2 = 1.0 / math.sqrt(2.0)
INV_SQRT_2PI = 1.0 / math.sqrt(2.0 * math.pi)
EPS = 1e-5


# --------------------------------------------------------------------- cases
def listed():
    return [
        # the block's second product for a decoding step of 16 sequences: latency, and reading W
        {"name": "linear_few", "op": "linear", "rows": 16, "n": 1024, "k": 4096, "form": "store", "transposed": False,
         "bits": 16, "bias": True, "residual": True, "save": False, "gap": 0},
        # gradient of a square projection of a small microbatch, joined with the residual's gradient
        {"name": "linear_small_bwd", "op": "linear", "rows": 512, "n": 1024, "k": 1024, "form": "store",
         "transposed": True, "bits": 16, "bias": False, "residual": True, "save": False, "gap": 0},
        # an odd number of tokens and odd widths, the operand a slice of a wider buffer, nothing kept for a backward pass
        {"name": "linear_ragged_gelu", "op": "linear", "rows": 2047, "n": 4104, "k": 1032, "form": "gelu",
         "transposed": False, "bits": 16, "bias": True, "residual": True, "save": False, "gap": 64},
        # gradient through an activation with a residual around both, a microbatch of 4 x 1024 tokens
        {"name": "linear_gelu_bwd", "op": "linear", "rows": 4096, "n": 4096, "k": 1024, "form": "grad",
         "transposed": True, "bits": 16, "bias": False, "residual": True, "save": False, "gap": 0},
        # output projection of the h = 4096 block onto an fp32 residual stream: bound by the matrix product
        {"name": "linear_train_fp32", "op": "linear", "rows": 8192, "n": 4096, "k": 4096, "form": "store",
         "transposed": False, "bits": 32, "bias": True, "residual": True, "save": False, "gap": 0},
        # a decoding step's norm: pure latency
        {"name": "norm_few", "op": "norm", "part": "fwd", "rows": 16, "width": 1024, "bits": 16, "beta": True},
        # a microbatch of 4 x 2048 tokens at h = 4096, fp32 residual stream
        {"name": "norm_train_fwd", "op": "norm", "part": "fwd", "rows": 8192, "width": 4096, "bits": 32, "beta": True},
        # backward of an odd number of tokens, bf16
        {"name": "norm_train_bwd", "op": "norm", "part": "bwd", "rows": 8191, "width": 2048, "bits": 16, "beta": True},
        # first stage's F: 8 x 1024 tokens, some padding
        {"name": "embedding_train", "op": "embedding", "part": "lookup", "tokens": 8192, "vocab": 50000, "width": 4096,
         "bits": 16, "padded": 200},
        # its W, an odd number of tokens, fp32 stream, odd sizes: mostly writing the table's gradient
        {"name": "embedding_grad_odd", "op": "embedding", "part": "grad", "tokens": 2047, "vocab": 50021, "width": 1032,
         "bits": 32, "padded": 0},
        # a large microbatch on a smaller vocabulary: a few ids have hundreds of tokens
        {"name": "embedding_grad", "op": "embedding", "part": "grad", "tokens": 16384, "vocab": 32000, "width": 2048,
         "bits": 16, "padded": 500},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    most_bytes = max(work(c)["bytes"] for c in listed())
    most_flops = max(work(c)["flops"] for c in listed())
    while True:
        case = _drawn(rng)
        w = work(case)
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops:
            return case


def _drawn(rng):
    op = rng.choice(["linear", "linear", "norm", "embedding"])
    if op == "linear":
        form = rng.choice(["store", "gelu", "grad"])
        return {"op": op, "rows": _log(rng, 1, 8192), "n": 8 * _log(rng, 8, 1024), "k": 8 * _log(rng, 8, 1024),
                "form": form, "transposed": form == "grad" or rng.random() < 0.4,
                "bits": rng.choice([16, 32]) if form == "store" else 16, "bias": form != "grad" and rng.random() < 0.7,
                "residual": rng.random() < 0.8, "save": form == "gelu" and rng.random() < 0.5,
                "gap": rng.choice([0, 0, 8, 128])}
    if op == "norm":
        return {"op": op, "part": rng.choice(["fwd", "bwd"]), "rows": _log(rng, 1, 8192),
                "width": 8 * _log(rng, 8, 1024), "bits": rng.choice([16, 32]), "beta": rng.random() < 0.8}
    tokens = _log(rng, 1, 16384)
    return {"op": op, "part": rng.choice(["lookup", "grad"]), "tokens": tokens, "vocab": _log(rng, 100, 65536),
            "width": 8 * _log(rng, 16, 512), "bits": rng.choice([16, 32]), "padded": rng.choice([0, tokens // 16])}


# -------------------------------------------------------------------- inputs
def _stream(case):
    return BF16 if case["bits"] == 16 else F32


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op = case["op"]
    s = {"case": dict(case)}
    kind = _stream(case)

    def normal(*shape, std=1.0, dtype=BF16):
        return (torch.randn(shape, generator=gen, device="cuda", dtype=F32) * std).to(dtype)

    def empty(*shape, dtype=BF16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op == "linear":
        M, N, K, gap = case["rows"], case["n"], case["k"], case["gap"]
        # a slice of a wider buffer (one of several projections' results) where there is a gap
        s["X"] = normal(M, K + gap)[:, :K]
        s["W"] = normal(*((N, K) if case["transposed"] else (K, N)), std=0.02)
        s["bias"] = normal(N, std=0.1) if case["bias"] else None
        s["R"] = normal(M, N, dtype=kind) if case["residual"] else None
        s["H"] = normal(M, N) if case["form"] == "grad" else None
        s["out"] = empty(M, N, dtype=kind)
        s["kept"] = empty(M, N) if case["save"] else None
    elif op == "norm":
        M, w = case["rows"], case["width"]
        # a residual stream: channels of different spread and offset
        spread = torch.exp(0.5 * torch.randn(w, generator=gen, device="cuda"))
        offset = 0.5 * torch.randn(w, generator=gen, device="cuda")
        s["X"] = (normal(M, w, dtype=F32) * spread + offset).to(kind)
        s["gamma"] = (1.0 + normal(w, std=0.2, dtype=F32)).to(BF16)
        s["beta"] = normal(w, std=0.2) if case["beta"] else None
        s["mean"], s["rstd"] = empty(M, dtype=F32), empty(M, dtype=F32)
        if case["part"] == "fwd":
            s["Y"] = empty(M, w)
        else:
            x = s["X"].to(F64)
            mean = x.mean(dim=1)
            s["mean"] = mean.to(F32)
            s["rstd"] = torch.rsqrt((x - mean[:, None]).square().mean(dim=1) + EPS).to(F32)
            s["dY"] = normal(M, w)
            s["dR"] = normal(M, w, dtype=kind)
            s["dX"] = empty(M, w, dtype=kind)
            s["dX16"] = empty(M, w) if case["bits"] == 32 else None
            s["dgamma"], s["dbeta"] = empty(w, dtype=F32), empty(w, dtype=F32) if case["beta"] else None
    else:
        T, V, w = case["tokens"], case["vocab"], case["width"]
        # ids by falling frequency, as words have, scattered over the vocabulary
        u = torch.rand(T, generator=gen, device="cuda", dtype=F64)
        rank = torch.floor(torch.exp(u * math.log(V + 1.0))).long().clamp(1, V) - 1
        ids = torch.randperm(V, generator=gen, device="cuda")[rank].to(torch.int32)
        if case["padded"]:
            ids[torch.randperm(T, generator=gen, device="cuda")[:case["padded"]]] = -1
        s["ids"] = ids
        s["scale"] = math.sqrt(w)
        if case["part"] == "lookup":
            s["E"] = normal(V, w, std=0.02)
            s["Y"] = empty(T, w, dtype=kind)
        else:
            s["dY"] = normal(T, w, dtype=kind)
            s["dE"] = empty(V, w, dtype=F32)
            s["order"], s["sorted"] = empty(T, dtype=torch.int32), empty(T, dtype=torch.int32)
            # what zb_embedding_workspace_bytes asks for at most: 2 x 8 bytes a token, 2 rows for each 32 tokens
            s["work"] = empty(16 * T + 8 * w * (T // 32 + 2) + (1 << 20), dtype=torch.uint8)
    return s


# ------------------------------------------------------------- the library's
def _run_own(s):
    from split_backward_gemms_gb300 import zb
    c = s["case"]
    dtype = zb.ZB_DT_BF16 if c["bits"] == 16 else zb.ZB_DT_F32
    if c["op"] == "linear":
        form = {"store": zb.ZB_LINEAR_STORE, "gelu": zb.ZB_LINEAR_GELU, "grad": zb.ZB_LINEAR_GELU_GRAD}[c["form"]]
        g = zb.make_linear(c["rows"], c["n"], c["k"], transposed=c["transposed"], epilogue=form, dtype=dtype,
                           ldx=s["X"].stride(0))
        if c["form"] == "gelu":
            zb.zb_linear_product(g, s["X"], s["W"], s["bias"], s["R"], None, s["kept"], s["out"])
            return {"Y": s["out"], "H": s["kept"]} if c["save"] else s["out"]
        zb.zb_linear_product(g, s["X"], s["W"], s["bias"], s["R"], s["H"], s["out"], None)
        return s["out"]
    if c["op"] == "norm":
        n = zb.make_layernorm(c["rows"], c["width"], dtype=dtype, eps=EPS)
        if c["part"] == "fwd":
            zb.zb_layernorm_forward(n, s["X"], s["gamma"], s["beta"], s["Y"], s["mean"], s["rstd"])
            return {"Y": s["Y"], "mean": s["mean"], "rstd": s["rstd"]}
        zb.zb_layernorm_backward_input(n, s["dY"], s["X"], s["gamma"], s["mean"], s["rstd"], s["dR"], s["dX"],
                                       s["dX16"])
        zb.zb_layernorm_backward_weight(n, s["dY"], s["X"], s["mean"], s["rstd"], s["dgamma"], s["dbeta"], 0)
        out = {"dX": s["dX"], "dgamma": s["dgamma"]}
        if s["dX16"] is not None:
            out["dX16"] = s["dX16"]
        if s["dbeta"] is not None:
            out["dbeta"] = s["dbeta"]
        return out
    e = zb.make_embedding(c["tokens"], c["vocab"], c["width"], dtype=dtype, scale=s["scale"])
    if c["part"] == "lookup":
        zb.zb_embedding_forward(e, s["ids"], s["E"], s["Y"])
        return s["Y"]
    zb.zb_embedding_sort(e, s["ids"], s["order"], s["sorted"], s["work"], s["work"].numel())
    zb.zb_embedding_backward(e, s["order"], s["sorted"], s["dY"], s["dE"], 0, s["work"], s["work"].numel())
    return {"dE": s["dE"], "order": s["order"]}


# ---------------------------------------------------------- the plain forms
def _gelu(x):
    return x * (0.5 * (1.0 + torch.erf(x * INV_SQRT2)))


def _gelu_grad(x):
    return 0.5 * (1.0 + torch.erf(x * INV_SQRT2)) + x * torch.exp(-0.5 * x * x) * INV_SQRT_2PI


def _run_plain(s):
    c = s["case"]
    kind = _stream(c)
    if c["op"] == "linear":
        w = s["W"].float()
        d = s["X"].float() @ (w.t() if c["transposed"] else w)
        if s["bias"] is not None:
            d = d + s["bias"].float()
        y = _gelu(d) if c["form"] == "gelu" else d * _gelu_grad(s["H"].float()) if c["form"] == "grad" else d
        if s["R"] is not None:
            y = y + s["R"].float()
        return {"Y": y.to(kind), "H": d.to(BF16)} if c["save"] else y.to(kind)
    if c["op"] == "norm":
        x, g = s["X"].float(), s["gamma"].float()
        if c["part"] == "fwd":
            mean = x.mean(dim=1, keepdim=True)
            d = x - mean
            rstd = 1.0 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + EPS)
            y = d * rstd * g
            if s["beta"] is not None:
                y = y + s["beta"].float()
            return {"Y": y.to(BF16), "mean": mean[:, 0], "rstd": rstd[:, 0]}
        rstd, dy = s["rstd"][:, None], s["dY"].float()
        xh = (x - s["mean"][:, None]) * rstd
        u = dy * g
        dx = rstd * (u - u.mean(dim=1, keepdim=True) - xh * (u * xh).mean(dim=1, keepdim=True)) + s["dR"].float()
        out = {"dX": dx.to(kind), "dgamma": (dy * xh).sum(dim=0)}
        if c["bits"] == 32:
            out["dX16"] = dx.to(BF16)
        if s["dbeta"] is not None:
            out["dbeta"] = dy.sum(dim=0)
        return out
    ids, V = s["ids"].long(), c["vocab"]
    on = (ids >= 0) & (ids < V)
    if c["part"] == "lookup":
        y = s["E"][torch.where(on, ids, 0)].float() * s["scale"]
        return torch.where(on[:, None], y, torch.zeros_like(y)).to(kind)
    order = torch.where(on, ids, V).argsort(stable=True)
    # long sums: a frequent id has thousands of terms
    dE = torch.zeros((V + 1, c["width"]), dtype=F64, device="cuda")
    dE.index_add_(0, torch.where(on, ids, V), s["dY"].to(F64))
    return {"dE": (dE[:V] * s["scale"]).to(F32), "order": order.to(torch.int32)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------ work and exact
def work(case):
    op, es = case["op"], case["bits"] // 8
    if op == "linear":
        M, N, K = case["rows"], case["n"], case["k"]
        sides = case["residual"] * es + (case["form"] == "grad") * 2 + es + case["save"] * 2
        return {"bytes": 2 * K * (M + N) + sides * M * N, "flops": 2 * M * N * K}
    if op == "norm":
        M, w = case["rows"], case["width"]
        if case["part"] == "fwd":
            return {"bytes": M * w * (es + 2) + 8 * M + 4 * w, "flops": 8 * M * w}
        # x, dy, dR read once, dx (and its copy) written
        return {"bytes": M * w * (3 * es + 2 + (2 if es == 4 else 0)) + 8 * M + 10 * w, "flops": 15 * M * w}
    T, V, w = case["tokens"], case["vocab"], case["width"]
    live = T - case["padded"]
    if case["part"] == "lookup":
        # distinct rows of the table, at most
        return {"bytes": min(live, V) * w * 2 + T * w * es + 4 * T, "flops": live * w}
    return {"bytes": live * w * es + 4 * V * w + 8 * T, "flops": live * w}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        W = s["W"].to(F64)
        if case["transposed"]:
            W = W.T.contiguous()
        D = torch.empty((case["rows"], case["n"]), dtype=F64, device="cuda")
        for r in range(0, case["rows"], 1024):
            D[r:r + 1024] = torch.matmul(s["X"][r:r + 1024].to(F64), W)
        if s["bias"] is not None:
            D += s["bias"].to(F64)
        H = D.clone() if case["save"] else None
        if case["form"] == "gelu":
            D *= torch.special.ndtr(D)
        elif case["form"] == "grad":
            h = s["H"].to(F64)
            D *= torch.special.ndtr(h) + h * torch.exp(-h * h / 2) / math.sqrt(2 * math.pi)
        if s["R"] is not None:
            D += s["R"].to(F64)
        return {"Y": D, "H": H} if case["save"] else D
    if case["op"] == "norm":
        x, w = s["X"].to(F64), case["width"]
        if case["part"] == "fwd":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = (var + EPS) ** -0.5
            Y = torch.einsum("rc,r,c->rc", x - mean[:, None], rstd, s["gamma"].to(F64))
            if s["beta"] is not None:
                Y += s["beta"].to(F64)[None]
            return {"Y": Y, "mean": mean, "rstd": rstd}
        mean, rstd, dy = s["mean"].to(F64), s["rstd"].to(F64), s["dY"].to(F64)
        xh = torch.einsum("rc,r->rc", x - mean[:, None], rstd)
        u = dy * s["gamma"].to(F64)
        along = torch.einsum("rc,rc->r", u, xh) / w
        dX = torch.einsum("rc,r->rc", u - (u.sum(dim=1) / w)[:, None] - xh * along[:, None], rstd) + s["dR"].to(F64)
        out = {"dX": dX, "dgamma": torch.einsum("rc,rc->c", dy, xh)}
        if case["bits"] == 32:
            out["dX16"] = dX
        if case["beta"]:
            out["dbeta"] = torch.einsum("rc->c", dy)
        return out
    ids, V = s["ids"].cpu().numpy(), case["vocab"]
    if case["part"] == "lookup":
        Y = torch.zeros((case["tokens"], case["width"]), dtype=F64, device="cuda")
        at = np.nonzero((ids >= 0) & (ids < V))[0]
        Y[torch.from_numpy(at).cuda()] = s["E"][torch.from_numpy(ids[at].astype(np.int64)).cuda()].to(F64) * s["scale"]
        return Y
    # segments of the sorted tokens, one product with a 0/1 matrix for each stretch of ids
    dE = torch.zeros((V, case["width"]), dtype=F64, device="cuda")
    live = np.nonzero((ids >= 0) & (ids < V))[0]
    live = live[np.argsort(ids[live], kind="stable")]
    at, first = np.unique(ids[live], return_index=True)
    last = np.append(first[1:], len(live))
    for a in range(0, len(at), 512):
        b = min(a + 512, len(at))
        tokens = live[first[a]:last[b - 1]]
        which = np.repeat(np.arange(b - a), last[a:b] - first[a:b])
        pick = torch.zeros((b - a, len(tokens)), dtype=F64, device="cuda")
        pick[torch.from_numpy(which).cuda(), torch.arange(len(tokens), device="cuda")] = s["scale"]
        dE[torch.from_numpy(at[a:b].astype(np.int64)).cuda()] = pick @ s["dY"][torch.from_numpy(tokens).cuda()].to(F64)
    return {"dE": dE, "order": None}
