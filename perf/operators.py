"""Timed cases of the mixture-of-experts and 8-bit operators.

A case is a dict of plain values; ``prepare`` makes what a user's program has
in hand before the call, ``run`` makes one pass through one operator and
returns its outputs, ``work`` gives the bytes and operations the pass cannot
do without, ``exact`` the same outputs from the definition in 64 bits.  With
``own`` false ``run`` computes the operator in its plain form (elementary
torch operations in 32 bits, rounded once at the end); with ``own`` true it
calls the library.

Operators (``op`` of a case)
  route          top-k gates of the router's logits, and the order of rows by
                 expert (offsets, row of a choice, token of a row)
  route_bwd      gradient of the gates to the logits
  dispatch       tokens copied to their rows, grouped by expert
  combine        tokens' weighted sums over their rows
  combine_bwd    gradients of combine to the rows and to the gates
  experts_fwd    F of the experts' blocks: H = X W1[e], A = GeLU(H), Y = A W2[e]
  experts_bwd    B: dH = (dY W2[e]^T) GeLU'(H), dX = dH W1[e]^T
  experts_wgrad  W: dW1[e] = X_e^T dH_e, dW2[e] = A_e^T dY_e (fp32)
  fp8_fwd        X quantised to e4m3 (a scale for each 1 x 128), then
                 Y = X W[e] with W held in e4m3 (a scale for each 128 x 128)
  fp8_bwd        dY quantised the same way, then dH = (dY W[e]^T) GeLU'(H)
"""

import math
import random

import numpy as np
import torch

own = False

INV_SQRT2 = 1.0 / math.sqrt(2.0)
INV_SQRT_2PI = 1.0 / math.sqrt(2.0 * math.pi)
E4M3_MAX = 448.0


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of a few sequences: pure latency
        {"name": "route_decode", "op": "route", "tokens": 16, "experts": 64, "topk": 6, "bits": 32, "renorm": True,
         "padded": 0},
        # a training microbatch of 16 x 1024 tokens, fine-grained experts, some padding tokens
        {"name": "route_train", "op": "route", "tokens": 16384, "experts": 128, "topk": 8, "bits": 32,
         "renorm": False, "padded": 500},
        # its gradient, bf16 logits, an odd number of tokens and of experts
        {"name": "route_grad", "op": "route_bwd", "tokens": 8191, "experts": 60, "topk": 4, "bits": 16,
         "renorm": True, "padded": 100},
        # a microbatch's tokens sent to two experts each
        {"name": "dispatch_train", "op": "dispatch", "tokens": 8192, "experts": 16, "topk": 2, "width": 4096,
         "padded": 0},
        # ... gathered back: eight rows a token
        {"name": "combine_fine", "op": "combine", "tokens": 4099, "experts": 64, "topk": 8, "width": 2048,
         "padded": 64},
        # ... and the gradient of that
        {"name": "combine_grad", "op": "combine_bwd", "tokens": 8192, "experts": 16, "topk": 2, "width": 4096,
         "padded": 0},
        # a decoding step of eight sequences: bound by reading the chosen experts' weights
        {"name": "experts_decode", "op": "experts_fwd", "rows": 16, "experts": 8, "h": 1024, "f": 4096},
        # F of a training microbatch, 8 wide experts: bound by the matrix products
        {"name": "experts_train", "op": "experts_fwd", "rows": 16384, "experts": 8, "h": 2048, "f": 8192},
        # B with many narrow experts, a few hundred rows each, ragged
        {"name": "experts_fine_bwd", "op": "experts_bwd", "rows": 24570, "experts": 64, "h": 2048, "f": 1536},
        # W of a microbatch of the h = 1024 block: about half of it is writing the fp32 gradients
        {"name": "experts_wgrad", "op": "experts_wgrad", "rows": 16384, "experts": 16, "h": 1024, "f": 4096},
        # the first linear of the h = 4096 block in 8 bits
        {"name": "fp8_dense", "op": "fp8_fwd", "rows": 4096, "experts": 1, "k": 4096, "n": 16384},
        # the critical-path gradient of grouped experts in 8 bits, odd sizes
        {"name": "fp8_grouped_bwd", "op": "fp8_bwd", "rows": 8190, "experts": 16, "k": 1040, "n": 4104},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        case = _drawn(rng)
        if work(case)["bytes"] <= most:
            return case


def _drawn(rng):
    op = rng.choice(["route", "route_bwd", "dispatch", "combine", "combine_bwd", "experts_fwd", "experts_bwd",
                     "experts_wgrad", "fp8_fwd", "fp8_bwd"])
    if op in ("route", "route_bwd"):
        experts = _log(rng, 4, 256)
        tokens = _log(rng, 1, 16384)
        return {"op": op, "tokens": tokens, "experts": experts, "topk": rng.randint(1, min(8, experts)),
                "bits": rng.choice([16, 32]), "renorm": rng.random() < 0.5,
                "padded": rng.choice([0, tokens // 16])}
    if op in ("dispatch", "combine", "combine_bwd"):
        tokens = _log(rng, 1, 8192)
        experts = _log(rng, 4, 128)
        return {"op": op, "tokens": tokens, "experts": experts, "topk": rng.randint(1, min(8, experts)),
                "width": 8 * _log(rng, 16, 512), "padded": rng.choice([0, tokens // 16])}
    rows = _log(rng, 1, 16384)
    experts = _log(rng, 1, 64)
    a = 8 * _log(rng, 16, 256)
    b = 8 * _log(rng, 16, 512)
    if op in ("fp8_fwd", "fp8_bwd"):
        return {"op": op, "rows": rows, "experts": experts, "k": 16 * max(8, a // 16), "n": b}
    return {"op": op, "rows": rows, "experts": experts, "h": a, "f": b}


# -------------------------------------------------------------------- inputs
def _split_rows(rows, experts, seed):
    """Rows of each expert: a multinomial draw over uneven popularities."""
    rng = np.random.default_rng(seed)
    p = np.exp(rng.normal(0.0, 0.5, experts))
    return rng.multinomial(rows, p / p.sum())


def _normal(gen, shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(torch.bfloat16)


def _choices(case, gen):
    """Distinct experts of each token with gates, and the rows' order by expert."""
    T, E, k = case["tokens"], case["experts"], case["topk"]
    z = torch.randn((T, E), generator=gen, device="cuda") + torch.randn((1, E), generator=gen, device="cuda") * 0.5
    pick = z.argsort(dim=1, descending=True)[:, :k]
    gates = torch.softmax(z, dim=1).gather(1, pick).contiguous()
    live = torch.ones(T, dtype=torch.bool, device="cuda")
    if case["padded"]:
        live[torch.randperm(T, generator=gen, device="cuda")[:case["padded"]]] = False
    key = torch.where(live[:, None], pick, E).reshape(-1)
    order = key.argsort(stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(T * k, device="cuda")
    row = torch.where(key < E, row, -1).reshape(T, k).to(torch.int32)
    return row.contiguous(), (gates * live[:, None]).contiguous()


def _quantised_weight(w):
    """w [E, K, N] (K and N in blocks of 128) as e4m3 with a power-of-two scale for each block."""
    E, K, N = w.shape
    kb, nb = -(-K // 128), -(-N // 128)
    pad = torch.zeros((E, kb * 128, nb * 128), device="cuda")
    pad[:, :K, :N] = w.float()
    blocks = pad.view(E, kb, 128, nb, 128)
    scale = _scale_of(blocks.abs().amax(dim=(2, 4)))
    q = (blocks / scale[:, :, None, :, None]).view(E, kb * 128, nb * 128)[:, :K, :N]
    return q.to(torch.float8_e4m3fn), scale


def _scale_of(amax):
    """The least power of two s with amax / s <= 448; 1 for a block of zeros."""
    mant, exp = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), exp - 9 + (mant > 0.875).to(exp.dtype))
    return torch.where(amax > 0, s, torch.ones_like(s))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op = case["op"]
    s = {"case": dict(case)}
    i32 = dict(dtype=torch.int32, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    if op in ("route", "route_bwd"):
        T, E, k = case["tokens"], case["experts"], case["topk"]
        z = torch.randn((T, E), generator=gen, device="cuda") + torch.randn((1, E), generator=gen, device="cuda") * 0.5
        if case["padded"]:
            # a padding token has no expert to go to: its whole row is masked
            z[torch.randperm(T, generator=gen, device="cuda")[:case["padded"]]] = -math.inf
        s["logits"] = z.to(torch.bfloat16 if case["bits"] == 16 else torch.float32)
        s["gates"] = torch.empty((T, k), device="cuda")
        s["expert"] = torch.empty((T, k), **i32)
        s["offsets"] = torch.empty(E + 1, **i32)
        s["row_of"] = torch.empty((T, k), **i32)
        s["token_of"] = torch.empty(T * k, **i32)
        s["work"] = torch.empty(4 << 20, dtype=torch.uint8, device="cuda")
        if op == "route_bwd":
            zf = s["logits"].float()
            val, pick = zf.sort(dim=1, descending=True, stable=True)
            val, pick = val[:, :k], pick[:, :k]
            p = torch.softmax(zf, dim=1).gather(1, pick)
            if case["renorm"]:
                p = p / p.sum(dim=1, keepdim=True)
            on = val > -math.inf
            s["gates"] = torch.where(on, p, torch.zeros_like(p)).contiguous()
            s["expert"] = torch.where(on, pick, -1).to(torch.int32).contiguous()
            s["dgates"] = torch.randn((T, k), generator=gen, device="cuda")
            s["dlogits"] = torch.empty_like(s["logits"])
    elif op in ("dispatch", "combine", "combine_bwd"):
        T, k, w = case["tokens"], case["topk"], case["width"]
        s["row_of"], s["gates"] = _choices(case, gen)
        live = T * k - case["padded"] * k
        s["live"] = live
        if op == "dispatch":
            s["X"] = _normal(gen, (T, w))
            s["Xp"] = torch.zeros((T * k, w), **bf)
        else:
            s["Yp"] = _normal(gen, (T * k, w))
            s["Y"] = torch.empty((T, w), **bf)
        if op == "combine_bwd":
            s["dY"] = _normal(gen, (T, w))
            s["dYp"] = torch.zeros((T * k, w), **bf)
            s["dgates"] = torch.empty((T, k), device="cuda")
    else:
        R, E = case["rows"], case["experts"]
        counts = _split_rows(R, E, seed)
        s["most"] = int(counts.max())
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
        if op in ("fp8_fwd", "fp8_bwd"):
            K, N = case["k"], case["n"]
            s["X"] = _normal(gen, (R, K))
            q, scale = _quantised_weight(_normal(gen, (E, K, N), 0.02).float())
            s["Wt"] = q.transpose(1, 2).contiguous()  # [E, N, K]
            s["scale"] = scale.transpose(1, 2).contiguous()  # [E, N/128, K/128]
            s["Xq"] = torch.empty((R, K), dtype=torch.float8_e4m3fn, device="cuda")
            s["Xs"] = torch.empty((R, -(-K // 128)), device="cuda")
            s["out"] = torch.empty((R, N), **bf)
            if op == "fp8_bwd":
                s["H"] = _normal(gen, (R, N))
        else:
            h, f = case["h"], case["f"]
            if op != "experts_wgrad":
                s["W1"], s["W2"] = _normal(gen, (E, h, f), 0.02), _normal(gen, (E, f, h), 0.02)
            if op == "experts_fwd":
                s["X"] = _normal(gen, (R, h))
                s["H"], s["A"], s["Y"] = (torch.empty((R, n), **bf) for n in (f, f, h))
            elif op == "experts_bwd":
                s["dY"], s["H"] = _normal(gen, (R, h)), _normal(gen, (R, f))
                s["dH"], s["dX"] = torch.empty((R, f), **bf), torch.empty((R, h), **bf)
            else:
                s["X"], s["A"] = _normal(gen, (R, h)), _normal(gen, (R, f), 0.5)
                s["dH"], s["dY"] = _normal(gen, (R, f)), _normal(gen, (R, h))
                s["dW1"] = torch.empty((E, h, f), device="cuda")
                s["dW2"] = torch.empty((E, f, h), device="cuda")
                s["work"] = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------- the library's
def _run_own(s):
    from split_backward_gemms_gb300 import zb
    c = s["case"]
    op = c["op"]
    if op in ("route", "route_bwd"):
        r = zb.make_router(c["tokens"], c["experts"], c["topk"],
                           dtype=zb.ZB_DT_BF16 if c["bits"] == 16 else zb.ZB_DT_F32, renorm=c["renorm"])
        if op == "route_bwd":
            zb.zb_moe_route_backward(r, s["logits"], s["expert"], s["gates"], s["dgates"], s["dlogits"])
            return s["dlogits"]
        zb.zb_moe_route(r, s["logits"], s["gates"], s["expert"], s["offsets"], s["row_of"], s["token_of"],
                        s["work"], s["work"].numel())
        return {n: s[n] for n in ("gates", "expert", "offsets", "row_of", "token_of")}
    if op == "dispatch":
        zb.zb_moe_dispatch(c["tokens"], c["topk"], c["width"], s["X"], s["row_of"], s["Xp"])
        return s["Xp"][:s["live"]]
    if op == "combine":
        zb.zb_moe_combine(c["tokens"], c["topk"], c["width"], s["Yp"], s["row_of"], s["gates"], s["Y"])
        return s["Y"]
    if op == "combine_bwd":
        zb.zb_moe_combine_backward(c["tokens"], c["topk"], c["width"], s["dY"], s["Yp"], s["row_of"], s["gates"],
                                   s["dYp"], s["dgates"])
        return {"dYp": s["dYp"][:s["live"]], "dgates": s["dgates"]}
    if op in ("fp8_fwd", "fp8_bwd"):
        zb.zb_fp8_quantize_rows(c["rows"], c["k"], s["X"], s["Xq"], s["Xs"])
        bwd = op == "fp8_bwd"
        g = zb.make_fp8_matmul(c["rows"], c["n"], c["k"], experts=c["experts"],
                               epilogue=zb.ZB_FP8_GELU_GRAD if bwd else zb.ZB_FP8_STORE)
        zb.zb_fp8_matmul(g, s["offsets"], s["Xq"], s["Xs"], s["Wt"], s["scale"], s["H"] if bwd else None, s["out"],
                         None)
        return s["out"]
    m = zb.make_moe(c["rows"], c["h"], c["f"], c["experts"])
    if op == "experts_fwd":
        zb.zb_moe_forward(m, s["offsets"], s["X"], s["W1"], s["W2"], None, None, s["H"], s["A"], s["Y"])
        return {"H": s["H"], "A": s["A"], "Y": s["Y"]}
    if op == "experts_bwd":
        zb.zb_moe_backward_input(m, s["offsets"], s["dY"], s["W1"], s["W2"], s["H"], s["dH"], s["dX"])
        return {"dH": s["dH"], "dX": s["dX"]}
    zb.zb_moe_backward_weight(m, s["offsets"], s["X"], s["A"], s["dH"], s["dY"], s["dW1"], s["dW2"], None, None, 0,
                              s["work"], s["work"].numel())
    return {"dW1": s["dW1"], "dW2": s["dW2"]}


# ---------------------------------------------------------- the plain forms
def _places(s):
    """Row index of each expert's places (clamped) with their mask; expert and place of each row."""
    off = s["offsets"].long()
    R = s["case"]["rows"]
    at = off[:-1, None] + torch.arange(s["most"], device="cuda")
    mask = at < off[1:, None]
    row = torch.arange(R, device="cuda")
    expert = torch.searchsorted(off, row, right=True) - 1
    return at.clamp(max=R - 1), mask, expert, row - off[expert]


def _gelu(x):
    return x * (0.5 * (1.0 + torch.erf(x * INV_SQRT2)))


def _gelu_grad(x):
    return 0.5 * (1.0 + torch.erf(x * INV_SQRT2)) + x * torch.exp(-0.5 * x * x) * INV_SQRT_2PI


def _quantised_rows(x):
    """x [R, K] rounded to e4m3 with a power-of-two scale for each 1 x 128, as the values it stands for."""
    R, K = x.shape
    kb = -(-K // 128)
    pad = torch.zeros((R, kb * 128), device="cuda")
    pad[:, :K] = x
    blocks = pad.view(R, kb, 128)
    scale = _scale_of(blocks.abs().amax(dim=2, keepdim=True))
    q = (blocks / scale).to(torch.float8_e4m3fn).float() * scale
    return q.view(R, kb * 128)[:, :K]


def _weight_values(s):
    """The e4m3 weight [E, N, K] as the fp32 values it stands for."""
    _, N, K = s["Wt"].shape
    big = s["scale"].repeat_interleave(128, dim=1)[:, :N].repeat_interleave(128, dim=2)[:, :, :K]
    return s["Wt"].float() * big


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    bf = torch.bfloat16
    if op == "route":
        T, E, k = c["tokens"], c["experts"], c["topk"]
        z = s["logits"].float()
        val, pick = z.sort(dim=1, descending=True, stable=True)
        val, pick = val[:, :k], pick[:, :k]
        on = val > -math.inf
        top = torch.where(on[:, :1], val[:, :1], torch.zeros_like(val[:, :1]))
        e = torch.exp(val - top)
        total = e.sum(dim=1, keepdim=True) if c["renorm"] else torch.exp(z - top).sum(dim=1, keepdim=True)
        gates = torch.where(on, e / total, torch.zeros_like(e))
        expert = torch.where(on, pick, -1)
        key = torch.where(on, pick, E).reshape(-1)
        srt, order = key.sort(stable=True)
        row = torch.empty_like(order)
        row[order] = torch.arange(T * k, device="cuda")
        offsets = torch.searchsorted(srt, torch.arange(E + 1, device="cuda"))
        return {"gates": gates, "expert": expert.to(torch.int32), "offsets": offsets.to(torch.int32),
                "row_of": torch.where(key < E, row, -1).reshape(T, k).to(torch.int32),
                "token_of": torch.where(srt < E, order // k, -1).to(torch.int32)}
    if op == "route_bwd":
        z, g, dg = s["logits"].float(), s["gates"], s["dgates"]
        on = s["expert"] >= 0
        col = s["expert"].clamp(min=0).long()
        inner = torch.where(on, g * dg, torch.zeros_like(g)).sum(dim=1, keepdim=True)
        if c["renorm"]:
            d = torch.where(on, g * (dg - inner), torch.zeros_like(g))
            dz = torch.zeros_like(z).scatter_add(1, col, d)
        else:
            top = z.amax(dim=1, keepdim=True)
            e = torch.exp(z - torch.where(top > -math.inf, top, torch.zeros_like(top)))
            p = e / e.sum(dim=1, keepdim=True).clamp(min=1e-30)
            dz = torch.zeros_like(z).scatter_add(1, col, torch.where(on, g * dg, torch.zeros_like(g))) - p * inner
        return dz.to(s["logits"].dtype)
    if op in ("dispatch", "combine", "combine_bwd"):
        T, k, w = c["tokens"], c["topk"], c["width"]
        on = s["row_of"] >= 0
        at = s["row_of"].clamp(min=0).long()
        # rows without a token land in a row past the end
        to = torch.where(on, at, T * k).reshape(-1)
        if op == "dispatch":
            out = torch.zeros((T * k + 1, w), dtype=bf, device="cuda")
            out[to] = s["X"][:, None, :].expand(T, k, w).reshape(T * k, w)
            return out[:s["live"]]
        g = torch.where(on, s["gates"], torch.zeros_like(s["gates"]))
        y = s["Yp"][at].float()
        if op == "combine":
            return (y * g[:, :, None]).sum(dim=1).to(bf)
        dy = s["dY"].float()
        out = torch.zeros((T * k + 1, w), dtype=bf, device="cuda")
        out[to] = (dy[:, None, :] * g[:, :, None]).reshape(T * k, w).to(bf)
        return {"dYp": out[:s["live"]], "dgates": torch.where(on, (y * dy[:, None, :]).sum(dim=2), torch.zeros_like(g))}
    at, mask, expert, place = _places(s)

    def grouped(x, w):  # x [R, K] fp32, w [E, K, N] fp32
        return torch.bmm(x[at], w)[expert, place]

    if op == "fp8_fwd":
        return grouped(_quantised_rows(s["X"].float()), _weight_values(s).transpose(1, 2)).to(bf)
    if op == "fp8_bwd":
        da = grouped(_quantised_rows(s["X"].float()), _weight_values(s).transpose(1, 2))
        return (da * _gelu_grad(s["H"].float())).to(bf)
    if op == "experts_fwd":
        H = grouped(s["X"].float(), s["W1"].float())
        A = _gelu(H)
        return {"H": H.to(bf), "A": A.to(bf), "Y": grouped(A, s["W2"].float()).to(bf)}
    if op == "experts_bwd":
        dH = grouped(s["dY"].float(), s["W2"].float().transpose(1, 2)) * _gelu_grad(s["H"].float())
        return {"dH": dH.to(bf), "dX": grouped(dH, s["W1"].float().transpose(1, 2)).to(bf)}

    def spread(x):
        return x.float()[at] * mask[:, :, None]

    return {"dW1": torch.bmm(spread(s["X"]).transpose(1, 2), spread(s["dH"])),
            "dW2": torch.bmm(spread(s["A"]).transpose(1, 2), spread(s["dY"]))}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------ work and exact
def work(case):
    op = case["op"]
    if op in ("route", "route_bwd"):
        T, E, k = case["tokens"], case["experts"], case["topk"]
        zb_ = T * E * case["bits"] // 8
        if op == "route":
            return {"bytes": zb_ + T * k * 16 + 4 * (E + 1), "flops": 4 * T * E}
        # softmax over the chosen experts alone does not need the logits
        return {"bytes": (zb_ if case["renorm"] else 2 * zb_) + T * k * 12, "flops": 4 * T * E}
    if op in ("dispatch", "combine", "combine_bwd"):
        T, k, w = case["tokens"], case["topk"], case["width"]
        live = T - case["padded"]
        if op == "dispatch":
            return {"bytes": 2 * w * live * (1 + k) + 4 * T * k, "flops": 0}
        if op == "combine":
            return {"bytes": 2 * w * (T + live * k) + 8 * T * k, "flops": 2 * live * k * w}
        return {"bytes": 2 * w * live * (1 + 2 * k) + 12 * T * k, "flops": 3 * live * k * w}
    R, E = case["rows"], case["experts"]
    # experts that get rows, at most
    used = min(R, E)
    if op in ("fp8_fwd", "fp8_bwd"):
        K, N = case["k"], case["n"]
        return {"bytes": 2 * R * K + used * K * N + 2 * R * N * (2 if op == "fp8_bwd" else 1), "flops": 2 * R * K * N}
    h, f = case["h"], case["f"]
    if op == "experts_wgrad":
        return {"bytes": 4 * R * (h + f) + 8 * E * h * f, "flops": 4 * R * h * f}
    rows = R * (2 * h + 2 * f)
    return {"bytes": 2 * (rows + 2 * used * h * f), "flops": 4 * R * h * f}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["topk"]
        z = s["logits"].to("cpu", f64).numpy()
        pick = np.argsort(-z, axis=1, kind="stable")[:, :k]
        val = np.take_along_axis(z, pick, 1)
        gates = np.zeros((T, k))
        for t in range(T):
            if val[t, 0] > -np.inf:
                e = np.exp(val[t] - val[t, 0])
                gates[t] = e / (e.sum() if case["renorm"] else np.exp(z[t] - val[t, 0]).sum())
        return {"gates": gates, "expert": None, "offsets": None, "row_of": None, "token_of": None}
    if op == "route_bwd":
        z = s["logits"].to(f64)
        ex, dg = s["expert"], s["dgates"].to(f64)
        T, E = z.shape
        chosen = torch.zeros((T, E), dtype=f64, device="cuda")
        grad = torch.zeros((T, E), dtype=f64, device="cuda")
        for j in range(case["topk"]):
            t = torch.nonzero(ex[:, j] >= 0)[:, 0]
            chosen[t, ex[t, j].long()] = 1.0
            grad[t, ex[t, j].long()] = dg[t, j]
        over = torch.where(chosen > 0, z, torch.full_like(z, -math.inf)) if case["renorm"] else z
        p = torch.nan_to_num(torch.softmax(over, dim=1), nan=0.0)
        return p * (grad * chosen - (p * grad * chosen).sum(dim=1, keepdim=True))
    if op in ("dispatch", "combine", "combine_bwd"):
        T, k = case["tokens"], case["topk"]
        if op == "dispatch":
            return None
        row, g = s["row_of"].long(), s["gates"].to(f64)
        Y = torch.zeros(s["Y"].shape, dtype=f64, device="cuda")
        dYp = torch.zeros(s["Yp"].shape, dtype=f64, device="cuda")
        dg = torch.zeros((T, k), dtype=f64, device="cuda")
        for j in range(k):
            t = torch.nonzero(row[:, j] >= 0)[:, 0]
            y = s["Yp"][row[t, j]].to(f64)
            Y[t] += g[t, j, None] * y
            if op == "combine_bwd":
                d = s["dY"][t].to(f64)
                dYp[row[t, j]] = g[t, j, None] * d
                dg[t, j] = (y * d).sum(dim=1)
        return Y if op == "combine" else {"dYp": dYp[:s["live"]], "dgates": dg}
    off = s["offsets"].tolist()
    spans = [(e, off[e], off[e + 1]) for e in range(case["experts"])]

    def phi(x):
        return 0.5 * torch.erfc(-x / math.sqrt(2.0))

    def dgelu(x):
        return phi(x) + x * torch.exp(-x * x / 2) / math.sqrt(2.0 * math.pi)

    if op in ("fp8_fwd", "fp8_bwd"):
        R, K, N = case["rows"], case["k"], case["n"]
        out = torch.empty((R, N), dtype=f64, device="cuda")
        X = s["X"].to(f64)
        for k0 in range(0, K, 128):
            a = X[:, k0:k0 + 128].abs().amax(dim=1, keepdim=True)
            sc = torch.where(a > 0, torch.exp2(torch.ceil(torch.log2(a / E4M3_MAX))), torch.ones_like(a))
            X[:, k0:k0 + 128] = (X[:, k0:k0 + 128] / sc).to(torch.float8_e4m3fn).to(f64) * sc
        for e, a, b in spans:
            if b > a:
                w = s["Wt"][e].to(f64)
                for n0 in range(0, N, 128):
                    for k0 in range(0, K, 128):
                        w[n0:n0 + 128, k0:k0 + 128] *= s["scale"][e, n0 // 128, k0 // 128].to(f64)
                out[a:b] = X[a:b] @ w.T
        return out if op == "fp8_fwd" else out * dgelu(s["H"].to(f64))
    h, f = case["h"], case["f"]
    if op == "experts_wgrad":
        dW1, dW2 = torch.zeros_like(s["dW1"], dtype=f64), torch.zeros_like(s["dW2"], dtype=f64)
        for e, a, b in spans:
            dW1[e] = s["X"][a:b].to(f64).T @ s["dH"][a:b].to(f64)
            dW2[e] = s["A"][a:b].to(f64).T @ s["dY"][a:b].to(f64)
        return {"dW1": dW1, "dW2": dW2}
    u = torch.empty((case["rows"], f), dtype=f64, device="cuda")
    v = torch.empty((case["rows"], h), dtype=f64, device="cuda")
    act = torch.empty_like(u)
    for e, a, b in spans:
        if b == a:
            continue
        if op == "experts_fwd":
            u[a:b] = s["X"][a:b].to(f64) @ s["W1"][e].to(f64)
            act[a:b] = u[a:b] * phi(u[a:b])
            v[a:b] = act[a:b] @ s["W2"][e].to(f64)
        else:
            u[a:b] = (s["dY"][a:b].to(f64) @ s["W2"][e].to(f64).T) * dgelu(s["H"][a:b].to(f64))
            v[a:b] = u[a:b] @ s["W1"][e].to(f64).T
    return {"H": u, "A": act, "Y": v} if op == "experts_fwd" else {"dH": u, "dX": v}
