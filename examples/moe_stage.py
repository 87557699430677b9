"""One mixture-of-experts pipeline stage with its backward split, on one GPU.

A stage of E expert MLP blocks learns to imitate a fixed teacher stage.  Each
step runs m microbatches in the order of a zero-bubble schedule: every
microbatch's F and B first, the weight gradients W afterwards, from what F and B
left in memory.

  F  route -> dispatch -> experts' F -> combine
  B  combine's gradient -> experts' B -> dispatch's gradient (a plain combine),
     and the gates' gradient to the router's logits
  W  experts' weight gradients, accumulated over the microbatches in fp32, then
     one AdamW step

With --fp8 the products of F and B (the critical path) run in 8 bits with a
scale for each block of 128; W stays in bf16.

    python examples/moe_stage.py [--fp8] [--steps 20] [--tokens 2048] ...
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from split_backward_gemms_gb300 import zb  # noqa: E402

BF16 = torch.bfloat16
E4M3 = torch.float8_e4m3fn


class Stage:
    """Buffers of one stage for m microbatches of `tokens` tokens."""

    def __init__(self, tokens, h, f, experts, topk, m, fp8=False, device="cuda"):
        self.T, self.h, self.f, self.E, self.k, self.m, self.fp8 = tokens, h, f, experts, topk, m, fp8
        rows = tokens * topk
        self.rows = rows
        self.router = zb.make_router(tokens, experts, topk, renorm=True)
        self.moe = zb.make_moe(rows, h, f, experts)

        def new(*shape, dtype=BF16):
            return torch.empty(shape, dtype=dtype, device=device)

        i32 = torch.int32
        self.micro = [dict(gates=new(tokens, topk, dtype=torch.float32), expert=new(tokens, topk, dtype=i32),
                           offsets=new(experts + 1, dtype=i32), row_of=new(tokens, topk, dtype=i32),
                           token_of=new(rows, dtype=i32), X=new(rows, h), H=new(rows, f), A=new(rows, f),
                           Y=new(rows, h), dY=new(rows, h), dH=new(rows, f), dX=new(rows, h),
                           dgates=new(tokens, topk, dtype=torch.float32), out=new(tokens, h), din=new(tokens, h),
                           dlogits=new(tokens, experts, dtype=torch.float32)) for _ in range(m)]
        self.route_ws = new(zb.zb_moe_route_workspace_bytes(self.router), dtype=torch.uint8)
        self.w_ws = new(zb.zb_moe_workspace_bytes(self.moe), dtype=torch.uint8)
        self.dW1 = new(experts, h, f, dtype=torch.float32)
        self.dW2 = new(experts, f, h, dtype=torch.float32)
        if fp8:
            hb, fb = -(-h // 128), -(-f // 128)
            # each weight twice: for Y = X W (transposed) and for dX = dY W^T
            self.q = {name: (new(experts, r, c, dtype=E4M3), new(experts, rb, cb, dtype=torch.float32),
                             new(experts, c, r, dtype=E4M3), new(experts, cb, rb, dtype=torch.float32))
                      for name, r, c, rb, cb in (("W1", h, f, hb, fb), ("W2", f, h, fb, hb))}
            self.xq = {h: (new(rows, h, dtype=E4M3), new(rows, hb, dtype=torch.float32)),
                       f: (new(rows, f, dtype=E4M3), new(rows, fb, dtype=torch.float32))}

    def set_weights(self, W1, W2):
        """bf16 W1 [E, h, f] and W2 [E, f, h] (kept; quantised here with fp8)."""
        self.W1, self.W2 = W1, W2
        if self.fp8:
            for name, W in (("W1", W1), ("W2", W2)):
                zb.zb_fp8_quantize_weight(self.E, W.shape[1], W.shape[2], W, *self.q[name])

    def _product8(self, b, X, weight, transposed, out0, out1=None, H=None, epilogue=zb.ZB_FP8_STORE):
        q, s, qt, st = self.q[weight]
        w, ws = (qt, st) if transposed else (q, s)
        xq, xs = self.xq[X.shape[1]]
        zb.zb_fp8_quantize_rows(self.rows, X.shape[1], X, xq, xs)
        g = zb.make_fp8_matmul(self.rows, w.shape[1], w.shape[2], self.E, epilogue)
        zb.zb_fp8_matmul(g, b["offsets"], xq, xs, w, ws, H, out0, out1)

    def forward(self, j, X, logits):
        """F of microbatch j: [T, h] tokens and [T, E] router logits -> [T, h]."""
        b = self.micro[j]
        zb.zb_moe_route(self.router, logits, b["gates"], b["expert"], b["offsets"], b["row_of"], b["token_of"],
                        self.route_ws, self.route_ws.numel())
        zb.zb_moe_dispatch(self.T, self.k, self.h, X, b["row_of"], b["X"])
        if self.fp8:
            self._product8(b, b["X"], "W1", True, b["H"], b["A"], epilogue=zb.ZB_FP8_GELU)
            self._product8(b, b["A"], "W2", True, b["Y"])
        else:
            zb.zb_moe_forward(self.moe, b["offsets"], b["X"], self.W1, self.W2, None, None, b["H"], b["A"], b["Y"])
        zb.zb_moe_combine(self.T, self.k, self.h, b["Y"], b["row_of"], b["gates"], b["out"])
        return b["out"]

    def backward_input(self, j, dout):
        """B of microbatch j: the gradient to its tokens (and to its logits, in micro[j])."""
        b = self.micro[j]
        zb.zb_moe_combine_backward(self.T, self.k, self.h, dout, b["Y"], b["row_of"], b["gates"], b["dY"],
                                   b["dgates"])
        if self.fp8:
            self._product8(b, b["dY"], "W2", False, b["dH"], H=b["H"], epilogue=zb.ZB_FP8_GELU_GRAD)
            self._product8(b, b["dH"], "W1", False, b["dX"])
        else:
            zb.zb_moe_backward_input(self.moe, b["offsets"], b["dY"], self.W1, self.W2, b["H"], b["dH"], b["dX"])
        zb.zb_moe_combine(self.T, self.k, self.h, b["dX"], b["row_of"], None, b["din"])
        zb.zb_moe_route_backward(self.router, None, b["expert"], b["gates"], b["dgates"], b["dlogits"])
        return b["din"]

    def backward_weight(self, j):
        """W of microbatch j, deferrable: the first one overwrites the gradients."""
        b = self.micro[j]
        zb.zb_moe_backward_weight(self.moe, b["offsets"], b["X"], b["A"], b["dH"], b["dY"], self.dW1, self.dW2, None,
                                  None, j > 0, self.w_ws, self.w_ws.numel())


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--fp8", action="store_true")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--h", type=int, default=512)
    ap.add_argument("--f", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--topk", type=int, default=2)
    ap.add_argument("--micro", type=int, default=4)
    a = ap.parse_args()
    torch.manual_seed(0)

    def weights(scale):
        return [(torch.randn(a.experts, r, c, device="cuda") * scale / r ** 0.5) for r, c in ((a.h, a.f), (a.f, a.h))]

    teacher = Stage(a.tokens, a.h, a.f, a.experts, a.topk, a.micro)
    teacher.set_weights(*(w.to(BF16) for w in weights(1.0)))
    stage = Stage(a.tokens, a.h, a.f, a.experts, a.topk, a.micro, fp8=a.fp8)
    theta = weights(1.0)
    copies = [t.to(BF16) for t in theta]
    moments = [(torch.zeros_like(t), torch.zeros_like(t)) for t in theta]
    gate = torch.randn(a.h, a.experts, device="cuda") / a.h ** 0.5
    decisions = torch.empty(40, dtype=torch.uint8, device="cuda")
    scratch = torch.empty(zb.zb_grad_stats_scratch_bytes(), dtype=torch.uint8, device="cuda")
    state = torch.empty(2, dtype=torch.float64, device="cuda")
    X = [torch.randn(a.tokens, a.h, device="cuda", dtype=BF16) for _ in range(a.micro)]
    logits = [x.float() @ gate for x in X]
    want = [teacher.forward(j, X[j], logits[j]).float() for j in range(a.micro)]
    losses = []
    for step in range(1, a.steps + 1):
        stage.set_weights(*copies)
        loss = 0.0
        for j in range(a.micro):
            err = stage.forward(j, X[j], logits[j]).float() - want[j]
            loss = loss + err.square().mean() / a.micro
            stage.backward_input(j, (2.0 * err / (a.tokens * a.micro)).to(BF16))
        for j in range(a.micro):  # the deferred half of the backward
            stage.backward_weight(j)
        grads = [stage.dW1, stage.dW2]
        zb.zb_grad_stats(grads, [g.numel() for g in grads], state, scratch, scratch.numel())
        tensors = [dict(theta=t, m=m, v=v, grad=g, weight_bf16=c, stage=0)
                   for t, (m, v), g, c in zip(theta, moments, grads, copies)]
        zb.zb_post_validated_adamw(1, [state], tensors, zb.make_adamw(lr=2e-3, weight_decay=0.0, max_norm=1.0, step=step),
                                   decisions)
        losses.append(float(loss))
        if step == 1 or step % 5 == 0:
            print(f"step {step:3d}  loss {losses[-1]:.5f}")
    zb.zb_sync_status()
    return losses


if __name__ == "__main__":
    main()
