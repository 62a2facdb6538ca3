"""A mixture-of-experts feed-forward layer on the framework's ragged operators.

    router logits -> moe_route -> moe_dispatch -> grouped_matmul (up, gate)
      -> silu(gate) * up -> grouped_matmul (down) -> moe_combine

No token is dropped and no expert is padded: the row counts stay on the device
from the router to the last product.  `forward` and `backward` are a training
step; `quantize` and `serve` are the same layer with 4-bit experts.

    python examples/moe_layer.py            # needs a GPU and the built library
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bmm_reducescatter_alltoall_gb300 as bra  # noqa: E402


def init(E, H, F, dtype=torch.bfloat16, seed=0):
    """Weights of E experts of width H -> F -> H: gate and up side by side."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")           # noqa: E731
    return {"router": rnd(H, E) * H ** -0.5,
            "up": (rnd(E, H, 2 * F) * H ** -0.5).to(dtype),
            "down": (rnd(E, F, H) * F ** -0.5).to(dtype)}


def forward(w, x, k):
    """y (T, H) of token rows x (T, H), and what backward needs."""
    logits = x.float() @ w["router"]
    r = bra.moe_route(logits, k)
    xs = bra.moe_dispatch(x, r["tokens"])
    gu = bra.grouped_matmul(xs, w["up"], r["counts"])
    gate, up = gu.chunk(2, dim=1)
    h = torch.nn.functional.silu(gate) * up
    ys = bra.grouped_matmul(h, w["down"], r["counts"])
    y = bra.moe_combine(ys, r["slots"], r["weights"])
    return y, (x, logits, r, xs, gu, h, ys)


def backward(w, saved, dy):
    """Gradients of x and of every weight for the gradient dy of y."""
    x, logits, r, xs, gu, h, ys = saved
    c = bra.moe_combine_grad(dy, ys, r["slots"], r["weights"], r["tokens"])
    down = bra.grouped_matmul_grad(c["dys"], h, w["down"], r["counts"], want=("dx", "dweight"))
    gate, up = (t.float() for t in gu.chunk(2, dim=1))
    s = torch.sigmoid(gate)
    dh = down["dx"].float()
    dgu = torch.cat([dh * up * s * (1 + gate * (1 - s)), dh * gate * s], 1).to(gu.dtype)
    up_g = bra.grouped_matmul_grad(dgu, xs, w["up"], r["counts"], want=("dx", "dweight"))
    dlogits = bra.moe_route_grad(c["dweights"], logits, r["ids"], r["weights"])
    dx = bra.moe_dispatch_grad(up_g["dx"], r["slots"]).float() + dlogits @ w["router"].t()
    return {"x": dx.to(x.dtype), "router": x.float().t() @ dlogits, "up": up_g["dweight"],
            "down": down["dweight"]}


def quantize(w):
    """The layer with its experts in 4 bits (their rows along the contraction)."""
    q = lambda t: bra.mxfp4_quantize(t.transpose(1, 2).contiguous())       # noqa: E731
    return {"router": w["router"], "up": q(w["up"]), "down": q(w["down"])}


def serve(w4, x, k):
    """forward with 4-bit experts: rows are quantized before each product."""
    r = bra.moe_route(x.float() @ w4["router"], k)
    product = lambda t, weight: bra.mxfp4_grouped_matmul(                  # noqa: E731
        bra.mxfp4_quantize(t, r["counts"]), weight, r["counts"], dtype=x.dtype)
    gate, up = product(bra.moe_dispatch(x, r["tokens"]), w4["up"]).chunk(2, dim=1)
    ys = product(torch.nn.functional.silu(gate) * up, w4["down"])
    return bra.moe_combine(ys, r["slots"], r["weights"])


def main():
    E, H, F, k, T = 16, 2048, 1024, 4, 4096
    w = init(E, H, F)
    w4 = quantize(w)
    x = torch.randn((T, H), device="cuda").bfloat16()
    dy = torch.randn((T, H), device="cuda").bfloat16()

    def timed(f, n=20):
        for _ in range(3):
            f()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        for _ in range(n):
            f()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) / n

    y, saved = forward(w, x, k)
    print(f"{E} experts, {T} tokens x {k}, width {H} -> {F}")
    print(f"forward            {timed(lambda: forward(w, x, k)):.3f} ms")
    print(f"forward + backward {timed(lambda: backward(w, forward(w, x, k)[1], dy)):.3f} ms")
    print(f"4-bit forward      {timed(lambda: serve(w4, x, k)):.3f} ms")
    y4 = serve(w4, x, k)
    print(f"4-bit output against bf16: {float((y4 - y).float().norm() / y.float().norm()):.3f} "
          "relative")
    print(f"4-bit forward, one token: {timed(lambda: serve(w4, x[:1], k)):.3f} ms")


if __name__ == "__main__":
    main()
