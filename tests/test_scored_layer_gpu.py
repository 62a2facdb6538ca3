"""The example layer routed by scores, trained, and served in 8 bits.

Bounds as in the plain layer's test: independent roundings of 2^-9 add up like the square root of
their number; the bound is four times that."""
import importlib.util
import os

import pytest
import torch

import bmm_reducescatter_alltoall_gb300 as bra

pytestmark = pytest.mark.gpu

spec = importlib.util.spec_from_file_location(
    "moe_layer", os.path.join(os.path.dirname(__file__), "..", "examples", "moe_layer.py"))
moe_layer = importlib.util.module_from_spec(spec)
spec.loader.exec_module(moe_layer)

near = lambda a, b: float((a.double() - b).norm() / b.norm())             # noqa: E731


def gate_of(E, score="sigmoid", renorm=True):
    g = torch.Generator(device="cuda").manual_seed(3)
    bias = torch.randint(-60, 61, (E,), generator=g, device="cuda") * 0.001
    return {"score": score, "bias": bias, "groups": 4, "top_groups": 2, "scale": 2.5,
            "renormalize": renorm}


def reference(w, x, ids, score, renorm):
    """The layer on leaf tensors in float64, with the chosen experts given."""
    l = x @ w["router"]
    p = (torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)).gather(1, ids)
    probs = 2.5 * (p / p.sum(1, keepdim=True) if renorm else p)
    y = torch.zeros_like(x)
    for e in range(w["up"].shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        gate, up = (x[t] @ w["up"][e]).chunk(2, 1)
        out = (torch.nn.functional.silu(gate) * up) @ w["down"][e]
        y = y.index_add(0, t, probs[t, j][:, None] * out)
    return y


@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("sigmoid", False), ("softmax", False)])
@pytest.mark.parametrize("T,E,H,F,k", [(300, 8, 256, 128, 2), (37, 12, 104, 72, 3), (1, 4, 64, 64, 2)])
def test_training_step_by_scores(T, E, H, F, k, score, renorm):
    w, gate = moe_layer.init(E, H, F), gate_of(E, score, renorm)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    dy = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    y, saved = moe_layer.forward(w, x, k, gate)
    grads = moe_layer.backward(w, saved, dy, gate)
    ids = saved[2]["ids"].long()
    assert (ids >= 0).all()
    leaf = {n: t.double().requires_grad_() for n, t in w.items()}
    xd = x.double().requires_grad_()
    want = reference(leaf, xd, ids, score, renorm)
    want.backward(dy.double())
    assert near(y, want.detach()) < 0.024
    assert near(grads["x"], xd.grad) < 0.024
    for n in w:
        assert near(grads[n], leaf[n].grad) < 0.024, n
    assert bra.fault_status() == 0


@pytest.mark.parametrize("T,E", [(1, 8), (5, 8), (700, 8), (4000, 4)])
def test_serving_in_8_bits(T, E):
    """The 8-bit layer against the same chain with the values of every 8-bit operand in 64 bits:
    three roundings to bf16 (each product's rows, the activation) and the last one."""
    H, F, k = 256, 136, 2
    w = moe_layer.init(E, H, F)
    w8, gate = moe_layer.quantize8(w), gate_of(E)
    x = torch.randn((T, H), device="cuda").bfloat16()
    y = moe_layer.serve8(w8, x, k, gate)
    r = bra.moe_route(x.float() @ w8["router"], k, **gate)
    owner = torch.repeat_interleave(torch.arange(E, device="cuda"), r["counts"])
    value = lambda q: bra.fp8_dequantize(q, torch.float32).double()       # noqa: E731

    def product(rows, weight):
        v, out = value(bra.fp8_quantize(rows)), []
        for e in range(E):
            out.append(v[owner == e] @ value(weight)[e].t())
        return torch.cat(out).to(rows.dtype)
    g, up = product(x[r["tokens"].long()], w8["up"]).chunk(2, 1)
    ys = product(torch.nn.functional.silu(g) * up, w8["down"])
    want = (ys.double()[r["slots"].long()] * r["weights"].double()[:, :, None]).sum(1)
    # a bf16 that falls to the other side of a tie moves an 8-bit code by 2^-3 of its value: those
    # are some 2^-16 / 2^-4 of the elements, far below the roundings' own share
    assert near(y, want) < 4 * 2 ** -9 * 3 ** 0.5
    assert bra.fault_status() == 0


def test_an_8_bit_layer_in_a_graph():
    E, H, F, k, T = 8, 128, 128, 2, 90
    w8, gate = moe_layer.quantize8(moe_layer.init(E, H, F)), gate_of(E)
    x = torch.randn((T, H), device="cuda").bfloat16()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        moe_layer.serve8(w8, x, k, gate)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = moe_layer.serve8(w8, x, k, gate)
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn((T, H), generator=g, device="cuda"))
        gate["bias"].copy_(torch.rand(E, generator=g, device="cuda") * 0.1)
        graph.replay()
        assert torch.equal(y, moe_layer.serve8(w8, x, k, gate))


def test_balance_runs_on_the_device():
    bias, counts = torch.zeros(4, device="cuda"), torch.tensor([1, 5, 3, 3], device="cuda")
    moe_layer.balance(bias, counts)
    assert torch.equal(bias, torch.tensor([0.001, -0.001, 0.0, 0.0], device="cuda"))
