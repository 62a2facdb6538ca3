"""The example layer: all ragged operators together, against torch's own
gradients of the same layer in float64.

The layer's intermediates are rounded to bf16 five times on the way forward
and four times back, each rounding 2^-9 of its values and independent over the
H or F terms of the next sum, so that relative errors (2-norm) add up like
sqrt(9) * 2^-9 = 0.006 at most; the bound is four times that."""
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


def reference(w, x, k, ids):
    """The layer on leaf tensors in float64, with the chosen experts given."""
    probs = torch.softmax((x @ w["router"]).gather(1, ids), 1)
    y = torch.zeros_like(x)
    for e in range(w["up"].shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        gate, up = (x[t] @ w["up"][e]).chunk(2, 1)
        out = (torch.nn.functional.silu(gate) * up) @ w["down"][e]
        y = y.index_add(0, t, probs[t, j][:, None] * out)
    return y


@pytest.mark.parametrize("T,E,H,F,k", [(300, 8, 256, 128, 2), (37, 12, 104, 72, 3), (1, 4, 64, 64, 2)])
def test_training_step(T, E, H, F, k):
    w = moe_layer.init(E, H, F)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    dy = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    y, saved = moe_layer.forward(w, x, k)
    grads = moe_layer.backward(w, saved, dy)
    leaf = {n: t.double().requires_grad_() for n, t in w.items()}
    xd = x.double().requires_grad_()
    want = reference(leaf, xd, k, saved[2]["ids"].long())
    want.backward(dy.double())
    near = lambda a, b: float((a.double() - b).norm() / b.norm())         # noqa: E731
    assert near(y, want.detach()) < 0.024
    assert near(grads["x"], xd.grad) < 0.024
    for n in w:
        assert near(grads[n], leaf[n].grad) < 0.024, n
    assert bra.fault_status() == 0


@pytest.mark.parametrize("T", [1, 5, 700])
def test_serving_in_4_bits(T):
    """The 4-bit layer against the same chain with every 4-bit operand turned back into bf16
    (which holds it exactly) and multiplied by grouped_matmul.  Both sum the same exact products
    in fp32, in another order (1e-6 apart at most here), so that about 1e-6 * 2^8 of the bf16
    values in between differ, by one unit of 2^-8, and of those one in fifty its 4-bit code, by a
    third of its value: sqrt(2.6e-4 / 50) / 3 = 8e-4 relative (2-norm), twice; bound 0.01."""
    w = moe_layer.init(8, 256, 128)
    w4 = moe_layer.quantize(w)
    x = torch.randn((T, 256), device="cuda").bfloat16()
    y4 = moe_layer.serve(w4, x, 2)
    r = bra.moe_route(x.float() @ w["router"], 2)
    back = lambda q: bra.mxfp4_dequantize(q, torch.bfloat16)              # noqa: E731
    product = lambda t, q: bra.grouped_matmul(                            # noqa: E731
        back(bra.mxfp4_quantize(t, r["counts"])), back(q), r["counts"], transpose_weight=True)
    gate, up = product(bra.moe_dispatch(x, r["tokens"]), w4["up"]).chunk(2, dim=1)
    ys = product(torch.nn.functional.silu(gate) * up, w4["down"])
    want = bra.moe_combine(ys, r["slots"], r["weights"]).double()
    assert float((y4.double() - want).norm() / want.norm()) < 0.01


def test_one_shot_calls_on_another_stream_own_their_buffers():
    """What a call allocates on a side stream is not handed to the current one while it runs."""
    s = torch.cuda.Stream()
    x = torch.randn((1000, 1026), device="cuda").half()
    w = torch.randn((4, 1026, 778), device="cuda").half()
    c = torch.tensor([250] * 4, device="cuda")
    want = bra.grouped_matmul(x, w, c)
    torch.cuda.synchronize()
    for _ in range(5):
        got = bra.grouped_matmul(x, w, c, stream=s)
        junk = [torch.full((4 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
        s.synchronize()
        assert torch.equal(got, want)
        del junk
    got = bra.grouped_matmul(x, w, c, stream=s.cuda_stream)     # a raw handle
    s.synchronize()
    assert torch.equal(got, want)


def test_a_training_step_in_a_graph():
    """The step's kernels overlap each other's ends; a replay gives the bits of the step run
    call by call, with each call waited for."""
    w = moe_layer.init(8, 264, 96)
    x = torch.randn((700, 264), device="cuda").bfloat16()
    dy = torch.randn((700, 264), device="cuda").bfloat16()
    r = bra.moe_route(x.float() @ w["router"], 2)
    xs = bra.moe_dispatch(x, r["tokens"])
    b = torch.randn((8, 192), device="cuda")
    plans = [bra.grouped_matmul_plan(xs, w["up"], r["counts"], bias=b)]
    plans += [bra.grouped_matmul_grad_plan(plans[0].result, xs, w["up"], r["counts"], bias=b)]
    plans += [bra.moe_dispatch_grad_plan(plans[1].result["dx"], r["slots"])]
    plans += [bra.mxfp4_quantize_plan(plans[1].result["dx"], r["counts"])]
    flat = lambda: [plans[0].result, *plans[1].result.values(), plans[2].result,     # noqa: E731
                    plans[3].result.codes]
    for p in plans:
        p.run()
        torch.cuda.synchronize()
    want = [t.clone() for t in flat()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for p in plans:
            p.run()
    for _ in range(20):
        for t in flat():
            t.zero_()
        graph.replay()
        for a, z in zip(flat(), want):
            assert torch.equal(a, z)
        for t in flat():
            t.zero_()
        for p in plans:
            p.run()
        for a, z in zip(flat(), want):
            assert torch.equal(a, z)


def test_rows_of_several_ranks_reach_their_experts():
    """The router's rows through all_to_all_v to ranks of several experts and on to their products:
    counts are turned into elements on the way, and what arrives by source is sorted by expert."""
    P, El, T, H, N, k = 3, 4, 70, 40, 48, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")                    # noqa: E731
    x = [rnd(T, H).bfloat16() for _ in range(P)]
    w = (rnd(P * El, H, N) * H ** -0.5).bfloat16()
    r = [bra.moe_route(rnd(T, P * El), k) for _ in range(P)]
    xs = [bra.moe_dispatch(x[i], r[i]["tokens"]) for i in range(P)]
    counts = torch.stack([t["counts"] for t in r])                 # (source, expert): rows
    to_rank = counts.view(P, P, El).sum(2)                         # (source, rank): rows
    got = [torch.empty((n, H), dtype=torch.bfloat16, device="cuda") for n in to_rank.sum(0).tolist()]
    bra.all_to_all_v([t.view(torch.int8).view(-1) for t in xs], to_rank * (H * 2),
                     [t.view(torch.int8).view(-1) for t in got], P)
    for j in range(P):
        mine = counts[:, j * El:(j + 1) * El]                      # (source, own expert): rows
        expert = torch.arange(El, device="cuda").repeat(P).repeat_interleave(mine.reshape(-1))
        order = torch.argsort(expert, stable=True)
        y = bra.grouped_matmul(bra.moe_dispatch(got[j], order.int()), w[j * El:(j + 1) * El],
                               mine.sum(0))
        # by the definition, source by source
        at = 0
        for e in range(El):
            rows = [xs[i][r[i]["counts"][:j * El + e].sum():][:r[i]["counts"][j * El + e]]
                    for i in range(P)]
            want = torch.cat(rows).double() @ w[j * El + e].double()
            # fp32 sums of 40 products, one rounding to bf16
            assert ((y[at:at + len(want)].double() - want).abs() <=
                    2.0 ** -8 * want.abs() + 2.0 ** -18).all()
            at += len(want)
        assert at == len(y)
