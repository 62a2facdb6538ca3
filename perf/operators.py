"""Workloads of the ragged mixture-of-experts operators: what is timed, and what it is compared with.

Kinds of case
  gmm       grouped_matmul: rows sorted by expert times that expert's weight (inference)
  train     grouped_matmul, then its gradients: y, dx, dweight and dbias of one step
  quantize  mxfp4_quantize, then mxfp4_dequantize: the values that 4 bits hold
  mx        mxfp4_quantize of the rows, then mxfp4_grouped_matmul with kept 4-bit weights
  route     moe_route; with "grad" also the gradient of the logits
  permute   moe_dispatch and moe_combine; with "grad" also their gradients

Every kind has a plain form in elementary torch operations in 32 bits, and the definition in 64
bits (`exact`).
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
LOWEST = torch.finfo(torch.float32).min
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MAX_FLOPS = 2.0 * 131072 * 2048 * 4096        # the largest product listed below


def listed():
    return [
        # One token's two experts: a single decoding step, where the weights' bytes and latency count.
        {"name": "gmm-token", "kind": "gmm", "dtype": "bf16", "E": 8, "tokens": 1, "k": 2,
         "K": 2048, "N": 4096, "bias": False, "wt": False, "skew": 0.0},
        # A decoding batch of 16 sequences over 64 experts: many experts, one to four rows each.
        {"name": "gmm-decode", "kind": "gmm", "dtype": "fp16", "E": 64, "tokens": 16, "k": 8,
         "K": 2048, "N": 4096, "bias": True, "wt": True, "skew": 0.0},
        # A prompt batch: 16384 tokens, eight experts each, unevenly loaded.
        {"name": "gmm-prefill", "kind": "gmm", "dtype": "bf16", "E": 64, "tokens": 16384, "k": 8,
         "K": 2048, "N": 4096, "bias": False, "wt": False, "skew": 1.0},
        # A training step with rows that have no 16-byte pitch and uneven, partly empty experts.
        {"name": "train-odd", "kind": "train", "dtype": "fp16", "E": 12, "tokens": 1021, "k": 3,
         "K": 1026, "N": 775, "bias": True, "wt": False, "skew": 1.5},
        # A training step of one rank's eight experts.
        {"name": "train", "kind": "train", "dtype": "bf16", "E": 8, "tokens": 8192, "k": 2,
         "K": 2048, "N": 4096, "bias": True, "wt": False, "skew": 0.5},
        # Quantising an activation or a weight block of 64 Mi values.
        {"name": "quantize", "kind": "quantize", "dtype": "bf16", "rows": 16384, "K": 4096},
        # The decoding batch on 4-bit experts.
        {"name": "mx-decode", "kind": "mx", "dtype": "bf16", "E": 64, "tokens": 16, "k": 8,
         "K": 2048, "N": 4096, "bias": False, "skew": 0.0},
        # A prompt batch on 4-bit experts.
        {"name": "mx-prefill", "kind": "mx", "dtype": "bf16", "E": 16, "tokens": 16384, "k": 4,
         "K": 4096, "N": 4096, "bias": True, "skew": 0.5},
        # The router of one decoding batch.
        {"name": "route-decode", "kind": "route", "dtype": "bf16", "tokens": 64, "E": 64, "k": 8,
         "renorm": True, "grad": False},
        # The router of a training batch, with masked experts and padding tokens.
        {"name": "route-train", "kind": "route", "dtype": "fp32", "tokens": 65536, "E": 128, "k": 8,
         "renorm": True, "grad": True},
        # Moving one decoding batch's rows to their experts and back.
        {"name": "permute-decode", "kind": "permute", "dtype": "fp16", "tokens": 16, "E": 64,
         "k": 8, "H": 4096, "grad": False},
        # The same for a training batch, with the gradients.
        {"name": "permute-train", "kind": "permute", "dtype": "bf16", "tokens": 16384, "E": 64,
         "k": 8, "H": 4096, "grad": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row length spread over the logarithm: odd, or an odd multiple of 8 or of 64."""
    m = rng.choice((1, 8, 64))
    return (_log(rng, lo, hi) // m | 1) * m


def draw(rng):
    kind = rng.choice(("gmm", "gmm", "train", "train", "quantize", "mx", "mx", "route", "permute"))
    half = rng.choice(("fp16", "bf16"))
    if kind in ("gmm", "train", "mx"):
        while True:
            E = _log(rng, 2, 64)
            c = {"kind": kind, "dtype": half, "E": E, "tokens": _log(rng, 1, 16384),
                 "k": rng.randint(1, min(8, E)), "K": _width(rng, 64, 4096),
                 "N": _width(rng, 64, 4096), "bias": rng.random() < 0.5}
            if kind != "mx":
                c["wt"] = rng.random() < 0.5
            c["skew"] = round(rng.uniform(0.0, 1.5), 2) if c["tokens"] * c["k"] >= 32 * E else 0.0
            if work(c)["flops"] <= MAX_FLOPS / 2:
                return c
    if kind == "quantize":
        return {"kind": kind, "dtype": half, "rows": _log(rng, 1, 16384), "K": _width(rng, 32, 4096)}
    if kind == "route":
        E = _log(rng, 2, 512)
        return {"kind": kind, "dtype": rng.choice(("fp32", half)),
                "tokens": _log(rng, 1, 65536 if E <= 128 else 16384), "E": E,
                "k": rng.randint(1, min(16, E)), "renorm": rng.random() < 0.5,
                "grad": rng.random() < 0.5}
    E = _log(rng, 2, 64)
    return {"kind": kind, "dtype": half, "tokens": _log(rng, 1, 16384), "E": E,
            "k": rng.randint(1, min(8, E)), "H": _width(rng, 64, 4096), "grad": rng.random() < 0.5}


# ---------------------------------------------------------------------------------------------
# Work
# ---------------------------------------------------------------------------------------------

def _active(c):
    """Experts that are expected to have rows (each token takes k different ones, evenly)."""
    return c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["tokens"])


def work(c):
    kind = c["kind"]
    if kind == "quantize":
        n = c["rows"] * c["K"]
        # 16 bits in, 4.25 bits held, 16 bits back out of them
        return {"bytes": n * (2 + 2 + 2 * 4.25 / 8), "flops": 0}
    if kind in ("gmm", "train", "mx"):
        R, K, N, E = c["tokens"] * c["k"], c["K"], c["N"], c["E"]
        flops = 2.0 * R * K * N
        if kind == "mx":
            # rows are read once in 16 bits, written and read in 4.25
            return {"bytes": R * K * (2 + 2 * 4.25 / 8) + _active(c) * K * N * 4.25 / 8 + 2 * R * N,
                    "flops": flops}
        fwd = 2.0 * (R * K + _active(c) * K * N + R * N)
        if kind == "gmm":
            return {"bytes": fwd, "flops": flops}
        # forward; then dy, x and the weight read, dx and every expert's dweight written
        return {"bytes": fwd + 2.0 * (R * N + R * K + _active(c) * K * N + R * K + E * K * N),
                "flops": 3 * flops}
    es = 4 if c["dtype"] == "fp32" else 2
    if kind == "route":
        T, E, k = c["tokens"], c["E"], c["k"]
        n = T * E * es + T * k * (4 + 4 + 4 + 4) + E * 8
        if c["grad"]:
            n += 2 * T * E * es + T * k * (4 + 4 + 4)
        return {"bytes": n, "flops": 0}
    T, k, H = c["tokens"], c["k"], c["H"]
    R = T * k
    n = (T + R) * H * es + R * 4              # dispatch: each token read once, each row written
    n += (R + T) * H * es + R * 8             # combine: each row read, each token written
    if c["grad"]:
        n += (R + T) * H * es + R * 4         # dispatch's: as combine
        n += (T + R + R) * H * es + R * 16    # combine's: dy and ys read, dys and dw written
    return {"bytes": n, "flops": 0}


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _routing(c, g, dev):
    """Each token's k different experts (int64 (tokens, k)): expert popularity with a log-normal
    spread of `skew`; with a spread, one expert in six gets nothing."""
    E, skew = c["E"], c.get("skew", 0.5)
    pop = torch.randn(E, generator=g, device=dev) * skew
    if skew > 0 and E - E // 6 >= c["k"]:
        pop[torch.randperm(E, generator=g, device=dev)[:E // 6]] = -1e9
    noise = torch.rand((c["tokens"], E), generator=g, device=dev).clamp_(1e-12, 1 - 1e-7)
    return (pop - torch.log(-torch.log(noise))).topk(c["k"], dim=1).indices


def _counts(c, g, dev):
    return torch.bincount(_routing(c, g, dev).reshape(-1), minlength=c["E"])


def _randn(shape, dtype, g, dev, scale=1.0):
    """Normal values, made 64 Mi at a time (the 32-bit intermediate stays small)."""
    t = torch.empty(shape, dtype=dtype, device=dev)
    for part in t.view(-1).split(1 << 26):
        part.copy_(torch.randn(part.shape, generator=g, device=dev).mul_(scale))
    return t


def _outliers(t, g, dev):
    """Activations with a few channels far larger than the rest, and rows of different scale."""
    T, K = t.shape
    t *= torch.exp2(torch.randint(-6, 7, (T, 1), generator=g, device=dev)).to(t.dtype)
    cols = torch.randint(0, K, (max(1, K // 100),), generator=g, device=dev)
    t[:, cols] *= 16
    return t


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 13)
    s = {"case": c}
    kind, dt = c["kind"], DTYPES[c["dtype"]]
    if kind in ("gmm", "train", "mx"):
        E, K, N, R = c["E"], c["K"], c["N"], c["tokens"] * c["k"]
        s["counts"] = _counts(c, g, dev)
        s["sizes"] = s["counts"].tolist()
        s["x"] = _randn((R, K), dt, g, dev)
        w = _randn((E, N, K) if kind == "mx" or c["wt"] else (E, K, N), dt, g, dev, K ** -0.5)
        bdt = torch.float16 if dt == torch.float16 else torch.float32
        s["bias"] = _randn((E, N), bdt, g, dev) if c["bias"] else None
        if kind == "train":
            s["dy"] = _randn((R, N), dt, g, dev)
        if kind == "mx":
            s["wcodes"], s["wscales"] = _quantize(w)
        else:
            s["weight"] = w
    elif kind == "quantize":
        s["x"] = _outliers(_randn((c["rows"], c["K"]), dt, g, dev), g, dev)
    elif kind == "route":
        T, E = c["tokens"], c["E"]
        l = _randn((T, E), torch.float32, g, dev, 2.0) + torch.randn(E, generator=g, device=dev)
        if E >= 8:
            l[:, torch.randint(0, E, (1,), generator=g, device=dev)] = -math.inf  # closed expert
        hidden = torch.rand((T, E), generator=g, device=dev) < 0.02
        l = l.masked_fill(hidden, torch.finfo(dt).min)
        padding = torch.rand((T, 1), generator=g, device=dev) < 0.03              # no experts
        s["logits"] = l.masked_fill(padding, -math.inf).to(dt)
        if c["grad"]:
            s["dw"] = _randn((T, c["k"]), torch.float32, g, dev)
    else:
        T, k, H = c["tokens"], c["k"], c["H"]
        ids = _routing(c, g, dev)
        order = torch.sort(ids.reshape(-1), stable=True).indices
        s["tokens"] = (order // k).to(torch.int32)
        slots = torch.empty(T * k, dtype=torch.int32, device=dev)
        slots[order] = torch.arange(T * k, dtype=torch.int32, device=dev)
        s["slots"] = slots.view(T, k)
        s["w"] = torch.softmax(torch.randn((T, k), generator=g, device=dev), dim=1)
        s["x"], s["ys"] = _randn((T, H), dt, g, dev), _randn((T * k, H), dt, g, dev)
        if c["grad"]:
            s["dxs"], s["dy"] = _randn((T * k, H), dt, g, dev), _randn((T, H), dt, g, dev)
    if own:
        s["calls"] = _calls(s, w if kind == "mx" else None)
    return s


# ---------------------------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------------------------

def _calls(s, w):
    """The calls of one pass, prepared once on the state's buffers."""
    import bmm_reducescatter_alltoall_gb300 as bra
    c, kind = s["case"], s["case"]["kind"]
    if kind in ("gmm", "train"):
        fwd = bra.grouped_matmul_plan(s["x"], s["weight"], s["counts"], bias=s["bias"],
                                      transpose_weight=c["wt"])
        if kind == "gmm":
            return [fwd]
        return [fwd, bra.grouped_matmul_grad_plan(s["dy"], s["x"], s["weight"], s["counts"],
                                                  bias=s["bias"], transpose_weight=c["wt"])]
    if kind == "quantize":
        q = bra.mxfp4_quantize_plan(s["x"])
        return [q, bra.mxfp4_dequantize_plan(q.result, s["x"].dtype)]
    if kind == "mx":
        q = bra.mxfp4_quantize_plan(s["x"], s["counts"])
        return [q, bra.mxfp4_grouped_matmul_plan(q.result, bra.mxfp4_quantize(w), s["counts"],
                                                 bias=s["bias"], dtype=s["x"].dtype)]
    if kind == "route":
        r = bra.moe_route_plan(s["logits"], c["k"], renormalize=c["renorm"])
        if not c["grad"]:
            return [r]
        return [r, bra.moe_route_grad_plan(s["dw"], s["logits"], r.result["ids"],
                                           r.result["weights"], renormalize=c["renorm"])]
    calls = [bra.moe_dispatch_plan(s["x"], s["tokens"]),
             bra.moe_combine_plan(s["ys"], s["slots"], s["w"])]
    if c["grad"]:
        calls += [bra.moe_dispatch_grad_plan(s["dxs"], s["slots"]),
                  bra.moe_combine_grad_plan(s["dy"], s["ys"], s["slots"], s["w"], s["tokens"])]
    return calls


def _run_own(s):
    kind = s["case"]["kind"]
    got = [call.run() for call in s["calls"]]
    if kind in ("gmm", "quantize", "mx"):
        return {("values" if kind == "quantize" else "y"): got[-1]}
    if kind == "train":
        out = {"y": got[0], "dx": got[1]["dx"], "dweight": got[1]["dweight"]}
        if s["bias"] is not None:
            out["dbias"] = got[1]["dbias"]
        return out
    if kind == "route":
        out = {n: got[0][n] for n in ("ids", "weights", "counts", "slots", "tokens")}
        if len(got) > 1:
            out["dlogits"] = got[1]
        return out
    out = {"xs": got[0], "y": got[1]}
    if len(got) > 2:
        out.update(dx=got[2], dys=got[3]["dys"], dw=got[3]["dweights"])
    return out


# ---------------------------------------------------------------------------------------------
# Plain form
# ---------------------------------------------------------------------------------------------

def _quantize(x):
    """Codes (a byte each, 0..15) and scale bytes of the last dimension in blocks of 32."""
    K = x.shape[-1]
    x = torch.nn.functional.pad(x.float(), (0, -K % 32)).unflatten(-1, (-1, 32))
    amax = x.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent.clamp(min=-10000) - 3, -127)
    e = e.clamp(-127, 127).to(torch.int32)
    a = x * ((127 - e) << 23).view(torch.float32)
    m = a.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) +
            (m >= 3.5) + (m > 5.0))
    code = code | (torch.signbit(a).to(torch.uint8) << 3)
    return code.flatten(-2)[..., :K].contiguous(), (e + 127).to(torch.uint8).squeeze(-1)


def _dequantize(codes, scales):
    K = codes.shape[-1]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    b = scales.to(torch.int32)
    s = torch.where(b > 0, b << 23, 1 << 22).view(torch.float32)      # 2^(b - 127)
    return table[codes.to(torch.int32)] * s.repeat_interleave(32, dim=-1)[..., :K]


def _parts(sizes):
    """(expert, first row, past the last row) of every expert that has rows."""
    at = [0]
    for n in sizes:
        at.append(at[-1] + n)
    return [(e, at[e], at[e + 1]) for e in range(len(sizes)) if sizes[e]]


def _grouped(x, sizes, weight_of, bias, out):
    for e, a, b in _parts(sizes):
        y = torch.matmul(x[a:b].float(), weight_of(e))
        out[a:b] = y if bias is None else y + bias[e].float()
    return out


def _plain_products(s):
    c, x, sizes = s["case"], s["x"], s["sizes"]
    y = torch.empty((x.shape[0], c["N"]), dtype=x.dtype, device=x.device)
    if c["kind"] == "mx":
        q = _dequantize(*_quantize(x))
        _grouped(q, sizes, lambda e: _dequantize(s["wcodes"][e], s["wscales"][e]).t(), s["bias"], y)
        return {"y": y}
    w = s["weight"].transpose(1, 2) if c["wt"] else s["weight"]
    _grouped(x, sizes, lambda e: w[e].float(), s["bias"], y)
    if c["kind"] == "gmm":
        return {"y": y}
    dx, dw = torch.empty_like(x), torch.zeros_like(s["weight"])
    dwv = dw.transpose(1, 2) if c["wt"] else dw
    out = {"y": y, "dx": dx, "dweight": dw}
    if s["bias"] is not None:
        out["dbias"] = torch.zeros_like(s["bias"])
    for e, a, b in _parts(sizes):
        d = s["dy"][a:b].float()
        dx[a:b] = torch.matmul(d, w[e].float().t())
        dwv[e] = torch.matmul(x[a:b].float().t(), d)
        if s["bias"] is not None:
            out["dbias"][e] = d.sum(0)
    return out


def _plain_route(s):
    c, k = s["case"], s["case"]["k"]
    l = s["logits"].float().clamp(max=-LOWEST)
    T, E = l.shape
    valid = l > -math.inf
    top, ids = torch.sort(l, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    has = top > -math.inf
    peak = torch.where(has[:, :1], top[:, :1], 0.0)
    p = torch.where(valid, torch.exp(l - peak), 0.0)
    p = p / p.sum(1, keepdim=True).clamp(min=1e-30)
    chosen = torch.where(has, torch.exp(top - peak), 0.0)
    if c["renorm"]:
        w = chosen / chosen.sum(1, keepdim=True).clamp(min=1e-30)
    else:
        w = torch.where(has, p.gather(1, ids), 0.0)
    group = torch.where(has, ids, E).reshape(-1)
    order = torch.sort(group, stable=True).indices
    counts = (group[:, None] == torch.arange(E, device=l.device)).sum(0) if T * k * E < 1 << 28 \
        else torch.bincount(group, minlength=E + 1)[:E]
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device=l.device)
    used = torch.arange(T * k, device=l.device) < counts.sum()
    out = {"ids": torch.where(has, ids, -1).to(torch.int32), "weights": w, "counts": counts,
           "slots": torch.where(has, place.view(T, k), -1).to(torch.int32),
           "tokens": torch.where(used, order // k, -1).to(torch.int32)}
    if c["grad"]:
        g = torch.where(has, s["dw"], 0.0)
        mean = (w * g).sum(1, keepdim=True)
        if c["renorm"]:
            d = torch.zeros_like(l).scatter_add(1, ids, w * (g - mean))
        else:
            d = p * (torch.zeros_like(l).scatter_add(1, ids, g) - mean)
        out["dlogits"] = d.to(s["logits"].dtype)
    return out


def _plain_permute(s):
    c, dt = s["case"], s["x"].dtype
    T, k, H = c["tokens"], c["k"], c["H"]
    tok, slot = s["tokens"].long(), s["slots"].long()
    out = {"xs": s["x"][tok],
           "y": (s["ys"][slot].float() * s["w"][:, :, None]).sum(1).to(dt)}
    if c["grad"]:
        out["dx"] = s["dxs"][slot].float().sum(1).to(dt)
        dy = s["dy"].float()
        dys = torch.empty_like(s["ys"])
        dys[slot.reshape(-1)] = (s["w"][:, :, None] * dy[:, None]).reshape(T * k, H).to(dt)
        out["dys"] = dys
        out["dw"] = (s["ys"][slot].float() * dy[:, None]).sum(2)
    return out


def _plain_quantize(s):
    return {"values": _dequantize(*_quantize(s["x"])).to(s["x"].dtype)}


_PLAIN = {"gmm": _plain_products, "train": _plain_products, "mx": _plain_products,
          "quantize": _plain_quantize, "route": _plain_route, "permute": _plain_permute}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["kind"]](state)


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _pow2(n):
    """2^n for whole n in double, by its exponent field."""
    return ((n.clamp(-1000, 1000).to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_mx(x):
    """The nearest multiple of each block's power of two among the eight magnitudes (a tie goes to
    the even code), as values, 16 Mi at a time."""
    K = x.shape[-1]
    rows = x.reshape(-1, K)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    out = torch.empty(rows.shape, dtype=torch.float64, device=x.device)
    step = max(1, (1 << 24) // K)
    for a in range(0, rows.shape[0], step):
        v = rows[a:a + step].double()
        n = -(-K // 32)
        v = torch.cat([v, v.new_zeros((v.shape[0], n * 32 - K))], 1).view(v.shape[0], n, 32)
        big = v.abs().max(2, keepdim=True).values
        f = torch.floor(torch.log2(big))                  # the logarithm is rounded: step to
        f = f + (_pow2(f + 1) <= big).double()            # the power of two that is not above
        f = f - (_pow2(f) > big).double()
        unit = _pow2((f - 2).clamp(-127, 127))
        u = (v / unit).abs()
        hi = torch.searchsorted(grid, u.contiguous()).clamp(1, 7)
        lo = hi - 1
        below, above = u - grid[lo], grid[hi] - u
        pick = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
        q = (grid[pick] * torch.sign(v) * unit).view(v.shape[0], n * 32)[:, :K]
        out[a:a + step] = q
    return out.view(x.shape)


def _exact_products(s):
    c = s["case"]
    K, N, E = c["K"], c["N"], c["E"]
    owner = torch.repeat_interleave(torch.arange(E, device="cuda"), s["counts"])
    if c["kind"] == "mx":
        x = _exact_mx(s["x"])
        lut = torch.tensor([v for v in E2M1] + [-v for v in E2M1], dtype=torch.float64,
                           device="cuda")
        weight = lambda e: (lut[s["wcodes"][e].long()] * _pow2(                      # noqa: E731
            s["wscales"][e].double() - 127)[:, torch.arange(K, device="cuda") // 32]).t()
    else:
        x = s["x"].double()
        weight = lambda e: (s["weight"][e].t() if c["wt"] else s["weight"][e]).double()  # noqa: E731
    y = torch.zeros((x.shape[0], N), dtype=torch.float64, device="cuda")
    out = {"y": y}
    if c["kind"] == "train":
        out["dx"] = torch.zeros((x.shape[0], K), dtype=torch.float64, device="cuda")
        out["dweight"] = torch.zeros(s["weight"].shape, dtype=torch.float64, device="cuda")
        if s["bias"] is not None:
            out["dbias"] = torch.zeros((E, N), dtype=torch.float64, device="cuda")
    for e in range(E):
        rows = (owner == e).nonzero().squeeze(1)
        if rows.numel() == 0:
            continue
        w, xe = weight(e), x[rows]
        y[rows] = torch.einsum("rk,kn->rn", xe, w)
        if s["bias"] is not None:
            y[rows] += s["bias"][e].double()
        if c["kind"] == "train":
            d = s["dy"][rows].double()
            out["dx"][rows] = torch.einsum("rn,kn->rk", d, w)
            out["dweight"][e] = torch.einsum("rn,rk->nk" if c["wt"] else "rk,rn->kn",
                                             *((d, xe) if c["wt"] else (xe, d)))
            if s["bias"] is not None:
                out["dbias"][e] = torch.einsum("rn->n", d)
    return out


def _exact_route(s):
    c, k = s["case"], s["case"]["k"]
    l = s["logits"].double()
    T, E = l.shape
    left, picks, tops = l.clone(), [], []
    for _ in range(k):
        v = left.max(1, keepdim=True).values
        first = (left == v).to(torch.int8).argmax(1, keepdim=True)      # the lowest index of a tie
        picks.append(first)
        tops.append(v)
        left.scatter_(1, first, -math.inf)
    ids, top = torch.cat(picks, 1), torch.cat(tops, 1)
    has = top > -math.inf
    some = has.any(1, keepdim=True)
    p = torch.nan_to_num(torch.softmax(l, 1), nan=0.0) * some
    w = p.gather(1, ids) * has
    if c["renorm"]:
        w = torch.nan_to_num(torch.softmax(torch.where(some, top, 0.0), 1)) * has
    out = {"ids": None, "weights": w, "counts": None, "slots": None, "tokens": None}
    if c["grad"]:
        onehot = torch.zeros((T, k, E), dtype=torch.bool, device="cuda") if T * k * E < 1 << 28 else None
        g = s["dw"].double() * has
        if c["renorm"]:
            d = torch.zeros_like(l)
            d.scatter_(1, ids, w * g - w * torch.einsum("tk,tk->t", w, g)[:, None])
        elif onehot is not None:
            onehot.scatter_(2, ids[:, :, None], True)
            gi = torch.einsum("tke,tk->te", onehot.double(), g)
            d = p * gi - p * torch.einsum("te,te->t", p, gi)[:, None]
        else:
            d = None
        out["dlogits"] = d
    return out


def _exact_permute(s):
    c = s["case"]
    T, k = c["tokens"], c["k"]
    slots = s["slots"].long()
    ident = s["x"].double().index_select(0, s["tokens"].long())
    y = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    for j in range(k):
        y += s["ys"].index_select(0, slots[:, j]).double() * s["w"][:, j:j + 1].double()
    out = {"xs": ident, "y": y}
    if c["grad"]:
        out["dx"], out["dys"] = torch.zeros_like(y), torch.zeros_like(ident)
        out["dw"] = torch.zeros((T, k), dtype=torch.float64, device="cuda")
        dy = s["dy"].double()
        for j in range(k):
            out["dx"] += s["dxs"].index_select(0, slots[:, j]).double()
            out["dys"].index_copy_(0, slots[:, j], dy * s["w"][:, j:j + 1].double())
            out["dw"][:, j] = torch.einsum(
                "th,th->t", dy, s["ys"].index_select(0, slots[:, j]).double())
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    kind = case["kind"]
    if kind == "quantize":
        return {"values": _exact_mx(s["x"])}
    if kind == "route":
        return _exact_route(s)
    if kind == "permute":
        return _exact_permute(s)
    return _exact_products(s)
