"""Workloads of the 8-bit expert products and of the scored router: what is timed, and what it is
compared with.

Kinds of case
  quantize  fp8_quantize, then fp8_dequantize: the values that 8 bits and the blocks' scales hold;
            rows with a scale to each 128 elements, or weights with one to each 128 x 128
  product   fp8_quantize of the rows, then fp8_grouped_matmul with kept 8-bit weights (inference)
  train     fp8_quantize of the weights, the rows and the output's gradient, fp8_grouped_matmul and
            fp8_grouped_matmul_grad: y and dx of one step
  route     moe_route by scores: sigmoid or softmax, a bias that moves the choice alone, experts
            limited to the best groups; with "grad" also the gradient of the logits

Every kind has a plain form in elementary torch operations in 32 bits (the router's choice in 64:
scores next to each other decide it), and the definition in 64 bits (`exact`).
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
FORMATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = torch.finfo(torch.float32).max
MAX_FLOPS = 2.0 * 65536 * 4096 * 4096         # the largest product listed below


def listed():
    return [
        # An activation matrix of one prompt batch, a scale to each 128 elements of a row.
        {"name": "quantize-rows", "kind": "quantize", "dtype": "bf16", "format": "e4m3",
         "E": 0, "N": 16384, "K": 4096},
        # Eight experts' weights, a scale to each 128 x 128.
        {"name": "quantize-weights", "kind": "quantize", "dtype": "bf16", "format": "e4m3",
         "E": 8, "N": 4096, "K": 2048},
        # One token's eight experts: a single decoding step, latency and the weights' bytes count.
        {"name": "product-token", "kind": "product", "dtype": "bf16", "E": 64, "tokens": 1, "k": 8,
         "K": 2048, "N": 4096, "bias": False, "skew": 0.0},
        # A decoding batch of 16 sequences over 64 experts: one to four rows each.
        {"name": "product-decode", "kind": "product", "dtype": "fp16", "E": 64, "tokens": 16, "k": 8,
         "K": 2048, "N": 4096, "bias": True, "skew": 0.0},
        # Ragged, partly empty experts with widths that fill no block.
        {"name": "product-odd", "kind": "product", "dtype": "fp16", "E": 12, "tokens": 1021, "k": 3,
         "K": 1026, "N": 775, "bias": True, "skew": 1.5},
        # A prompt batch on 16 experts.
        {"name": "product-prefill", "kind": "product", "dtype": "bf16", "E": 16, "tokens": 16384,
         "k": 4, "K": 4096, "N": 4096, "bias": True, "skew": 0.5},
        # A training step of ragged experts with odd widths.
        {"name": "train-odd", "kind": "train", "dtype": "fp16", "dy": "e4m3", "E": 12,
         "tokens": 1021, "k": 3, "K": 1026, "N": 775, "skew": 1.5},
        # A training step of one rank's eight experts; the gradient in the format of wider range.
        {"name": "train", "kind": "train", "dtype": "bf16", "dy": "e5m2", "E": 8, "tokens": 8192,
         "k": 2, "K": 2048, "N": 4096, "skew": 0.5},
        # The router of one decoding batch: 8 of 256 experts from the best 4 of 8 groups.
        {"name": "route-decode", "kind": "route", "dtype": "bf16", "tokens": 64, "E": 256, "k": 8,
         "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_best": 2,
         "renorm": True, "scale": 2.5, "grad": False},
        # A prompt batch by softmax scores, groups ranked by their best expert.
        {"name": "route-prefill", "kind": "route", "dtype": "bf16", "tokens": 16384, "E": 160,
         "k": 6, "score": "softmax", "bias": False, "groups": 8, "top_groups": 3, "group_best": 1,
         "renorm": False, "scale": 1.0, "grad": False},
        # A training batch without groups: the bias alone balances.
        {"name": "route-bias", "kind": "route", "dtype": "fp32", "tokens": 16384, "E": 64, "k": 6,
         "score": "softmax", "bias": True, "groups": 1, "top_groups": 1, "group_best": 2,
         "renorm": False, "scale": 1.0, "grad": True},
        # A training batch, masked experts and padding tokens among it.
        {"name": "route-train", "kind": "route", "dtype": "fp32", "tokens": 65536, "E": 256, "k": 8,
         "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_best": 2,
         "renorm": True, "scale": 2.5, "grad": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row length spread over the logarithm: odd, or an odd multiple of 8, of 64 or of 128."""
    m = rng.choice((1, 8, 64, 128))
    return (_log(rng, lo, hi) // m | 1) * m


def draw(rng):
    kind = rng.choice(("quantize", "product", "product", "product", "train", "train", "route",
                       "route", "route"))
    half = rng.choice(("fp16", "bf16"))
    if kind == "quantize":
        c = {"kind": kind, "dtype": rng.choice((half, half, "fp32")),
             "format": rng.choice(("e4m3", "e4m3", "e5m2")),
             "E": rng.choice((0, 0, _log(rng, 1, 16))), "K": _width(rng, 32, 4096)}
        c["N"] = _log(rng, 1, 16384) if c["E"] == 0 else _width(rng, 8, 16384 // c["E"])
        return c
    if kind in ("product", "train"):
        while True:
            E = _log(rng, 2, 64)
            c = {"kind": kind, "dtype": half, "E": E, "tokens": _log(rng, 1, 16384),
                 "k": rng.randint(1, min(8, E)), "K": _width(rng, 64, 4096),
                 "N": _width(rng, 64, 4096)}
            if kind == "product":
                c["bias"] = rng.random() < 0.5
            else:
                c["dy"] = rng.choice(("e4m3", "e5m2"))
            c["skew"] = round(rng.uniform(0.0, 1.5), 2) if c["tokens"] * c["k"] >= 32 * E else 0.0
            if work(c)["flops"] <= MAX_FLOPS / 2:
                return c
    groups = rng.choice((1, 2, 4, 8, 8, 16))
    E = groups * _log(rng, 2, 512 // groups)
    kept = rng.randint(1, groups)
    return {"kind": kind, "dtype": rng.choice(("fp32", half)),
            "tokens": _log(rng, 1, 65536 if E <= 256 else 16384), "E": E,
            "k": rng.randint(1, min(16, E // groups * kept)),
            "score": rng.choice(("sigmoid", "sigmoid", "softmax")), "bias": rng.random() < 0.7,
            "groups": groups, "top_groups": kept, "group_best": rng.choice((1, 2)),
            "renorm": rng.random() < 0.5, "scale": rng.choice((1.0, 2.5)),
            "grad": rng.random() < 0.5}


# ---------------------------------------------------------------------------------------------
# Work
# ---------------------------------------------------------------------------------------------

def _active(c):
    """Experts that are expected to have rows (each token takes k different ones, evenly)."""
    return c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["tokens"])


def work(c):
    kind = c["kind"]
    es = 4 if c["dtype"] == "fp32" else 2
    if kind == "quantize":
        n = max(c["E"], 1) * c["N"] * c["K"]
        s = 4.0 * n / 128 if c["E"] == 0 else 4.0 * n / 128 / 128
        return {"bytes": n * (es + 1 + 1 + es) + 2 * s, "flops": 0}
    if kind in ("product", "train"):
        R, K, N, E = c["tokens"] * c["k"], c["K"], c["N"], c["E"]
        held = 2 * (1 + 4.0 / 128)               # a row's element written and read in 8 bits
        if kind == "product":
            return {"bytes": R * K * (2 + held) + _active(c) * K * N + 2 * R * N,
                    "flops": 2.0 * R * K * N}
        # every weight quantized, then those of the experts with rows read twice
        return {"bytes": E * K * N * 3 + 2 * _active(c) * K * N + R * K * (2 + held) + 2 * R * N
                + R * N * (2 + held) + 2 * R * K,
                "flops": 4.0 * R * K * N}
    T, E, k = c["tokens"], c["E"], c["k"]
    n = T * E * es + T * k * (4 + 4 + 4 + 4) + E * 8 + (E * 4 if c["bias"] else 0)
    if c["grad"]:
        # the logits are needed at the chosen experts, or (softmax over all) everywhere
        n += T * E * es + T * k * (4 + 4 + 4)
        n += T * k * es if c["score"] == "sigmoid" else 0 if c["renorm"] else T * E * es
    return {"bytes": n, "flops": 0}


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _counts(c, g, dev):
    """Rows of each expert when every token takes k different ones: expert popularity with a
    log-normal spread of `skew`; with a spread, one expert in six gets nothing."""
    E, skew = c["E"], c["skew"]
    pop = torch.randn(E, generator=g, device=dev) * skew
    if skew > 0 and E - E // 6 >= c["k"]:
        pop[torch.randperm(E, generator=g, device=dev)[:E // 6]] = -1e9
    noise = torch.rand((c["tokens"], E), generator=g, device=dev).clamp_(1e-12, 1 - 1e-7)
    ids = (pop - torch.log(-torch.log(noise))).topk(c["k"], dim=1).indices
    return torch.bincount(ids.reshape(-1), minlength=E)


def _randn(shape, dtype, g, dev, scale=1.0):
    """Normal values, made 64 Mi at a time (the 32-bit intermediate stays small)."""
    t = torch.empty(shape, dtype=dtype, device=dev)
    for part in t.view(-1).split(1 << 26):
        part.copy_(torch.randn(part.shape, generator=g, device=dev).mul_(scale))
    return t


def _outliers(t, g, dev):
    """Activations with a few channels far larger than the rest, and rows of different scale."""
    rows = t.view(-1, t.shape[-1])
    R, K = rows.shape
    rows *= torch.exp2(torch.randint(-6, 7, (R, 1), generator=g, device=dev)).to(t.dtype)
    rows[:, torch.randint(0, K, (max(1, K // 100),), generator=g, device=dev)] *= 16
    return t


def _checkpoint(w):
    """Weights as checkpoints hold them: e4m3 codes and, to each 128 x 128, the 32-bit scale
    (largest magnitude) / 448."""
    E, N, K = w.shape
    codes = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=w.device)
    scales = torch.empty((E, -(-N // 128), -(-K // 128)), dtype=torch.float32, device=w.device)
    for e in range(E):
        scales[e] = _block_max(w[e].float(), 128).clamp(min=1e-30) / 448
        codes[e] = (w[e].float() / _spread(scales[e], 128, N, K)).clamp(-448, 448).to(codes.dtype)
    return codes, scales


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)
    s = {"case": c}
    kind, dt = c["kind"], DTYPES[c["dtype"]]
    if kind == "quantize":
        shape = (c["N"], c["K"]) if c["E"] == 0 else (c["E"], c["N"], c["K"])
        s["x"] = _outliers(_randn(shape, dt, g, dev), g, dev)
    elif kind in ("product", "train"):
        E, K, N, R = c["E"], c["K"], c["N"], c["tokens"] * c["k"]
        s["counts"] = _counts(c, g, dev)
        s["sizes"] = s["counts"].tolist()
        s["x"] = _outliers(_randn((R, K), dt, g, dev), g, dev)
        w = _randn((E, N, K), dt, g, dev, K ** -0.5)
        if kind == "train":
            s["w"] = w
            s["dy"] = _randn((R, N), dt, g, dev)
        else:
            bdt = torch.float16 if dt == torch.float16 else torch.float32
            s["bias"] = _randn((E, N), bdt, g, dev) if c["bias"] else None
            s["codes"], s["scales"] = _checkpoint(w)
    else:
        T, E = c["tokens"], c["E"]
        l = _randn((T, E), torch.float32, g, dev, 1.5) + torch.randn(E, generator=g, device=dev)
        if E >= 8:
            l[:, torch.randint(0, E, (1,), generator=g, device=dev)] = -math.inf  # closed expert
        hidden = torch.rand((T, E), generator=g, device=dev) < 0.02
        l = l.masked_fill(hidden, torch.finfo(dt).min)
        padding = torch.rand((T, 1), generator=g, device=dev) < 0.03              # no experts
        s["logits"] = l.masked_fill(padding, -math.inf).to(dt)
        # a bias that was moved by steps of 0.001: several experts have the same
        step = 0.001 if c["score"] == "sigmoid" else 0.0001
        s["bias"] = torch.randint(-60, 61, (E,), generator=g, device=dev) * step if c["bias"] else None
        if c["grad"]:
            s["dw"] = _randn((T, c["k"]), torch.float32, g, dev)
    if own:
        s["calls"] = _calls(s)
    return s


# ---------------------------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------------------------

def _calls(s):
    """The calls of one pass, prepared once on the state's buffers."""
    import bmm_reducescatter_alltoall_gb300 as bra
    c, kind = s["case"], s["case"]["kind"]
    if kind == "quantize":
        q = bra.fp8_quantize_plan(s["x"], format=FORMATS[c["format"]])
        return [q, bra.fp8_dequantize_plan(q.result, s["x"].dtype)]
    if kind == "product":
        E, N, K = s["codes"].shape
        padded = torch.zeros((E, N, -(-K // 16) * 16), dtype=torch.uint8, device="cuda")
        padded[:, :, :K] = s["codes"].view(torch.uint8)           # rows have a 16-byte pitch
        w = bra.Fp8Tensor(padded.view(torch.float8_e4m3fn), s["scales"], (E, N, K))
        q = bra.fp8_quantize_plan(s["x"], s["counts"])
        return [q, bra.fp8_grouped_matmul_plan(q.result, w, s["counts"], bias=s["bias"],
                                               dtype=s["x"].dtype)]
    if kind == "train":
        w = bra.fp8_quantize_plan(s["w"])
        x = bra.fp8_quantize_plan(s["x"], s["counts"])
        dy = bra.fp8_quantize_plan(s["dy"], s["counts"], format=FORMATS[c["dy"]])
        return [w, x, bra.fp8_grouped_matmul_plan(x.result, w.result, s["counts"],
                                                  dtype=s["x"].dtype),
                dy, bra.fp8_grouped_matmul_grad_plan(dy.result, w.result, s["counts"],
                                                     dtype=s["x"].dtype)]
    r = bra.moe_route_plan(s["logits"], c["k"], renormalize=c["renorm"], score=c["score"],
                           bias=s["bias"], groups=c["groups"], top_groups=c["top_groups"],
                           group_best=c["group_best"], scale=c["scale"])
    if not c["grad"]:
        return [r]
    return [r, bra.moe_route_grad_plan(s["dw"], s["logits"], r.result["ids"], r.result["weights"],
                                       renormalize=c["renorm"], score=c["score"], scale=c["scale"])]


def _run_own(s):
    kind = s["case"]["kind"]
    got = [call.run() for call in s["calls"]]
    if kind == "quantize":
        return {"values": got[1]}
    if kind == "product":
        return {"y": got[1]}
    if kind == "train":
        return {"y": got[2], "dx": got[4]}
    out = {n: got[0][n] for n in ("ids", "weights", "counts", "slots", "tokens")}
    if len(got) > 1:
        out["dlogits"] = got[1]
    return out


# ---------------------------------------------------------------------------------------------
# Plain form
# ---------------------------------------------------------------------------------------------

def _blocks(x, rows):
    """x (M, K) in blocks of `rows` x 128, padded with zeros: (M/rows, rows, K/128, 128)."""
    M, K = x.shape
    return torch.nn.functional.pad(x, (0, -K % 128, 0, -M % rows)).unflatten(1, (-1, 128)).unflatten(
        0, (-1, rows))


def _block_max(x, rows):
    return _blocks(x.abs(), rows).amax((1, 3))


def _spread(scales, rows, M, K):
    """A value to each element from one to each block."""
    return scales.repeat_interleave(rows, 0).repeat_interleave(128, 1)[:M, :K]


def _quantized(x, rows, fmt):
    """The values of x (M, K) that 8 bits and a power of two to each block hold, in 32 bits."""
    M, K = x.shape
    x = x.float()
    amax = _block_max(x, rows)
    m, e = torch.frexp(amax)
    e = e - 1 - (8 if fmt == "e4m3" else 15) + (2 * m > 1.75)     # amax <= 1.75 * 2^(8 or 15) * 2^e
    e = torch.where(amax > 0, e, -126).clamp(min=-126).to(torch.int32)
    up, down = ((127 + e) << 23).view(torch.float32), ((127 - e) << 23).view(torch.float32)
    ok = torch.isfinite(amax)
    up = torch.where(ok, up, math.nan)
    code = (x * _spread(down, rows, M, K)).to(FORMATS[fmt])
    return code.float() * _spread(up, rows, M, K)


def _plain_quantize(s):
    c, x = s["case"], s["x"]
    if c["E"] == 0:
        return {"values": _quantized(x, 1, c["format"]).to(x.dtype)}
    out = torch.empty_like(x)
    for e in range(c["E"]):
        out[e] = _quantized(x[e], 128, c["format"]).to(x.dtype)
    return {"values": out}


def _parts(sizes):
    """(expert, first row, past the last row) of every expert that has rows."""
    at = [0]
    for n in sizes:
        at.append(at[-1] + n)
    return [(e, at[e], at[e + 1]) for e in range(len(sizes)) if sizes[e]]


def _plain_product(s):
    c, x = s["case"], s["x"]
    y = torch.empty((x.shape[0], c["N"]), dtype=x.dtype, device=x.device)
    xq = _quantized(x, 1, "e4m3")
    for e, a, b in _parts(s["sizes"]):
        w = s["codes"][e].float() * _spread(s["scales"][e], 128, c["N"], c["K"])
        z = torch.matmul(xq[a:b], w.t())
        y[a:b] = z if s["bias"] is None else z + s["bias"][e].float()
    return {"y": y}


def _plain_train(s):
    c, x = s["case"], s["x"]
    y = torch.empty((x.shape[0], c["N"]), dtype=x.dtype, device=x.device)
    dx = torch.empty_like(x)
    xq, dq = _quantized(x, 1, "e4m3"), _quantized(s["dy"], 1, c["dy"])
    for e, a, b in _parts(s["sizes"]):
        w = _quantized(s["w"][e], 128, "e4m3")
        y[a:b] = torch.matmul(xq[a:b], w.t())
        dx[a:b] = torch.matmul(dq[a:b], w)
    return {"y": y, "dx": dx}


def _scores(l, open_, score):
    """Scores of the open experts, 0 for the others, in l's precision."""
    if score == "sigmoid":
        return torch.where(open_, 1.0 / (1.0 + torch.exp(-l)), 0.0)
    some = open_.any(1, keepdim=True)
    peak = torch.where(some, l.amax(1, keepdim=True), 0.0)
    p = torch.where(open_, torch.exp(l - peak), 0.0)
    return p / p.sum(1, keepdim=True).clamp(min=1e-30)


def _plain_route(s):
    c, k, G = s["case"], s["case"]["k"], s["case"]["groups"]
    l = s["logits"].float().clamp(max=LARGEST)
    T, E = l.shape
    open_ = l > -math.inf
    # the choice, in 64 bits: by score and bias, or (no bias) by the logits, which order alike
    by = l.double()
    score = _scores(by, open_, c["score"])
    rank = by if s["bias"] is None else torch.where(open_, score + s["bias"].double(), -math.inf)
    if c["top_groups"] < G:
        grouped = rank.view(T, G, E // G)
        if c["group_best"] == 1:
            group = grouped.amax(2)
        else:
            of = grouped if s["bias"] is not None else torch.where(
                open_, score, -math.inf).view(T, G, E // G)
            best = torch.sort(of, dim=2, descending=True).values[:, :, :2]
            group = torch.where(best > -math.inf, best, 0.0).sum(2)
            group = torch.where(best[:, :, 0] > -math.inf, group, -math.inf)
        order = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, order, True)
        rank = torch.where(kept.repeat_interleave(E // G, 1), rank, -math.inf)
    top, ids = torch.sort(rank, dim=1, descending=True, stable=True)
    ids, has = ids[:, :k], top[:, :k] > -math.inf
    del by, score, rank, top
    # the weights, in 32
    p = _scores(l, open_, c["score"])
    at = l.gather(1, ids)
    if c["score"] == "sigmoid":
        w = torch.where(has, p.gather(1, ids), 0.0)
        if c["renorm"]:
            w = w / (w.sum(1, keepdim=True) + 1e-20)
    elif c["renorm"]:
        peak = torch.where(has, at, -math.inf).amax(1, keepdim=True)
        w = torch.where(has, torch.exp(at - torch.where(has[:, :1], peak, 0.0)), 0.0)
        w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    else:
        w = torch.where(has, p.gather(1, ids), 0.0)
    group = torch.where(has, ids, E).reshape(-1)
    order = torch.sort(group, stable=True).indices
    counts = torch.bincount(group, minlength=E + 1)[:E]
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device=l.device)
    used = torch.arange(T * k, device=l.device) < counts.sum()
    out = {"ids": torch.where(has, ids, -1).to(torch.int32), "weights": w * c["scale"],
           "counts": counts, "slots": torch.where(has, place.view(T, k), -1).to(torch.int32),
           "tokens": torch.where(used, order // k, -1).to(torch.int32)}
    if c["grad"]:
        g = torch.where(has, s["dw"], 0.0)
        mean = (w * g).sum(1, keepdim=True)
        if c["score"] == "sigmoid":
            d = w * (g - (mean if c["renorm"] else 0.0)) / (1.0 + torch.exp(at))   # 1 - sigmoid
            d = torch.zeros_like(l).scatter_add(1, ids, torch.where(has, d, 0.0))
        elif c["renorm"]:
            d = torch.zeros_like(l).scatter_add(1, ids, w * (g - mean))
        else:
            d = p * (torch.zeros_like(l).scatter_add(1, ids, g) - mean)
        out["dlogits"] = (d * c["scale"]).to(s["logits"].dtype)
    return out


_PLAIN = {"quantize": _plain_quantize, "product": _plain_product, "train": _plain_train,
          "route": _plain_route}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["kind"]](state)


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _pow2(n):
    """2^n for whole n in double, by its exponent field."""
    return ((n.clamp(-1000, 1000).to(torch.int64) + 1023) << 52).view(torch.float64)


def _floor_log2(v):
    """The exponent of the power of two at or below v > 0 (the logarithm is rounded: corrected)."""
    f = torch.floor(torch.log2(v.clamp(min=1e-300)))
    f = f + (_pow2(f + 1) <= v).double()
    return f - (_pow2(f) > v).double()


def _exact_fp8(x, fmt, rows):
    """Each block's smallest power of two at which its values stay within the format, and the
    nearest multiple of the format's step (a tie goes to the even one), 16 Mi at a time."""
    digits, low, most = (3, -6, 448.0) if fmt == "e4m3" else (2, -14, 57344.0)
    M, K = x.shape
    out = torch.empty((M, K), dtype=torch.float64, device=x.device)
    step = max(rows, (1 << 24) // K // rows * rows)
    for a in range(0, M, step):
        v = x[a:a + step].double()
        m, n = v.shape[0], -(-K // 128)
        full = torch.zeros((-(-m // rows) * rows, n * 128), dtype=torch.float64, device=x.device)
        full[:m, :K] = v
        b = full.view(-1, rows, n, 128)
        big = torch.einsum("arnc->anrc", b).abs().flatten(2).max(2).values[:, None, :, None]
        f = _floor_log2(big / most)
        f = torch.where(_pow2(f) * most < big, f + 1, f)
        f = torch.where(big > 0, f, torch.full_like(f, -126.0)).clamp(min=-126)
        u = b / _pow2(f)
        unit = _pow2(_floor_log2(u.abs()).clamp(min=low) - digits)
        q = torch.round(u / unit) * unit * _pow2(f)                  # round: half to even
        out[a:a + step] = q.reshape(full.shape)[:m, :K]
    return out


def _exact_products(s):
    c = s["case"]
    K, N, E = c["K"], c["N"], c["E"]
    owner = torch.repeat_interleave(torch.arange(E, device="cuda"), s["counts"])
    x = _exact_fp8(s["x"], "e4m3", 1)
    y = torch.zeros((x.shape[0], N), dtype=torch.float64, device="cuda")
    out = {"y": y}
    if c["kind"] == "train":
        d = _exact_fp8(s["dy"], c["dy"], 1)
        out["dx"] = torch.zeros((x.shape[0], K), dtype=torch.float64, device="cuda")
    n_of, k_of = torch.arange(N, device="cuda") // 128, torch.arange(K, device="cuda") // 128
    for e in range(E):
        rows = (owner == e).nonzero().squeeze(1)
        if rows.numel() == 0:
            continue
        if c["kind"] == "train":
            w = _exact_fp8(s["w"][e], "e4m3", 128)
            out["dx"][rows] = torch.einsum("rn,nk->rk", d[rows], w)
        else:
            w = s["codes"][e].float().double() * s["scales"][e].double()[n_of][:, k_of]
        y[rows] = torch.einsum("rk,nk->rn", x[rows], w)
        if c["kind"] == "product" and s["bias"] is not None:
            y[rows] += s["bias"][e].double()
    return out


def _exact_route(s):
    c, k, G = s["case"], s["case"]["k"], s["case"]["groups"]
    l = torch.nan_to_num(s["logits"].double(), nan=-math.inf, posinf=LARGEST, neginf=-math.inf)
    T, E = l.shape
    shut = l == -math.inf
    none = shut.all(1, keepdim=True)
    if c["score"] == "sigmoid":
        p = torch.sigmoid(l)
    else:
        p = torch.nan_to_num(torch.softmax(l.masked_fill(none, 0.0), 1)) * ~none
    left = l.clone() if s["bias"] is None else (p + s["bias"].double()).masked_fill(shut, -math.inf)
    if c["top_groups"] < G:
        of = left.clone() if s["bias"] is not None or c["group_best"] == 1 else \
            p.masked_fill(shut, -math.inf)
        value = torch.zeros((T, G), dtype=torch.float64, device="cuda")
        for g in range(G):
            part = of[:, g * (E // G):(g + 1) * (E // G)].clone()
            first, at = part.max(1)
            value[:, g] = first
            if c["group_best"] == 2:
                second = part.scatter(1, at[:, None], -math.inf).max(1).values
                value[:, g] += second.masked_fill(second == -math.inf, 0.0)
        for g in range(G):
            better = (value > value[:, g:g + 1]).sum(1) + (value[:, :g] == value[:, g:g + 1]).sum(1)
            left[:, g * (E // G):(g + 1) * (E // G)].masked_fill_(
                (better >= c["top_groups"])[:, None], -math.inf)
    picks, has = [], []
    for _ in range(k):
        v = left.max(1, keepdim=True).values
        first = (left == v).to(torch.int8).argmax(1, keepdim=True)      # the lowest index of a tie
        picks.append(first)
        has.append(v > -math.inf)
        left.scatter_(1, first, -math.inf)
    ids, has = torch.cat(picks, 1), torch.cat(has, 1)
    at, w = l.gather(1, ids), p.gather(1, ids) * has
    if c["renorm"]:
        if c["score"] == "sigmoid":
            w = w / (torch.einsum("tk->t", w) + 1e-20)[:, None]
        else:
            w = torch.nan_to_num(torch.softmax(at.masked_fill(~has, -math.inf), 1))
    out = {"ids": None, "weights": w * c["scale"], "counts": None, "slots": None, "tokens": None}
    if c["grad"]:
        g = s["dw"].double() * has
        mean = torch.einsum("tk,tk->t", w, g)[:, None]
        if c["score"] == "sigmoid":
            d = w * torch.sigmoid(-at) * (g - mean if c["renorm"] else g)
            out["dlogits"] = torch.zeros_like(l).scatter_add_(1, ids, d.masked_fill(~has, 0.0))
        elif c["renorm"]:
            out["dlogits"] = torch.zeros_like(l).scatter_add_(1, ids, w * g - w * mean)
        else:
            gi = torch.zeros_like(l).scatter_add_(1, ids, g)
            out["dlogits"] = p * gi - p * mean
        out["dlogits"] *= c["scale"]
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
        x, c = s["x"], s["case"]
        if c["E"] == 0:
            return {"values": _exact_fp8(x, c["format"], 1)}
        return {"values": torch.stack([_exact_fp8(x[e], c["format"], 128) for e in range(c["E"])])}
    if kind == "route":
        return _exact_route(s)
    return _exact_products(s)
