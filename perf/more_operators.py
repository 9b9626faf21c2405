"""Measured cases of score routing and of the experts' products in block-scaled fp8.

Three families: routing by softmax or sigmoid scores with a balance bias, groups and
renormalised weights, and its gradient (`moe_route_scores`, `moe_route_scores_bwd`);
E4M3 codes with one fp32 scale per 128 elements of a row, of a column or per 128 x 128
tile (`moe_quantize_fp8`, `moe_quantize_fp8_tiles`); the experts' products on such
operands, forward, with respect to the rows and with respect to the weights
(`moe_product_fp8`, `moe_product_fp8_dx`, `moe_product_fp8_dw`).  With `own` false `run`
computes them with elementary torch operations in 32 bits (the order of the experts in
64, where two scores lie next to each other); with `own` true it makes the library's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
BLOCK = 128


def listed():
    return [
        # a decode batch: sigmoid scores with a balance bias, the best 4 of 8 groups; latency
        dict(name="route decode groups", kind="route", T=128, E=256, R=8, dtype="fp32",
             score="sigmoid", bias=True, groups=8, top_groups=4, group_keys=2, renormalise=True,
             scale=2.5, closed=0.0),
        # a long prefill over many experts, no groups
        dict(name="route prefill", kind="route", T=65536, E=384, R=8, dtype="fp32",
             score="sigmoid", bias=True, groups=1, top_groups=1, group_keys=1, renormalise=True,
             scale=2.0, closed=0.0),
        # gradient at the training shape, softmax over all experts: every logit gets one
        dict(name="route grad train", kind="route_grad", T=16384, E=128, R=8, dtype="fp32",
             score="softmax", bias=False, groups=1, top_groups=1, group_keys=1,
             renormalise=False, scale=1.0, closed=0.0),
        # odd sizes, bf16 logits, renormalised sigmoid scores, some experts closed
        dict(name="route grad odd bf16", kind="route_grad", T=4099, E=60, R=3, dtype="bf16",
             score="sigmoid", bias=True, groups=1, top_groups=1, group_keys=1, renormalise=True,
             scale=1.0, closed=0.1),
        # sorted rows of a training batch: codes by row for the product, by column for the
        # weights' gradient, in one pass
        dict(name="quantize train rows columns", kind="quantize", N=131072, K=4096, dtype="bf16",
             form="both"),
        # the weights of a mid-sized layer's experts, once a step
        dict(name="quantize mid weights", kind="quantize", E=64, n=1408, K=2048, dtype="bf16",
             form="tile"),
        # a decode batch: 1024 rows over 256 experts, bound by the weights
        dict(name="product decode", kind="product", T=128, R=8, E=256, n=2048, K=7168, align=1,
             dtype="bf16"),
        # gate or up projection of a training batch, segments padded to tiles: the largest
        dict(name="product train", kind="product", T=16384, R=8, E=128, n=1536, K=4096, align=128,
             dtype="bf16"),
        # gradient with respect to a mid-sized layer's rows
        dict(name="dx mid", kind="product_dx", T=4096, R=6, E=64, n=1408, K=2048, align=1,
             dtype="bf16"),
        # one plain matrix product's gradient, odd sizes, fp32 result
        dict(name="dx one odd fp32", kind="product_dx", T=1001, R=1, E=1, n=2064, K=1040, align=1,
             dtype="fp32"),
        # gradient with respect to the training batch's weights, fp32
        dict(name="dw train", kind="product_dw", T=16384, R=8, E=128, n=1536, K=4096, align=128,
             dtype="fp32", accumulate=False),
        # added to the gradient of an earlier part of the batch, odd sizes
        dict(name="dw accumulate odd", kind="product_dw", T=1237, R=4, E=12, n=1040, K=2064,
             align=128, dtype="fp32", accumulate=True),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["route", "route_grad", "quantize", "quantize", "product", "product",
                       "product_dx", "product_dw"])
    if kind in ("route", "route_grad"):
        groups = rng.choice([1, 1, 4, 8])
        E = groups * log_int(rng, 2, 384 // groups)
        top = 1 if groups == 1 else rng.randint(1, groups)
        R = min(rng.choice([1, 2, 3, 4, 6, 8, 8]), top * (E // groups))
        return dict(kind=kind, T=log_int(rng, 1, 65536), E=E, R=R,
                    dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                    score=rng.choice(["softmax", "sigmoid", "sigmoid"]),
                    bias=rng.random() < 0.6, groups=groups, top_groups=top,
                    group_keys=rng.choice([1, 2]) if groups > 1 else 1,
                    renormalise=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                    closed=rng.choice([0.0, 0.0, 0.1]))
    K = 16 * log_int(rng, 4, 512)
    if kind == "quantize":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        form = rng.choice(["row", "col", "both", "tile"])
        most = 400_000_000
        if form == "tile":
            n = 16 * log_int(rng, 4, 256)
            E = log_int(rng, 1, max(1, min(256, most // (n * K))))
            return dict(kind=kind, E=E, n=n, K=K, dtype=dtype, form=form)
        return dict(kind=kind, N=log_int(rng, 1, most // K), K=K, dtype=dtype, form=form)
    n = 16 * log_int(rng, 4, 256)
    E = log_int(rng, 1, max(1, min(256, 1_000_000_000 // (n * K))))
    R = min(E, rng.choice([1, 2, 4, 8]))
    T = log_int(rng, 1, max(1, min(16384, 500_000_000_000 // (R * n * K))))
    align = 128 if kind == "product_dw" else rng.choice([1, 1, 128])
    c = dict(kind=kind, T=T, R=R, E=E, n=n, K=K, align=align,
             dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if kind == "product_dw":
        c["dtype"] = rng.choice(["fp32", "bf16"])
        c["accumulate"] = rng.random() < 0.3
    return c


# ---------------------------------------------------------------- inputs
def blocks(n):
    return -(-n // BLOCK)


def plain_codes(x, form):
    """E4M3 codes and fp32 scales (largest magnitude of a block / 448) of a matrix or a stack of
    matrices: blocks of 128 elements of a row, of 128 of a column, or tiles of 128 x 128."""
    n, K = x.shape[-2:]
    bn, bk = (1 if form == "row" else BLOCK), (1 if form == "col" else BLOCK)
    full = torch.zeros(x.shape[:-2] + (-(-n // bn) * bn, -(-K // bk) * bk), device=x.device)
    full[..., :n, :K] = x.float()
    full = full.view(x.shape[:-2] + (full.shape[-2] // bn, bn, full.shape[-1] // bk, bk))
    scale = torch.nan_to_num(full.abs(), nan=0.0, posinf=math.inf).amax((-3, -1)) / E4M3_MAX
    part = scale[..., :, None, :, None]
    q = torch.where(part > 0, full / part, torch.where(full.isnan(), full, 0.0))
    codes = q.clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3)
    codes = codes.view(x.shape[:-2] + (codes.shape[-4] * bn, codes.shape[-2] * bk))
    return codes[..., :n, :K].contiguous(), scale


def made_codes(shape, scale, form, g, zero_from=None):
    """Codes and scales of normal numbers, made in parts; rows from `zero_from` on are zeros."""
    n, K = shape[-2:]
    unit = BLOCK if len(shape) == 2 else 1
    per = max(1, 2 ** 27 // (unit * K if len(shape) == 2 else n * K)) * unit
    codes, scales = [], []
    for at in range(0, shape[0], per):
        count = min(per, shape[0] - at)
        part = torch.randn((count,) + tuple(shape[1:]), device="cuda", generator=g)
        if len(shape) == 2:                         # rows of unlike magnitude
            size = torch.rand(count, 1, device="cuda", generator=g).mul_(2.0).sub_(1.0).exp2_()
            part = part * size
        part = part.mul_(scale).bfloat16()
        if zero_from is not None and at + count > zero_from:
            part[max(0, zero_from - at):] = 0.0
        c, s = plain_codes(part, form)
        codes.append(c)
        scales.append(s)
    return torch.cat(codes), torch.cat(scales)


def rows_bound(T, R, E, align):
    """Rows that hold every plan of this shape."""
    n = T * R
    return (n + min(E, n) * (align - 1)) // align * align


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]
    s = {"case": case}
    dev = dict(device="cuda", generator=g)
    if kind in ("route", "route_grad"):
        T, E, R = case["T"], case["E"], case["R"]
        liking = torch.randn(E, **dev) * 0.5                    # some experts are hotter
        logits = (torch.randn(T, E, **dev) + liking).to(DTYPES[case["dtype"]])
        if case["closed"]:
            logits.masked_fill_(torch.rand(E, **dev) < case["closed"], -math.inf)
        s["logits"] = logits
        s["bias"] = torch.randn(E, **dev).mul_(0.05) if case["bias"] else None
        if kind == "route_grad":
            s["idx"] = plain_choice(s)
            s["dw"] = torch.randn(T, R, **dev)
    elif kind == "quantize":
        shape = (case["E"], case["n"]) if case["form"] == "tile" else (case["N"],)
        x = torch.empty(shape + (case["K"],), dtype=DTYPES[case["dtype"]], device="cuda")
        for part in x.view(-1, case["K"]).split(max(1, 2 ** 27 // case["K"])):
            size = torch.rand(part.shape[0], 1, **dev).mul_(2.0).sub_(1.0).exp2_()
            part.copy_(torch.randn(part.shape, **dev).mul_(size))
        s["x"] = x
    else:
        T, R, E, n, K = (case[k] for k in ("T", "R", "E", "n", "K"))
        liking = torch.randn(E, **dev) * 0.5
        u = torch.rand(T, E, **dev).clamp_(1e-20, 1 - 1e-7)
        idx = torch.topk(liking - torch.log(-torch.log(u)), R, dim=1)[1]
        counts = torch.bincount(idx.reshape(-1), minlength=E)
        align = case["align"]
        ends = ((counts + align - 1) // align * align).cumsum(0)
        s["offsets"] = torch.cat([ends.new_zeros(1), ends]).int()
        s["ends"] = [0] + ends.tolist()                         # the plain form's copy
        N = rows_bound(T, R, E, align)
        form = "col" if kind == "product_dw" else "row"
        if kind != "product_dw":
            s["w"], s["ws"] = made_codes((E, n, K), 0.02, "tile", g)
        if kind != "product":
            s["dy"], s["dys"] = made_codes((N, n), 1e-3, form, g, zero_from=s["ends"][-1])
        if kind != "product_dx":
            s["x"], s["xs"] = made_codes((N, K), 1.0, form, g, zero_from=s["ends"][-1])
        if kind == "product_dw" and case["accumulate"]:
            s["dw"] = torch.randn(E, n, K, **dev).mul_(1e-2).to(DTYPES[case["dtype"]])
    if own:
        buffers(s)
    return s


def buffers(s):
    """What a program that calls the library keeps: output buffers, workspaces, the router."""
    from expert_moe_route_gb300 import binding as B
    case = s["case"]
    kind = case["kind"]
    dev = dict(device="cuda")
    if kind in ("route", "route_grad"):
        T, E, R = case["T"], case["E"], case["R"]
        s["router"] = B.Router(score=case["score"], groups=case["groups"],
                               top_groups=case["top_groups"], group_keys=case["group_keys"],
                               renormalise=case["renormalise"], scale=case["scale"])
        if kind == "route":
            s["idx"] = torch.empty((T, R), dtype=torch.int32, **dev)
            s["topk_w"] = torch.empty((T, R), dtype=torch.float32, **dev)
        else:
            s["dlogits"] = torch.empty_like(s["logits"])
    elif kind == "quantize":
        x = s["x"]
        n, K = x.shape[-2:]
        form = case["form"]
        if form == "tile":
            s["codes"] = torch.empty(x.shape, dtype=E4M3, **dev)
            s["scales"] = torch.empty((x.shape[0], blocks(n), blocks(K)), **dev)
        if form in ("row", "both"):
            s["codes"] = torch.empty(x.shape, dtype=E4M3, **dev)
            s["scales"] = torch.empty((n, blocks(K)), **dev)
        if form in ("col", "both"):
            s["col_codes"] = torch.empty(x.shape, dtype=E4M3, **dev)
            s["col_scales"] = torch.empty((blocks(n), K), **dev)
    else:
        E, n, K = case["E"], case["n"], case["K"]
        N = (s["x"] if kind != "product_dx" else s["dy"]).shape[0]
        dtype = DTYPES[case["dtype"]]
        if kind == "product_dw":
            if not case["accumulate"]:
                s["dw"] = torch.empty((E, n, K), dtype=dtype, **dev)
        else:       # rows behind the last segment are left as they are
            s["out"] = torch.zeros((N, n if kind == "product" else K), dtype=dtype, **dev)
        s["space"] = B.workspace(B.product_fp8_ws_bytes(N, n, K, E))


# ---------------------------------------------------------------- one pass
def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    from expert_moe_route_gb300 import binding as B
    case = s["case"]
    kind = case["kind"]
    if kind == "route":
        B.moe_route_scores(s["logits"], s["router"], s["idx"], s["topk_w"], bias=s["bias"])
        return {"idx": s["idx"], "w": s["topk_w"]}
    if kind == "route_grad":
        B.moe_route_scores_bwd(s["logits"], s["router"], s["idx"], s["dw"], s["dlogits"])
        return {"dlogits": s["dlogits"]}
    if kind == "quantize":
        form = case["form"]
        if form == "tile":
            B.moe_quantize_fp8_tiles(s["x"], s["codes"], s["scales"])
        else:
            B.moe_quantize_fp8(s["x"], s.get("codes"), s.get("scales"), s.get("col_codes"),
                               s.get("col_scales"))
        return {k: s[k] for k in ("codes", "scales", "col_codes", "col_scales") if k in s}
    if kind == "product":
        B.moe_product_fp8(s["x"], s["xs"], s["w"], s["ws"], s["out"], s["space"],
                          offsets=s["offsets"])
        return {"out": s["out"]}
    if kind == "product_dx":
        B.moe_product_fp8_dx(s["dy"], s["dys"], s["w"], s["ws"], s["out"], s["space"],
                             offsets=s["offsets"])
        return {"dx": s["out"]}
    B.moe_product_fp8_dw(s["dy"], s["dys"], s["x"], s["xs"], s["dw"], s["space"],
                         offsets=s["offsets"], accumulate=case["accumulate"])
    return {"dw": s["dw"]}


def plain_scores(x, score):
    """The experts' scores; a closed expert (logit -inf) has none."""
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    z = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e30))
    return z / z.sum(1, keepdim=True).clamp(min=1e-30)


def plain_choice(s):
    """The chosen experts [T, R], best first, ties to the lower one; -1 where none is left.  In 64
    bits: scores next to each other decide."""
    case = s["case"]
    E, G, R = case["E"], case["groups"], case["R"]
    x = s["logits"].double()
    order = x
    if case["bias"] or case["group_keys"] == 2:
        score = plain_scores(x, case["score"])
        key = score + s["bias"].double() if case["bias"] else score
        key = torch.where(x == -math.inf, -math.inf, key)
        if case["bias"]:
            order = key
    else:
        key = x
    if G > 1:
        best = torch.sort(key.view(-1, G, E // G), dim=2, descending=True)[0]
        worth = best[..., 0]
        if case["group_keys"] == 2:
            second = best[..., 1] if E // G > 1 else torch.full_like(worth, -math.inf)
            worth = worth + second
        place = torch.sort(worth, dim=1, descending=True, stable=True)[1][:, :case["top_groups"]]
        open_ = torch.zeros_like(worth, dtype=torch.bool).scatter_(1, place, True)
        order = torch.where(open_.repeat_interleave(E // G, dim=1), order, -math.inf)
    value, idx = torch.sort(order, dim=1, descending=True, stable=True)
    return torch.where(value[:, :R] == -math.inf, -1, idx[:, :R]).int()


def plain_weights(s, idx):
    """Scores of the chosen experts in 32 bits, and the weights made of them."""
    case = s["case"]
    x = s["logits"].float()
    here = idx >= 0
    score = plain_scores(x, case["score"])
    got = torch.where(here, torch.gather(score, 1, idx.long().clamp(min=0)), 0.0)
    if not case["renormalise"]:
        return score, got, got * case["scale"]
    total = got.sum(1, keepdim=True)
    return score, got, torch.where(total > 0, got / total, 0.0) * case["scale"]


def plain_dequant(codes, scales, form):
    n, K = codes.shape[-2:]
    if form != "row":
        scales = scales.repeat_interleave(BLOCK, dim=-2)[..., :n, :]
    if form != "col":
        scales = scales.repeat_interleave(BLOCK, dim=-1)[..., :K]
    return codes.float() * scales


def run_plain(s):
    case = s["case"]
    kind = case["kind"]
    if kind == "route":
        idx = plain_choice(s)
        return {"idx": idx, "w": plain_weights(s, idx)[2]}
    if kind == "route_grad":
        idx, here = s["idx"].long().clamp(min=0), s["idx"] >= 0
        score, got, w = plain_weights(s, s["idx"])
        dw = torch.where(here, s["dw"], 0.0) * case["scale"]
        if case["renormalise"]:
            total = got.sum(1, keepdim=True)
            share = w / case["scale"]
            dw = torch.where(total > 0, (dw - (dw * share).sum(1, keepdim=True)) / total, 0.0)
        ds = torch.zeros_like(score).scatter_add_(1, idx, torch.where(here, dw, 0.0))
        if case["score"] == "sigmoid":
            dl = ds * score / (1.0 + torch.exp(s["logits"].float()))
        else:
            dl = score * (ds - (ds * score).sum(1, keepdim=True))
        return {"dlogits": dl.to(DTYPES[case["dtype"]])}
    if kind == "quantize":
        form = case["form"]
        out = {}
        if form != "col":
            out["codes"], out["scales"] = plain_codes(s["x"], "tile" if form == "tile" else "row")
        if form in ("col", "both"):
            out["col_codes"], out["col_scales"] = plain_codes(s["x"], "col")
        return out
    E, n, K = case["E"], case["n"], case["K"]
    dtype = DTYPES[case["dtype"]]
    ends = s["ends"]
    if kind == "product_dw":
        fresh = None if case["accumulate"] else torch.zeros((E, n, K), dtype=dtype, device="cuda")
        for e in range(E):
            a, b = ends[e], ends[e + 1]
            if a == b:
                continue
            rows = slice(a // BLOCK, blocks(b))
            dy = plain_dequant(s["dy"][a:b], s["dys"][rows], "col")
            x = plain_dequant(s["x"][a:b], s["xs"][rows], "col")
            grad = dy.t() @ x
            if case["accumulate"]:
                s["dw"][e].copy_(s["dw"][e].float() + grad)
            else:
                fresh[e] = grad
        return {"dw": s["dw"] if case["accumulate"] else fresh}
    rows, scales = (s["x"], s["xs"]) if kind == "product" else (s["dy"], s["dys"])
    out = torch.zeros((rows.shape[0], n if kind == "product" else K), dtype=dtype, device="cuda")
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        w = plain_dequant(s["w"][e], s["ws"][e], "tile")
        x = plain_dequant(rows[a:b], scales[a:b], "row")
        out[a:b] = x @ (w.t() if kind == "product" else w)
    return {"out" if kind == "product" else "dx": out}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    kind = case["kind"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if kind in ("route", "route_grad"):
        T, E, R = case["T"], case["E"], case["R"]
        b = size[case["dtype"]]
        if kind == "route":
            return {"bytes": T * E * b + 4 * E * case["bias"] + 8 * T * R, "flops": 4 * T * E}
        dense = case["score"] == "softmax" and not case["renormalise"]
        return {"bytes": T * E * b + (T * E * b if dense else T * R * b) + 8 * T * R,
                "flops": (6 * T * E if dense else 0) + 8 * T * R}
    b = size[case["dtype"]]
    if kind == "quantize":
        K = case["K"]
        if case["form"] == "tile":
            E, n = case["E"], case["n"]
            return {"bytes": E * n * K * (b + 1) + 4 * E * blocks(n) * blocks(K),
                    "flops": 2 * E * n * K}
        N = case["N"]
        row, col = case["form"] in ("row", "both"), case["form"] in ("col", "both")
        return {"bytes": N * K * (b + row + col) + 4 * row * N * blocks(K) + 4 * col * blocks(N) * K,
                "flops": (row + col) * 2 * N * K}
    T, R, E, n, K = (case[k] for k in ("T", "R", "E", "n", "K"))
    rows = T * R
    used = E * (1.0 - (1.0 - R / E) ** T)       # experts with a row, were they equally liked
    flops = 2 * rows * n * K
    if kind == "product_dw":
        stored = E * n * K * b * (2 if case["accumulate"] else 1)
        return {"bytes": rows * (n + K) * (1 + 4 / BLOCK) + stored, "flops": flops}
    inner, outer = (K, n) if kind == "product" else (n, K)
    return {"bytes": rows * inner * (1 + 4 / BLOCK) + used * n * K + rows * outer * b + 4 * E,
            "flops": flops}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact_scores(x, score):
    if score == "sigmoid":
        return torch.sigmoid(x)
    return torch.softmax(x, 1)


def exact_choice(x, s):
    """By counting, for each expert, the ones before it."""
    case = s["case"]
    E, G, R = case["E"], case["groups"], case["R"]
    n = x.shape[0]
    key = exact_scores(x, case["score"])
    if case["bias"]:
        key = key + s["bias"].double()
    key = key.masked_fill(x == -math.inf, -math.inf)
    by = key if case["bias"] else x
    alive = x > -math.inf
    if G > 1:
        per = E // G
        top = torch.topk(key.view(n, G, per), min(per, case["group_keys"]), dim=2)[0].sum(2)
        if per < case["group_keys"]:
            top = torch.full_like(top, -math.inf)
        g = torch.arange(G, device=x.device)
        ahead = (top[:, None, :] > top[:, :, None]) | (
            (top[:, None, :] == top[:, :, None]) & (g[None, None, :] < g[None, :, None]))
        keep = ahead.sum(2) < case["top_groups"]
        alive = alive & keep[:, torch.arange(E, device=x.device) // per]
    by = torch.where(alive, by, -math.inf)
    e = torch.arange(E, device=x.device)
    ahead = (by[:, None, :] > by[:, :, None]) | (
        (by[:, None, :] == by[:, :, None]) & (e[None, None, :] < e[None, :, None]))
    rank = torch.where(alive, ahead.sum(2), E)
    idx = torch.full((n, R), -1, dtype=torch.long, device=x.device)
    at, expert = ((rank < R) & alive).nonzero(as_tuple=True)
    idx[at, rank[at, expert]] = expert
    return idx


def exact_weights(x, idx, case):
    here = idx >= 0
    chosen = torch.gather(exact_scores(x, case["score"]), 1, idx.clamp(min=0))
    chosen = torch.where(here, chosen, 0.0)
    if case["renormalise"]:
        chosen = chosen / chosen.sum(1, keepdim=True).clamp(min=1e-300)
    return chosen * case["scale"]


def exact_values(codes, scales, form, rows=slice(None), first=0):
    """The numbers that codes stand for; `first` is the place of the first row."""
    c = codes[rows].double()
    i = (torch.arange(c.shape[0], device=c.device) + first) // (1 if form == "row" else BLOCK)
    j = torch.arange(c.shape[1], device=c.device) // (1 if form == "col" else BLOCK)
    return c * scales.double()[i][:, j]


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("route", "route_grad"):
        T, E = case["T"], case["E"]
        parts = []
        for at in range(0, T, max(1, 2 ** 27 // (E * E))):
            x = s["logits"][at:at + max(1, 2 ** 27 // (E * E))].double()
            if kind == "route":
                parts.append(exact_weights(x, exact_choice(x, s), case))
                continue
            # the derivative of sum(w * dw), by automatic differentiation
            idx = s["idx"][at:at + x.shape[0]].long()
            dw = torch.where(idx >= 0, s["dw"][at:at + x.shape[0]].double(), 0.0)
            closed = x == -math.inf
            x = x.masked_fill(closed, -1e4).requires_grad_(True)
            (exact_weights(x, idx, case) * dw).sum().backward()
            parts.append(x.grad.masked_fill(closed, 0.0))
        if kind == "route":
            return {"idx": None, "w": torch.cat(parts)}
        return {"dlogits": torch.cat(parts)}
    if kind == "quantize":
        form = case["form"]
        x = s["x"] if form == "tile" else s["x"][None]
        n, K = x.shape[-2:]
        out = {}
        if form == "tile":
            top = x.new_zeros((x.shape[0], blocks(n), blocks(K)), dtype=torch.float64)
            for i in range(blocks(n)):
                for j in range(blocks(K)):
                    part = x[:, i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
                    top[:, i, j] = part.abs().amax((1, 2)).double()
            return {"codes": None, "scales": top / E4M3_MAX}
        if form in ("row", "both"):
            cols = [x[0][:, j * BLOCK:(j + 1) * BLOCK].abs().amax(1) for j in range(blocks(K))]
            out["codes"], out["scales"] = None, torch.stack(cols, 1).double() / E4M3_MAX
        if form in ("col", "both"):
            rows = [part.abs().amax(0) for part in x[0].split(BLOCK)]
            out["col_codes"], out["col_scales"] = None, torch.stack(rows).double() / E4M3_MAX
        return out
    E, n, K = case["E"], case["n"], case["K"]
    ends = s["offsets"].tolist()
    if kind == "product_dw":
        out = torch.zeros(E, n, K, dtype=torch.float64, device="cuda")
        if case["accumulate"]:
            out += s["dw"].double()
    else:
        rows = s["x" if kind == "product" else "dy"]
        out = torch.zeros(rows.shape[0], n if kind == "product" else K, dtype=torch.float64,
                          device="cuda")
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        if kind == "product_dw":
            out[e] += torch.einsum("in,ik->nk",
                                   exact_values(s["dy"], s["dys"], "col", slice(a, b), a),
                                   exact_values(s["x"], s["xs"], "col", slice(a, b), a))
            continue
        w = exact_values(s["w"][e], s["ws"][e], "tile")
        if kind == "product":
            x = exact_values(s["x"][a:b], s["xs"][a:b], "row")
            out[a:b] = torch.einsum("ik,nk->in", x, w)
        else:
            dy = exact_values(s["dy"][a:b], s["dys"][a:b], "row")
            out[a:b] = torch.einsum("in,nk->ik", dy, w)
    return {"out" if kind == "product" else "dw" if kind == "product_dw" else "dx": out}
