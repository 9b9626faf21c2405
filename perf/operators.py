"""Measured cases of the training-side operators around the MoE layer.

Three families: slots sorted by expert and back with the gate weights applied
(`moe_sort`, `moe_permute`, `moe_unpermute` and their gradients), the embedding
lookup and its gradient by sorted tokens (`moe_embed`, `moe_embed_bwd`), and the
optimiser step (`moe_grad_norm`, `moe_adamw_step`).  With `own` false `run`
computes them with elementary torch operations in 32 bits; with `own` true it
makes the library's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 256            # elements that share one scale of an 8-bit optimiser state
E4M3_MAX = 448.0
ADAMW = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, step=100, seed=20)
DECAY = 0.1            # weight decay of the matrices; tensors under 65536 elements get none
MAX_NORM = 1.0


def listed():
    layer = {"mid": "1*131072f 1*64f 3*184549376h", "tiny": "1*4096f 1*8f 3*4194304h"}
    return [
        # a decode batch of 128 tokens: plan and rows, segments padded to 16 rows; latency
        dict(name="sort decode", kind="sort", T=128, d=7168, E=256, R=8, dtype="bf16",
             weights=False, align=16, capacity=0, drop=0.0),
        # a training batch whose rows carry their gate weight into the experts, tiles of 128 rows
        dict(name="sort train weighted", kind="sort", T=16384, d=4096, E=128, R=8, dtype="bf16",
             weights=True, align=128, capacity=0, drop=0.0),
        # gradient of the weighted sort: some slots empty, at most 512 rows an expert
        dict(name="sort grad capacity", kind="sort_grad", T=4096, d=2048, E=64, R=6, dtype="bf16",
             weights=True, align=1, capacity=512, drop=0.05),
        # a long prefill brought back to token order: the largest case
        dict(name="back prefill", kind="back", T=65536, d=7168, E=256, R=8, dtype="bf16",
             weights=True, align=1, capacity=0, drop=0.0),
        # gradient of the weighted sum at the training shape
        dict(name="back grad train", kind="back_grad", T=16384, d=4096, E=128, R=8, dtype="bf16",
             weights=True, align=128, capacity=0, drop=0.0),
        # odd sizes in fp32, a third of the slots on other ranks' experts (empty here)
        dict(name="back grad odd fp32", kind="back_grad", T=1001, d=1001, E=60, R=3, dtype="fp32",
             weights=True, align=1, capacity=0, drop=0.33),
        # every parameter of a small layer, states in 32 bits, clipped: few megabytes, latency
        dict(name="adamw tiny layer", kind="adamw", sizes=layer["tiny"], states=32, master=False,
             grads="fp32", clip=True, packed=False),
        # every parameter of a mid-sized layer, states in 8 bits, clipped
        dict(name="adamw8 mid layer", kind="adamw", sizes=layer["mid"], states=8, master=False,
             grads="fp32", clip=True, packed=False),
        # each expert's matrices as tensors of their own, odd sizes, fp32 master copies, bf16 gradients
        dict(name="adamw master experts", kind="adamw", sizes="1*61440f 1*60f 180*1409025h",
             states=32, master=True, grads="bf16", clip=False, packed=False),
        # a prefill batch of token ids looked up in a bf16 table, scaled
        dict(name="embed prefill", kind="embed", n=32768, V=65536, d=4096, dtype="bf16",
             out="bf16", ids="int64", masked=0.0),
        # its gradient for a training batch: a whole fp32 table gradient
        dict(name="embed grad train", kind="embed_grad", n=16384, V=65536, d=4096, dtype="bf16",
             out="fp32", ids="int64", masked=0.0, accumulate=False),
        # gradient added into the one that is there, masked positions, an odd vocabulary
        dict(name="embed grad accumulate", kind="embed_grad", n=49999, V=32003, d=2048,
             dtype="bf16", out="fp32", ids="int32", masked=0.1, accumulate=True),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["sort", "sort_grad", "back", "back_grad", "adamw", "embed", "embed_grad"])
    if kind == "adamw":
        count = log_int(rng, 1, 120)
        most = 200_000_000 // count
        size = log_int(rng, 1000, most)
        bf16 = rng.random() < 0.7
        sizes = "%d*%d%s 1*%df" % (count, size, "h" if bf16 else "f", log_int(rng, 1, 70000))
        return dict(kind=kind, sizes=sizes, states=rng.choice([8, 32]),
                    master=bf16 and rng.random() < 0.4, grads=rng.choice(["fp32", "bf16"]),
                    clip=rng.random() < 0.5, packed=rng.random() < 0.2)
    d = 8 * log_int(rng, 8, 1024) if rng.random() < 0.75 else log_int(rng, 61, 4099)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if kind in ("embed", "embed_grad"):
        V = log_int(rng, 1000, 100_000)
        c = dict(kind=kind, n=log_int(rng, 1, 60_000), V=V, d=min(d, 400_000_000 // V), dtype=dtype,
                 out=rng.choice([dtype, "fp32"] if kind == "embed_grad" else [dtype]),
                 ids=rng.choice(["int32", "int64"]), masked=rng.choice([0.0, 0.2]))
        if kind == "embed_grad":
            c["accumulate"] = rng.random() < 0.4
        return c
    E = log_int(rng, 2, 512)
    R = min(E, rng.choice([1, 2, 3, 4, 6, 8, 8]))
    T = min(log_int(rng, 1, 65536), max(1, 1_500_000_000 // (R * d)))
    weights = kind in ("sort_grad", "back_grad") or rng.random() < 0.7
    capacity = rng.choice([0, 0, max(1, int(1.25 * T * R / E))])
    return dict(kind=kind, T=T, d=d, E=E, R=R, dtype=dtype, weights=weights,
                align=rng.choice([1, 1, 16, 128]), capacity=capacity,
                drop=rng.choice([0.0, 0.0, 0.25]))


# ---------------------------------------------------------------- inputs
def rows_bound(T, R, E, align, capacity):
    """Rows that hold every plan of this shape."""
    n = T * R
    most = (n + min(E, n) * (align - 1)) // align * align
    return min(most, E * (-(-capacity // align) * align)) if capacity > 0 else most


def plan(idx, E, align, capacity, N):
    """counts, offsets, row_slot, slot_row: each expert's slots in slot order, at most `capacity`
    of them, segments starting at multiples of `align`; -1 where a slot has no row or a row no slot."""
    flat = idx.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    key, order = torch.sort(key, stable=True)
    start = torch.searchsorted(key, torch.arange(E + 1, device=idx.device))
    kept = start[1:] - start[:-1]
    kept = kept.clamp(max=capacity) if capacity > 0 else kept
    padded = (kept + align - 1) // align * align
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    rank = torch.arange(n, device=idx.device) - start[key]
    has = (key < E) & (rank < torch.cat([kept, kept.new_zeros(1)])[key])
    row = torch.where(has, offsets[key] + rank, torch.full_like(key, -1))
    slot_row = torch.empty_like(row).scatter_(0, order, row)
    row_slot = row.new_full((N + 1,), -1).scatter_(0, torch.where(has, row, N), order)[:N]
    return kept.int(), offsets.int(), row_slot.int(), slot_row.int().reshape(idx.shape)


def flat_layout(sizes, packed):
    """[(numel, is bf16, offset in its flat buffer, first scale)] of the tensors that `sizes` names."""
    out, at, blocks = [], {True: 0, False: 0}, {True: 0, False: 0}
    for item in sizes.split():
        count, numel = item[:-1].split("*")
        half = item[-1] == "h"
        for _ in range(int(count)):
            out.append((int(numel), half, at[half], blocks[half]))
            at[half] += int(numel) if packed else -(-int(numel) // 128) * 128
            blocks[half] += -(-int(numel) // BLOCK)
    return out, at, blocks


def adamw_inputs(case, g):
    layout, total, blocks = flat_layout(case["sizes"], case["packed"])
    state = {"layout": layout, "flat": {}}
    for half in (True, False):
        n = total[half]
        if not n:
            continue
        dev = dict(device="cuda", generator=g)

        def normal(scale):
            return torch.randn(n, **dev).mul_(scale)

        quiet = (torch.rand(-(-n // 4096), **dev) < 0.05).repeat_interleave(4096)[:n]
        f = {}
        p = normal(0.02)
        f["p"] = p.bfloat16() if half else p
        if half and case["master"]:
            f["master"] = f["p"].float().add_(normal(1e-5))
        grad = normal(1e-3).masked_fill_(quiet, 0.0)    # experts without tokens
        f["g"] = grad.to(torch.bfloat16 if half and case["grads"] == "bf16" else torch.float32)
        if case["states"] == 32:
            f["m"] = normal(3e-4)
            f["v"] = normal(1e-3).square_()
        else:
            f["m"] = normal(112.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            f["v"] = normal(112.0).abs_().clamp_(2.0 ** -9, E4M3_MAX).to(torch.float8_e4m3fn)
            b = blocks[half]
            empty = torch.rand(b, **dev) < 0.02             # blocks that no step has reached
            f["m_scale"] = torch.rand(b, **dev).mul_(2e-6).add_(5e-7).masked_fill_(empty, 0.0)
            f["v_scale"] = torch.rand(b, **dev).mul_(6e-6).add_(2e-6).masked_fill_(empty, 0.0)
        state["flat"][half] = f
    state["norm"] = torch.zeros(4, device="cuda")
    return state


def views(state, k):
    """The k-th tensor's parts: views of the flat buffers."""
    n, half, at, first = state["layout"][k]
    f = state["flat"][half]
    out = {name: t[at:at + n] for name, t in f.items() if not name.endswith("scale")}
    for name in ("m_scale", "v_scale"):
        if name in f:
            out[name] = f[name][first:first + -(-n // BLOCK)]
    return out


def token_ids(case, g):
    """Ids whose frequency falls off as 1 / rank, some positions without a token."""
    u = torch.rand(case["n"], device="cuda", generator=g, dtype=torch.float64)
    ids = torch.exp(u * math.log(case["V"] + 1)).long().sub_(1).clamp_(0, case["V"] - 1)
    none = torch.rand(case["n"], device="cuda", generator=g) < case["masked"]
    ids = torch.where(none, torch.full_like(ids, -1), ids)
    return ids.to(torch.int32 if case["ids"] == "int32" else torch.int64)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]
    s = {"case": case}
    if kind == "adamw":
        s.update(adamw_inputs(case, g))
    elif kind in ("embed", "embed_grad"):
        n, V, d = case["n"], case["V"], case["d"]
        dtype = DTYPES[case["dtype"]]
        s["ids"] = token_ids(case, g)
        s["scale"] = math.sqrt(d)
        if kind == "embed":
            s["table"] = torch.randn(V, d, device="cuda", generator=g).mul_(0.02).to(dtype)
        else:
            s["dout"] = torch.randn(n, d, device="cuda", generator=g).to(dtype)
            if case["accumulate"]:
                s["dtable"] = torch.randn(V, d, device="cuda", generator=g).to(DTYPES[case["out"]])
    else:
        T, d, E, R = case["T"], case["d"], case["E"], case["R"]
        dtype = DTYPES[case["dtype"]]
        liking = torch.randn(E, device="cuda", generator=g)     # some experts are hotter
        u = torch.rand(T, E, device="cuda", generator=g).clamp_(1e-20, 1 - 1e-7)
        logits, idx = torch.topk(liking - torch.log(-torch.log(u)), R, dim=1)
        s["w"] = torch.softmax(logits, 1)
        drop = torch.rand(T, R, device="cuda", generator=g) < case["drop"]
        s["idx"] = torch.where(drop, torch.full_like(idx, -1), idx).int()
        s["N"] = N = rows_bound(T, R, E, case["align"], case["capacity"])
        if kind != "sort":
            s["counts"], s["offsets"], s["row_slot"], s["slot_row"] = plan(
                s["idx"], E, case["align"], case["capacity"], N)
        if kind in ("sort", "sort_grad"):
            s["x"] = torch.randn(T, d, device="cuda", generator=g).to(dtype)
        if kind == "back_grad":
            s["dy"] = torch.randn(T, d, device="cuda", generator=g).to(dtype)
        if kind != "sort":
            s["rows"] = torch.randn(N, d, device="cuda", generator=g, dtype=dtype)
    if own:
        buffers(s)
    return s


def buffers(s):
    """What a program that calls the library keeps: output buffers, workspaces, the optimiser's list."""
    from expert_moe_route_gb300 import binding as B
    case = s["case"]
    kind = case["kind"]
    dev = dict(device="cuda")
    if kind == "adamw":
        tensors = []
        for k, (n, half, _, _) in enumerate(s["layout"]):
            t = views(s, k)
            tensors.append(B.AdamWTensor(t["p"], t["g"], t["m"], t["v"], master=t.get("master"),
                                         m_scale=t.get("m_scale"), v_scale=t.get("v_scale"),
                                         weight_decay=DECAY if n >= 65536 else 0.0))
        s["list"] = B.AdamWList(tensors)
        s["ws"] = B.workspace(B.grad_norm_ws_bytes(s["list"]))
    elif kind == "embed":
        s["out"] = torch.empty((case["n"], case["d"]), dtype=DTYPES[case["out"]], **dev)
    elif kind == "embed_grad":
        if not case["accumulate"]:
            s["dtable"] = torch.empty((case["V"], case["d"]), dtype=DTYPES[case["out"]], **dev)
        s["ws"] = B.workspace(B.embed_bwd_ws_bytes(case["n"], case["V"], case["d"]))
    else:
        T, d, E, R = case["T"], case["d"], case["E"], case["R"]
        dtype = DTYPES[case["dtype"]]
        if kind == "sort":
            s["counts"] = torch.empty(E, dtype=torch.int32, **dev)
            s["offsets"] = torch.empty(E + 1, dtype=torch.int32, **dev)
            s["row_slot"] = torch.empty(s["N"], dtype=torch.int32, **dev)
            s["slot_row"] = torch.empty((T, R), dtype=torch.int32, **dev)
            s["ws"] = B.workspace(B.sort_ws_bytes(T, E, R))
        if kind in ("sort", "back_grad"):
            s["rows_out"] = torch.empty((s["N"], d), dtype=dtype, **dev)
        if kind in ("sort_grad", "back"):
            s["y"] = torch.empty((T, d), dtype=dtype, **dev)
        if kind in ("sort_grad", "back_grad"):
            s["dw"] = torch.empty((T, R), dtype=torch.float32, **dev)


# ---------------------------------------------------------------- one pass
def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    from expert_moe_route_gb300 import binding as B
    case = s["case"]
    kind = case["kind"]
    w = s["w"] if case.get("weights") else None
    if kind == "sort":
        B.moe_sort(s["idx"], case["E"], s["counts"], s["offsets"], s["row_slot"], s["slot_row"],
                   s["ws"], align=case["align"], capacity=case["capacity"])
        B.moe_permute(s["x"], w, s["row_slot"], s["slot_row"], s["rows_out"])
        return {"counts": s["counts"], "offsets": s["offsets"], "row_slot": s["row_slot"],
                "slot_row": s["slot_row"], "rows": s["rows_out"]}
    if kind == "sort_grad":
        B.moe_permute_bwd(s["rows"], s["slot_row"], w, s["x"], s["y"], s["dw"])
        return {"dx": s["y"], "dw": s["dw"]}
    if kind == "back":
        B.moe_unpermute(s["rows"], s["slot_row"], w, s["y"])
        return {"y": s["y"]}
    if kind == "back_grad":
        B.moe_unpermute_bwd(s["dy"], s["row_slot"], s["slot_row"], w, s["rows"], s["rows_out"],
                            s["dw"])
        return {"drows": s["rows_out"], "dw": s["dw"]}
    if kind == "embed":
        B.moe_embed(s["ids"], s["table"], s["out"], scale=s["scale"])
        return {"out": s["out"]}
    if kind == "embed_grad":
        B.moe_embed_bwd(s["dout"], s["ids"], s["dtable"], s["ws"], scale=s["scale"],
                        accumulate=case["accumulate"])
        return {"dtable": s["dtable"]}
    norm = None
    if case["clip"]:
        norm = s["norm"]
        B.moe_grad_norm(s["list"], MAX_NORM, norm, s["ws"])
    B.moe_adamw_step(s["list"], norm=norm, **ADAMW)
    return adamw_outputs(s)


def run_plain(s):
    case = s["case"]
    kind = case["kind"]
    if kind == "adamw":
        return plain_adamw(s)
    if kind == "embed":
        ids = s["ids"].long()
        here = (ids >= 0) & (ids < case["V"])
        rows = s["table"][torch.where(here, ids, 0)].float() * s["scale"]
        return {"out": torch.where(here[:, None], rows, 0.0).to(DTYPES[case["out"]])}
    if kind == "embed_grad":
        ids = s["ids"].long()
        key = torch.where((ids >= 0) & (ids < case["V"]), ids, case["V"])
        sums = torch.zeros(case["V"] + 1, case["d"], device="cuda")
        grad = sums.index_add_(0, key, s["dout"].float())[:-1] * s["scale"]
        if not case["accumulate"]:
            return {"dtable": grad.to(DTYPES[case["out"]])}
        return {"dtable": s["dtable"].copy_(s["dtable"].float() + grad)}
    T, d, R, N = case["T"], case["d"], case["R"], s["N"]
    dtype = DTYPES[case["dtype"]]
    w = s["w"] if case["weights"] else torch.ones_like(s["w"])
    if kind == "sort":
        counts, offsets, row_slot, slot_row = plan(s["idx"], case["E"], case["align"],
                                                   case["capacity"], N)
        slot = row_slot.long().clamp(min=0)
        rows = s["x"][slot // R].float() * w.reshape(-1)[slot][:, None]
        rows = torch.where((row_slot >= 0)[:, None], rows, 0.0).to(dtype)
        return {"counts": counts, "offsets": offsets, "row_slot": row_slot, "slot_row": slot_row,
                "rows": rows}
    here = s["slot_row"] >= 0
    at = s["slot_row"].long().clamp(min=0)
    if kind == "back_grad":
        slot = s["row_slot"].long().clamp(min=0)
        drows = s["dy"][slot // R].float() * w.reshape(-1)[slot][:, None]
        drows = torch.where((s["row_slot"] >= 0)[:, None], drows, 0.0).to(dtype)
        dw = (s["rows"][at].float() * s["dy"].float()[:, None]).sum(2)
        return {"drows": drows, "dw": torch.where(here, dw, 0.0)}
    rows = torch.where(here[..., None], s["rows"][at].float(), 0.0)     # [T, R, d]
    y = (rows * w[..., None]).sum(1).to(dtype)
    if kind == "back":
        return {"y": y}
    return {"dx": y, "dw": (rows * s["x"].float()[:, None]).sum(2)}


def adamw_outputs(s):
    """Parameters, master copies, states (8-bit ones as the numbers they hold, with their scales),
    the norm's record."""
    out = {}
    for half, f in s["flat"].items():
        out["bf16" if half else "fp32"] = {k: t for k, t in f.items() if k != "g"}
    if s["case"]["clip"]:
        out["norm"] = s["norm"]
    return out


def plain_adamw(s):
    norm = coef = None
    if s["case"]["clip"]:
        sums = [views(s, k)["g"].float().square().sum() for k in range(len(s["layout"]))]
        norm = torch.stack(sums).sum().sqrt()
        coef = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)
        ok = torch.isfinite(norm).float()
        s["norm"].copy_(torch.stack([norm, coef, ok, torch.zeros_like(ok)]))
    b1, b2, t = ADAMW["beta1"], ADAMW["beta2"], ADAMW["step"]
    step_size = ADAMW["lr"] / (1.0 - b1 ** t)
    root = 1.0 / math.sqrt(1.0 - b2 ** t)
    for k, (n, half, _, _) in enumerate(s["layout"]):
        x = views(s, k)
        decay = 1.0 - ADAMW["lr"] * (DECAY if n >= 65536 else 0.0)
        g = x["g"].float() if coef is None else x["g"].float() * coef
        m, v = x["m"], x["v"]
        if "m_scale" in x:
            m = m.float() * x["m_scale"].repeat_interleave(BLOCK)[:n]
            v = (v.float() * x["v_scale"].repeat_interleave(BLOCK)[:n]).square()
        m = m * b1 + g * (1.0 - b1)
        v = v * b2 + g * g * (1.0 - b2)
        u = torch.sqrt(v)
        p = x.get("master", x["p"])
        p = p.float() * decay - m * step_size / (u * root + ADAMW["eps"])
        x["p"].copy_(p)
        if "master" in x:
            x["master"].copy_(p)
        if "m_scale" in x:
            dither = plain_dither(n, k)
            plain_store(m, dither, 0.0, x["m"], x["m_scale"])
            plain_store(u, dither, 2.0 ** -9, x["v"], x["v_scale"])
        else:
            x["m"].copy_(m)
            x["v"].copy_(v)
    return adamw_outputs(s)


def plain_mix(x):
    """A 32-bit hash of whole numbers held in 64 bits."""
    x = (x ^ (x >> 16)) * 0x6A09E667 & 0xFFFFFFFF
    x = (x ^ (x >> 15)) * 0xBB67AE85 & 0xFFFFFFFF
    return x ^ (x >> 16)


def plain_dither(n, k):
    """20 bits an element from the step's seed, the tensor's place in the list and the element's:
    neighbours in a pair take the halves of one hash."""
    place = plain_mix(torch.full((), ADAMW["seed"] + k * 0x9E3779B1 & 0xFFFFFFFF, device="cuda",
                                 dtype=torch.int64))
    pair = torch.arange(-(-n // 2), device="cuda")
    h = plain_mix((pair * 0x9E3779B1 + place) & 0xFFFFFFFF)
    bits = torch.stack([h & 0xFFFF, h >> 16], 1).reshape(-1)[:n]
    return (bits << 4 | 8).int()


def plain_store(x, dither, least, codes, scales):
    """x in blocks of 256 with one scale (largest magnitude / 448), each value rounded to one of
    its two E4M3 neighbours by the dither; values that are not zero are at least `least`."""
    n = x.numel()
    full = torch.zeros(scales.numel() * BLOCK, device=x.device)
    full[:n] = x
    scale = full.view(-1, BLOCK).abs().amax(1) / E4M3_MAX
    inv = torch.where(scale >= 2.0 ** -126, 1.0 / scale, 0.0)
    r = (x.abs() * inv.repeat_interleave(BLOCK)[:n]).clamp(max=E4M3_MAX)
    shift = (r < 2.0 ** -6) * 2.0 ** -6      # below the normal range: fixed steps of 2^-9
    q = ((r + shift).view(torch.int32) + dither & -0x100000).view(torch.float32) - shift
    q = torch.where(r > 0, q.clamp(least, E4M3_MAX), 0.0)
    codes.copy_(torch.copysign(q, x))
    scales.copy_(torch.where(inv > 0, scale, 0.0))


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    kind = case["kind"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if kind == "adamw":
        total = flops = 0
        for n, half, _, _ in flat_layout(case["sizes"], case["packed"])[0]:
            p = (4 if half else 8) + (8 if half and case["master"] else 0)
            if half and case["master"]:
                p -= 2                                          # the bf16 copy is written only
            g = 2 if half and case["grads"] == "bf16" else 4
            total += n * (p + g + (16 if case["states"] == 32 else 4))
            total += 0 if case["states"] == 32 else 16 * -(-n // BLOCK)
            flops += n * (16 + 3 * case["clip"])
        return {"bytes": total, "flops": flops}
    if kind in ("embed", "embed_grad"):
        n, V, d = case["n"], case["V"], case["d"]
        live = n * (1 - case["masked"])
        # ids of frequency ~ 1 / rank: the distinct ones among the live positions, expected
        distinct = sum((1 - (1 - math.log1p(1.0 / (i + 1)) / math.log(V + 1)) ** live)
                       for i in range(V))
        ids = n * (4 if case["ids"] == "int32" else 8)
        if kind == "embed":
            return {"bytes": ids + distinct * d * size[case["dtype"]] + n * d * size[case["out"]],
                    "flops": n * d}
        table = 2 * distinct if case["accumulate"] else V
        return {"bytes": ids + live * d * size[case["dtype"]] + table * d * size[case["out"]],
                "flops": live * d + distinct * d}
    T, d, E, R = case["T"], case["d"], case["E"], case["R"]
    N = rows_bound(T, R, E, case["align"], case["capacity"])
    b = size[case["dtype"]]
    kept = T * R * (1 - case["drop"])
    if case["capacity"] > 0:
        kept = min(kept, E * case["capacity"])
    slots, tokens = 4 * T * R, T * d * b
    weights = slots if case["weights"] else 0
    if kind == "sort":
        return {"bytes": 2 * slots + 4 * N + 8 * E + weights + tokens + N * d * b,
                "flops": kept * d if case["weights"] else 0}
    if kind == "back":
        return {"bytes": slots + weights + kept * d * b + tokens, "flops": 2 * kept * d}
    if kind == "sort_grad":
        return {"bytes": 2 * slots + weights + kept * d * b + 2 * tokens, "flops": 4 * kept * d}
    return {"bytes": 2 * slots + weights + 4 * N + tokens + kept * d * b + N * d * b,
            "flops": 3 * kept * d}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    f8 = torch.float64
    if kind == "adamw":
        return exact_adamw(s)
    if kind in ("embed", "embed_grad"):
        V, d = case["V"], case["d"]
        ids = s["ids"].long()
        live = ((ids >= 0) & (ids < V)).nonzero()[:, 0]
        if kind == "embed":
            out = torch.zeros(case["n"], d, dtype=f8, device="cuda")
            out[live] = s["table"].to(f8)[ids[live]].mul_(s["scale"])
            return {"out": out}
        out = torch.zeros(V, d, dtype=f8, device="cuda")
        order = live[torch.argsort(ids[live])]
        for part in order.split(4096):
            out.index_add_(0, ids[part], s["dout"][part].to(f8), alpha=s["scale"])
        return {"dtable": out + s["dtable"].to(f8) if case["accumulate"] else out}
    T, d, E, R, N = case["T"], case["d"], case["E"], case["R"], s["N"]
    w = s["w"].to(f8) if case["weights"] else torch.ones(T, R, dtype=f8, device="cuda")
    if kind == "sort":
        slot_row = plan(s["idx"], E, case["align"], case["capacity"], N)[3]
    else:
        slot_row = s["slot_row"]
    wide = torch.zeros(N if kind in ("sort", "back_grad") else T, d, dtype=f8, device="cuda")
    dots = torch.zeros(T, R, dtype=f8, device="cuda")
    for r in range(R):
        for t in (slot_row[:, r] >= 0).nonzero()[:, 0].split(8192):
            row = slot_row[t, r].long()
            if kind in ("sort", "back_grad"):
                token = s["x" if kind == "sort" else "dy"][t].to(f8)
                wide[row] = token * w[t, r, None]
                if kind == "back_grad":
                    dots[t, r] = (token * s["rows"][row].to(f8)).sum(1)
            else:
                value = s["rows"][row].to(f8)
                wide[t] += value * w[t, r, None]
                if kind == "sort_grad":
                    dots[t, r] = (value * s["x"][t].to(f8)).sum(1)
    if kind == "sort":
        return {"counts": None, "offsets": None, "row_slot": None, "slot_row": None, "rows": wide}
    if kind == "back":
        return {"y": wide}
    return {"drows" if kind == "back_grad" else "dx": wide, "dw": dots}


def exact_adamw(s):
    case, f8 = s["case"], torch.float64
    coef, record = 1.0, None
    if case["clip"]:
        total = math.sqrt(sum(float(views(s, k)["g"].to(f8).square().sum())
                              for k in range(len(s["layout"]))))
        coef = min(1.0, MAX_NORM / (total + 1e-6))
        record = torch.tensor([total, coef, 1.0, 0.0], dtype=f8, device="cuda")
    outs = {half: {name: None if t.dtype == torch.float8_e4m3fn else t.to(f8)
                   for name, t in f.items() if name != "g"} for half, f in s["flat"].items()}
    c1 = 1.0 - ADAMW["beta1"] ** ADAMW["step"]
    c2 = 1.0 - ADAMW["beta2"] ** ADAMW["step"]
    for k, (n, half, at, first) in enumerate(s["layout"]):
        x, o = views(s, k), outs[half]
        g = x["g"].to(f8) * coef
        m, v = x["m"].to(f8), x["v"].to(f8)
        blocks = -(-n // BLOCK)
        if case["states"] == 8:
            owner = torch.arange(n, device="cuda") // BLOCK
            m = m * x["m_scale"].to(f8)[owner]
            v = (v * x["v_scale"].to(f8)[owner]) ** 2
        m = ADAMW["beta1"] * m + (1.0 - ADAMW["beta1"]) * g
        v = ADAMW["beta2"] * v + (1.0 - ADAMW["beta2"]) * g ** 2
        old = x.get("master", x["p"]).to(f8)
        wd = DECAY if n >= 65536 else 0.0
        new = old - ADAMW["lr"] * (m / c1 / (torch.sqrt(v / c2) + ADAMW["eps"]) + wd * old)
        o["p"][at:at + n] = new
        if "master" in o:
            o["master"][at:at + n] = new
        if case["states"] == 32:
            o["m"][at:at + n], o["v"][at:at + n] = m, v
        else:
            for name, value in (("m_scale", m.abs()), ("v_scale", v.sqrt())):
                top = torch.zeros(blocks, dtype=f8, device="cuda")
                o[name][first:first + blocks] = top.scatter_reduce_(0, owner, value,
                                                                    "amax") / E4M3_MAX
    out = {"bf16" if half else "fp32": o for half, o in outs.items()}
    if record is not None:
        out["norm"] = record
    return out
