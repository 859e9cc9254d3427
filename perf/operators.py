"""The measured cases of the layer's separate operators: rows sorted by expert and back with their
gradients, and products in 8-bit integers with a scale per token and per output channel.

Every case is one call (or the pair of calls that belong together: a row quantisation and the
product it feeds). With `own` false, `run` computes the operators from elementary torch
operations; with `own` true it calls the library. Shapes follow the layer's rounds: hidden 2048,
256 experts, top-8, expert intermediate 512, rounds of 4, 32, 192, 4097 and 8192 tokens; the
dense product also takes a generic square shape.

Tables of a case: `rows` [T * 8] int32 gives the sorted row of pair t * 8 + k (-1: its expert is
not on this shard), `perm` the kept pairs in sorted order, `offsets` [E + 1] the first row of each
expert.
"""
import math

import numpy as np
import torch

own = False

TOP_K = 8
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one decode round's rows in front of the experts' products: latency only
        {"name": "sort_decode_t4", "op": "sort", "T": 4, "H": 2048, "E": 256, "kept": 256,
         "skew": False, "dtype": "bf16"},
        # a prefill chunk (or a training micro-batch): eight copies of every token
        {"name": "sort_prefill_t8192", "op": "sort", "T": 8192, "H": 2048, "E": 256, "kept": 256,
         "skew": False, "dtype": "bf16"},
        # one of four expert shards, fp32: three quarters of the pairs belong to other shards
        {"name": "sort_shard_f32_t4097", "op": "sort", "T": 4097, "H": 2048, "E": 256, "kept": 64,
         "skew": True, "dtype": "f32"},
        # the gradient of the sort in a training step
        {"name": "sort_grad_t8192", "op": "sort_grad", "T": 8192, "H": 2048, "E": 256,
         "kept": 256, "skew": False, "dtype": "bf16"},
        # the weighted return of a batched decode round with the gated shared expert
        {"name": "back_decode_t32", "op": "back", "T": 32, "H": 2048, "E": 256, "kept": 256,
         "skew": False, "dtype": "bf16", "out": "f32", "shared": True},
        # the same for a prefill chunk
        {"name": "back_prefill_t8192", "op": "back", "T": 8192, "H": 2048, "E": 256, "kept": 256,
         "skew": False, "dtype": "bf16", "out": "bf16", "shared": True},
        # its gradient in a training step: an odd micro-batch
        {"name": "back_grad_t4097", "op": "back_grad", "T": 4097, "H": 2048, "E": 256,
         "kept": 256, "skew": True, "dtype": "bf16", "out": "f32", "shared": True},
        # the shared expert's gate/up product of a decode round: one dense matrix, four tokens
        {"name": "linear_i8_decode_t4", "op": "linear_i8", "T": 4, "K": 2048, "M": 1024,
         "dtype": "bf16", "out": "bf16", "swiglu": True},
        # a dense projection of a prefill chunk
        {"name": "linear_i8_prefill_t8192", "op": "linear_i8", "T": 8192, "K": 4096, "M": 4096,
         "dtype": "bf16", "out": "bf16", "swiglu": False},
        # the experts' gate/up of a batched decode round: one stream of most experts' weights
        {"name": "gate_up_i8_decode_t32", "op": "gate_up_i8", "T": 32, "K": 2048, "M": 1024,
         "E": 256, "skew": False, "dtype": "bf16", "out": "bf16"},
        # and of a prefill chunk: every expert's weights and 65536 rows
        {"name": "gate_up_i8_prefill_t8192", "op": "gate_up_i8", "T": 8192, "K": 2048, "M": 1024,
         "E": 256, "skew": False, "dtype": "bf16", "out": "bf16"},
        # the experts' down product of a verify round with skewed routing, rows kept in fp32
        {"name": "down_i8_verify_t192", "op": "down_i8", "T": 192, "K": 512, "M": 2048, "E": 256,
         "skew": True, "dtype": "bf16", "out": "f32"},
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("sort", "sort_grad", "back", "back_grad", "linear_i8", "gate_up_i8",
                     "down_i8"))
    case = {"op": op, "dtype": rng.choice(("f32", "bf16")), "T": _log(rng, 1, 8192)}
    if op.endswith("_i8"):
        # at most the prefill product's operations and weights
        case["K"] = 16 * _log(rng, 1, 256)
        case["M"] = 16 * _log(rng, 2, 256)
        case["out"] = rng.choice(("f32", "bf16"))
        if op == "linear_i8":
            case["swiglu"] = rng.random() < 0.5
            return case
        case["E"] = rng.choice((8, 16, 60, 64, 128, 255, 256))
        case["skew"] = rng.random() < 0.5
        while case["E"] * case["M"] * case["K"] > 2 ** 29:
            case["M"] = max(16, case["M"] // 32 * 16)
            case["K"] = max(16, case["K"] // 32 * 16)
        while case["T"] * case["M"] * case["K"] > 2 ** 34:
            case["T"] = case["T"] // 2
        return case
    case["H"] = 8 * _log(rng, 8, 512)
    if case["T"] * case["H"] > 2 ** 24:
        case["T"] = 2 ** 24 // case["H"]
    case["E"] = rng.choice((8, 16, 60, 64, 128, 255, 256))
    case["kept"] = case["E"] if rng.random() < 0.6 else max(1, case["E"] // rng.choice((2, 4, 8)))
    case["skew"] = rng.random() < 0.5
    if op in ("back", "back_grad"):
        case["out"] = rng.choice(("f32", "bf16"))
        case["shared"] = rng.random() < 0.5
    return case


def _routing(case, gen):
    """ids [T][8] (distinct per token, ranked) and softmax weights, as the layer's router gives
    them; skew: a bias per expert of variance 2."""
    T, E = case["T"], case["E"]
    z = torch.randn((T, E), generator=gen, device="cuda")
    if case["skew"]:
        z += torch.randn((E,), generator=gen, device="cuda") * math.sqrt(2.0)
    top, ids = z.topk(TOP_K, dim=1)
    return ids.to(torch.int32), torch.softmax(top, dim=1)


def _tables(ids, kept):
    """(rows, perm, offsets, counts on the host) of a stable sort of the pairs by expert; pairs of
    experts outside [0, kept) are dropped."""
    flat = ids.reshape(-1).long()
    order = torch.argsort(torch.where(flat < kept, flat, kept), stable=True)
    counts = torch.bincount(flat[flat < kept], minlength=kept)
    n = int(counts.sum())
    perm = order[:n]
    rows = torch.full_like(flat, -1)
    rows[perm] = torch.arange(n, device=flat.device)
    offsets = torch.zeros(kept + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = counts.cumsum(0)
    return rows.to(torch.int32), perm, offsets, counts.tolist()


def _weight_codes(gen, E, M, K):
    """(codes [E][M][K] int8, scales [E][M] fp32) of N(0, 1/K) weights, one scale per channel."""
    codes = torch.empty((E, M, K), dtype=torch.int8, device="cuda")
    scales = torch.empty((E, M), dtype=torch.float32, device="cuda")
    step = max(1, 2 ** 27 // (M * K))
    for e in range(0, E, step):
        v = torch.randn((min(step, E - e), M, K), generator=gen, device="cuda") / math.sqrt(K)
        s = v.abs().amax(dim=-1) / 127.0
        codes[e:e + step] = torch.round(v / s[..., None]).to(torch.int8)
        scales[e:e + step] = s
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, T, dt = case["op"], case["T"], DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dt)

    s = {"case": dict(case)}
    if op == "linear_i8":
        s["x"] = normal(T, case["K"])
        s["w"], s["w_scale"] = _weight_codes(gen, 1, case["M"], case["K"])
        return s
    ids, s["weights"] = _routing(case, gen)
    kept = case.get("kept", case["E"])
    s["rows"], s["perm"], s["offsets"], s["counts"] = _tables(ids, kept)
    s["ids"] = ids
    N = T * TOP_K  # row capacity: an expert shard's row count is known on the device only
    if op in ("gate_up_i8", "down_i8"):
        s["w"], s["w_scale"] = _weight_codes(gen, case["E"], case["M"], case["K"])
        if op == "gate_up_i8":
            s["x"] = normal(T, case["K"])
        else:  # the rows a SwiGLU gives
            g = torch.randn((N, case["K"]), generator=gen, device="cuda")
            u = torch.randn((N, case["K"]), generator=gen, device="cuda")
            s["x"] = (g * torch.sigmoid(g) * u).to(dt)
        return s
    H = case["H"]
    if op == "sort":
        s["x"] = normal(T, H)
        s["xs"] = torch.zeros((N, H), dtype=dt, device="cuda")  # the experts' input buffer
    elif op == "sort_grad":
        s["dxs"] = normal(N, H, scale=1e-2)
    else:
        s["ys"] = normal(N, H, scale=0.5)
        if case["shared"]:
            s["shared"] = normal(T, H, scale=0.5)
            s["gate"] = torch.sigmoid(torch.randn((T,), generator=gen, device="cuda"))
        if op == "back_grad":
            s["dy"] = (torch.randn((T, H), generator=gen, device="cuda") * 1e-2).to(
                DTYPES[case["out"]])
            s["dys"] = torch.zeros((N, H), dtype=dt, device="cuda")  # the experts' gradient buffer
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from sparse_moe_routing_amd import binding
    c = s["case"]
    op = c["op"]
    if op == "sort":
        return binding.permute(s["x"], s["rows"], xs=s["xs"])
    if op == "sort_grad":
        return binding.permute_backward(s["dxs"], s["rows"])
    if op == "back":
        return binding.unpermute(s["ys"], s["rows"], s["weights"], shared=s.get("shared"),
                                 gate=s.get("gate"), dtype=DTYPES[c["out"]])
    if op == "back_grad":
        g = binding.unpermute_backward(s["dy"], s["ys"], s["rows"], s["weights"],
                                       shared=s.get("shared"), gate=s.get("gate"), dys=s["dys"])
        return [t for t in g if t is not None]
    if op == "gate_up_i8":
        q, q_scale = binding.permute_i8(s["x"], s["rows"])
        return binding.matmul_i8(q, q_scale, s["w"], s["w_scale"], offsets=s["offsets"],
                                 swiglu=True, dtype=DTYPES[c["out"]])
    q, q_scale = binding.quantize_i8(s["x"])
    if op == "down_i8":
        return binding.matmul_i8(q, q_scale, s["w"], s["w_scale"], offsets=s["offsets"],
                                 dtype=DTYPES[c["out"]])
    return binding.matmul_i8(q, q_scale, s["w"], s["w_scale"], swiglu=c["swiglu"],
                             dtype=DTYPES[c["out"]])


def _quantize(x):
    """(codes as fp32, scales): scale the fp32 value nearest to amax / 127, code the integer
    nearest to x / scale. Both quotients are formed in 64 bits: a scale one step off would move
    the many values that lie half way between two codes."""
    scale = (x.abs().amax(dim=1).double() / 127.0).float()
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return torch.round(x.double() / scale.double()[:, None]).float(), scale


def _product(q, q_scale, w, w_scale, swiglu):
    """q [n][K], w [M][K] codes: the scaled product, or its SwiGLU (gate rows first), in fp32."""
    z = (q @ w.float().t()) * q_scale[:, None] * w_scale[None, :]
    if not swiglu:
        return z
    half = z.shape[1] // 2
    g, u = z[:, :half], z[:, half:]
    return g / (1.0 + torch.exp(-g)) * u


def _run_plain(s):
    c = s["case"]
    op, T = c["op"], c["T"]
    if op == "linear_i8":
        q, q_scale = _quantize(s["x"])
        return _product(q, q_scale, s["w"][0], s["w_scale"][0], c["swiglu"]).to(DTYPES[c["out"]])
    if op in ("gate_up_i8", "down_i8"):
        swiglu = op == "gate_up_i8"
        q, q_scale = _quantize(s["x"])
        if swiglu:
            tok = s["perm"] // TOP_K
            q, q_scale = q[tok], q_scale[tok]
        y = torch.empty((T * TOP_K, c["M"] // 2 if swiglu else c["M"]), dtype=DTYPES[c["out"]],
                        device="cuda")
        at = 0
        for e, n in enumerate(s["counts"]):
            if n:
                y[at:at + n] = _product(q[at:at + n], q_scale[at:at + n], s["w"][e],
                                        s["w_scale"][e], swiglu).to(y.dtype)
                at += n
        return y
    if op == "sort":
        s["xs"][:s["perm"].numel()] = s["x"][s["perm"] // TOP_K]
        return s["xs"]
    rows = s["rows"].long().reshape(T, TOP_K)
    on = rows >= 0
    if op == "sort_grad":
        v = s["dxs"][rows.clamp(min=0)].float()
        return torch.where(on[:, :, None], v, torch.zeros_like(v)).sum(dim=1).to(s["dxs"].dtype)
    wide = s["ys"][rows.clamp(min=0)].float()
    wide = torch.where(on[:, :, None], wide, torch.zeros_like(wide))
    if op == "back":
        y = (s["weights"][:, :, None] * wide).sum(dim=1)
        if c["shared"]:
            y = y + s["gate"][:, None] * s["shared"].float()
        return y.to(DTYPES[c["out"]])
    dy = s["dy"].float()
    dw = (dy[:, None, :] * wide).sum(dim=2)
    pair_w = s["weights"].reshape(-1)[s["perm"]]
    s["dys"][:s["perm"].numel()] = (pair_w[:, None] * dy[s["perm"] // TOP_K]).to(s["dys"].dtype)
    if not c["shared"]:
        return [s["dys"], dw]
    dshared = (s["gate"][:, None] * dy).to(s["shared"].dtype)
    return [s["dys"], dw, dshared, (dy * s["shared"].float()).sum(dim=1)]


def work(case):
    op, T = case["op"], case["T"]
    es = BYTES[case["dtype"]]
    if op.endswith("_i8"):
        K, M, eo = case["K"], case["M"], BYTES[case["out"]]
        E = case.get("E", 1)
        n = T if op == "linear_i8" else T * TOP_K
        # distinct experts that T tokens touch, routing taken as uniform
        touched = 1 if E == 1 else E * (1.0 - (1.0 - TOP_K / E) ** T)
        swiglu = op == "gate_up_i8" or case.get("swiglu", False)
        read = (n if op == "down_i8" else T) * K * es + touched * M * (K + 4)
        if op != "linear_i8":
            read += 4 * (E + 1) + (4 * n if op == "gate_up_i8" else 0)
        return {"bytes": int(read + n * (M // 2 if swiglu else M) * eo),
                "flops": 2 * n * M * K}
    H = case["H"]
    token, kept = T * H, T * TOP_K * case["kept"] / case["E"] * H
    rows = 4 * T * TOP_K
    if op in ("sort", "sort_grad"):
        return {"bytes": int((token + kept) * es + rows),
                "flops": int(kept if op == "sort_grad" else 0)}
    eo = BYTES[case["out"]]
    shared = token if case["shared"] else 0
    if op == "back":
        return {"bytes": int((kept + shared) * es + token * eo + 2 * rows),
                "flops": int(2 * (kept + shared))}
    return {"bytes": int((2 * kept + 2 * shared) * es + token * eo + 3 * rows),
            "flops": int(3 * (kept + shared))}


def exact(case, seed):
    """The operators' outputs in 64 bits, pair by pair from the routing ids (not from the tables
    that the other forms use)."""
    s = prepare(case, seed)
    op, T = case["op"], case["T"]
    if op.endswith("_i8"):
        x = s["x"].double()
        amax = x.abs().max(dim=1).values
        # the scale is an fp32 number by definition
        scale = torch.where(amax > 0, (amax / 127.0).float().double(), torch.ones_like(amax))
        codes = (x / scale[:, None]).round_()
        if op == "linear_i8":
            groups = [(0, torch.arange(T, device="cuda"), 0)]
        else:
            ids, groups, at = s["ids"].long(), [], 0
            for e in range(case["E"]):
                hit = (ids.reshape(-1) == e).nonzero()[:, 0]  # pairs of the expert, in order
                src = hit // TOP_K if op == "gate_up_i8" else torch.arange(
                    at, at + hit.numel(), device="cuda")
                groups.append((e, src, at))
                at += hit.numel()
        swiglu = op == "gate_up_i8" or case.get("swiglu", False)
        n = T if op == "linear_i8" else T * TOP_K
        out = torch.empty((n, case["M"] // 2 if swiglu else case["M"]), dtype=torch.float64,
                          device="cuda")
        for e, src, at in groups:
            if src.numel() == 0:
                continue
            w = s["w"][e].double() * s["w_scale"][e].double()[:, None]
            z = torch.matmul(codes[src] * scale[src][:, None], w.t().contiguous())
            if swiglu:
                half = case["M"] // 2
                z = z[:, :half] * torch.sigmoid(z[:, :half]) * z[:, half:]
            out[at:at + src.numel()] = z
        return out
    H, ids = case["H"], s["ids"].cpu().numpy()
    kept = case["kept"]
    # sorted rows by expert, then token, then rank
    pairs = [(e, t, k) for t, row in enumerate(ids.tolist()) for k, e in enumerate(row) if e < kept]
    pairs.sort()
    tok = torch.from_numpy(np.array([p[1] for p in pairs], np.int64)).cuda()
    rank = torch.from_numpy(np.array([p[2] for p in pairs], np.int64)).cuda()
    n = len(pairs)
    if op == "sort":
        xs = torch.zeros((T * TOP_K, H), dtype=torch.float64, device="cuda")
        xs[:n] = s["x"].double().index_select(0, tok)
        return xs
    if op == "sort_grad":
        dx = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        return dx.index_add_(0, tok, s["dxs"][:n].double())
    w, ys = s["weights"].double(), s["ys"][:n].double()
    wr = w[tok, rank]
    if op == "back":
        y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        y.index_add_(0, tok, ys * wr[:, None])
        if case["shared"]:
            y += s["shared"].double() * s["gate"].double()[:, None]
        return y
    dy = s["dy"].double()
    dys = torch.zeros((T * TOP_K, H), dtype=torch.float64, device="cuda")
    dys[:n] = dy[tok] * wr[:, None]
    dw = torch.zeros((T, TOP_K), dtype=torch.float64, device="cuda")
    dw[tok, rank] = torch.linalg.vecdot(dy[tok], ys)
    if not case["shared"]:
        return [dys, dw]
    return [dys, dw, dy * s["gate"].double()[:, None], torch.linalg.vecdot(dy, s["shared"].double())]
