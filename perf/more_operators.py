"""The measured cases of three further operators of the layer: products with 4-bit weights (dense and
by expert), the balance loss of the routing with the experts' counts and its gradient, and the
gradient of the selection's weights in the logits.

Every case is one pass as a program makes it: one product; the loss and its gradient; the gradient
of a selection. With `own` false, `run` computes the operators from elementary torch operations in
32 bits; with `own` true it calls the library. Shapes follow the layer's rounds (hidden 2048, 256
experts and the shared expert's gate, top-8, expert intermediate 512, rounds of 4, 32, 192, 4097 and
8192 tokens); the dense products also take generic shapes.

4-bit weights: codes 0..15, two per byte along K (the even column in the low nibble), w [E][M][K/2];
scale [E][K/G][M] of groups of G columns; zero [E][K/G][M] uint8, or 8 for every group:
weight = scale * (code - zero). Rows are sorted by expert, offsets [E + 1] holds each expert's
first row.
"""
import math

import torch

own = False

TOP_K = 8
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


def listed():
    return [
        # the shared expert's gate/up product of a decode round: one small matrix, four tokens
        {"name": "linear_w4_decode_t4", "op": "linear_w4", "T": 4, "K": 2048, "M": 1024, "G": 128,
         "zero": False, "sdt": "bf16", "dtype": "bf16", "out": "bf16", "swiglu": True},
        # one token's projection onto 65536 channels (a vocabulary): a matrix-vector product
        {"name": "linear_w4_wide_t1", "op": "linear_w4", "T": 1, "K": 4096, "M": 65536, "G": 64,
         "zero": True, "sdt": "bf16", "dtype": "bf16", "out": "f32", "swiglu": False},
        # a dense projection of a batched decode round
        {"name": "linear_w4_batch_t32", "op": "linear_w4", "T": 32, "K": 4096, "M": 4096, "G": 128,
         "zero": False, "sdt": "bf16", "dtype": "bf16", "out": "bf16", "swiglu": False},
        # the same projection of a prefill chunk
        {"name": "linear_w4_prefill_t8192", "op": "linear_w4", "T": 8192, "K": 4096, "M": 4096,
         "G": 128, "zero": False, "sdt": "bf16", "dtype": "bf16", "out": "bf16", "swiglu": False},
        # the experts' gate/up of a batched decode round: one stream of most experts' weights
        {"name": "gate_up_w4_decode_t32", "op": "gate_up_w4", "T": 32, "K": 2048, "M": 1024,
         "G": 128, "E": 256, "skew": False, "zero": False, "sdt": "bf16", "dtype": "bf16",
         "out": "bf16"},
        # and of a prefill chunk: every expert's weights and 65536 rows
        {"name": "gate_up_w4_prefill_t8192", "op": "gate_up_w4", "T": 8192, "K": 2048, "M": 1024,
         "G": 64, "E": 256, "skew": False, "zero": False, "sdt": "bf16", "dtype": "bf16",
         "out": "bf16"},
        # the experts' down product of a verify round with skewed routing: rows kept in fp32 on
        # both sides, weights with zero points in small groups
        {"name": "down_w4_verify_t192", "op": "down_w4", "T": 192, "K": 512, "M": 2048, "G": 32,
         "E": 256, "skew": True, "zero": True, "sdt": "f32", "dtype": "f32", "out": "f32"},
        # the balance of a small training or tuning batch: latency only
        {"name": "balance_t192", "op": "balance", "T": 192, "E": 256, "gate": True, "skew": True,
         "mask": False, "dtype": "f32"},
        # of a training micro-batch
        {"name": "balance_t8192", "op": "balance", "T": 8192, "E": 256, "gate": True,
         "skew": False, "mask": False, "dtype": "f32"},
        # of a large padded batch, bf16 logits without the shared expert's column
        {"name": "balance_padded_t131072", "op": "balance", "T": 131072, "E": 256, "gate": False,
         "skew": True, "mask": True, "dtype": "bf16"},
        # the selection's gradient of an odd micro-batch
        {"name": "select_grad_t4097", "op": "select_grad", "T": 4097, "E": 256, "gate": True},
        # and of a large batch
        {"name": "select_grad_t131072", "op": "select_grad", "T": 131072, "E": 256, "gate": True},
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear_w4", "linear_w4", "gate_up_w4", "down_w4", "balance", "select_grad"))
    experts = rng.choice((8, 16, 60, 64, 128, 255, 256))
    if op in ("balance", "select_grad"):
        # eight experts are all chosen by every token: nothing to balance
        case = {"op": op, "T": _log(rng, 1, 131072), "E": max(experts, 9),
                "gate": rng.random() < 0.5}
        if op == "balance":
            case.update(skew=rng.random() < 0.5, mask=rng.random() < 0.5,
                        dtype=rng.choice(("f32", "bf16")))
        return case
    G = rng.choice((32, 64, 128))
    case = {"op": op, "T": _log(rng, 1, 8192), "G": G, "zero": rng.random() < 0.4,
            "sdt": rng.choice(("f32", "bf16")), "dtype": rng.choice(("f32", "bf16", "bf16")),
            "out": rng.choice(("f32", "bf16"))}
    if op == "linear_w4":
        case["K"] = G * _log(rng, 1, 8192 // G)
        case["M"] = 16 * _log(rng, 1, 4096)
        case["swiglu"] = rng.random() < 0.4
        while case["M"] * case["K"] > 2 ** 28:
            case["M"] = case["M"] // 32 * 16
        while case["T"] * case["M"] * case["K"] > 2 ** 37:
            case["T"] = case["T"] // 2
        return case
    case["K"] = G * _log(rng, 1, 4096 // G)
    case["M"] = 16 * _log(rng, 1, 256)
    case["E"] = experts
    case["skew"] = rng.random() < 0.5
    while experts * case["M"] * case["K"] > 2 ** 29:
        case["M"] = max(16, case["M"] // 32 * 16)
        case["K"] = max(G, case["K"] // (2 * G) * G)
    # the rows of a skewed routing may nearly all belong to the same few experts
    rows = experts if case["skew"] else TOP_K
    while rows * case["T"] * case["M"] * case["K"] > 2 ** 37:
        case["T"] = case["T"] // 2
    return case


def _scores(case, gen):
    """Router scores [T][E] fp32; skew: a bias per expert of variance 2."""
    z = torch.randn((case["T"], case["E"]), generator=gen, device="cuda")
    if case.get("skew"):
        z += torch.randn((case["E"],), generator=gen, device="cuda") * math.sqrt(2.0)
    return z


def _weights(gen, E, M, K, G, zero, sdt):
    """(codes [E][M][K/2], scale [E][K/G][M], zero [E][K/G][M] or None) of N(0, 1/K) weights. With
    zeros the weights are off centre and each group's range is taken, without them its largest
    absolute value."""
    w = torch.empty((E, M, K // 2), dtype=torch.uint8, device="cuda")
    scale = torch.empty((E, K // G, M), dtype=sdt, device="cuda")
    zeros = torch.empty((E, K // G, M), dtype=torch.uint8, device="cuda") if zero else None
    step = max(1, 2 ** 27 // (M * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        v = torch.randn((n, M, K // G, G), generator=gen, device="cuda") / math.sqrt(K)
        z = torch.full((n, M, K // G), 8.0, device="cuda")
        if zero:
            v += 0.5 / math.sqrt(K) * torch.randn((n, M, K // G, 1), generator=gen, device="cuda")
            lo, hi = v.amin(dim=-1), v.amax(dim=-1)
            s = ((hi - lo) / 15.0).to(sdt).float()
            z = torch.round(-lo / s).clamp(0, 15)
            zeros[e:e + n] = z.transpose(1, 2).to(torch.uint8)
        else:
            s = (v.abs().amax(dim=-1) / 7.0).to(sdt).float()
        scale[e:e + n] = s.transpose(1, 2).to(sdt)
        c = (torch.round(v / s[..., None]) + z[..., None]).clamp(0, 15).to(torch.uint8)
        c = c.reshape(n, M, K // 2, 2)
        w[e:e + n] = c[..., 0] | (c[..., 1] << 4)
    return w, scale, zeros


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, T = case["op"], case["T"]
    s = {"case": dict(case)}
    if op in ("balance", "select_grad"):
        E = case["E"]
        z = _scores(case, gen)
        top, ids = z.topk(TOP_K, dim=1)
        s["ids"] = ids.to(torch.int32)
        if op == "balance":
            if case["gate"]:  # the shared expert's score beside the experts'
                z = torch.cat([z, torch.randn((T, 1), generator=gen, device="cuda")], dim=1)
            s["logits"] = z.to(DTYPES[case["dtype"]]).contiguous()
            # sequences padded at their ends: tokens that do not count
            s["mask"] = None
            if case["mask"]:
                at = torch.arange(T, device="cuda")
                length = torch.randint(1, 513, (T // 512 + 1,), generator=gen, device="cuda")
                s["mask"] = at % 512 < length[at // 512]
            s["dloss"] = torch.full((), 0.01, device="cuda")  # the loss's weight in the whole
            return s
        s["w"] = torch.softmax(top, dim=1)
        s["dw"] = torch.randn((T, TOP_K), generator=gen, device="cuda") * 1e-2
        s["gate"] = s["dgate"] = None
        if case["gate"]:
            s["gate"] = torch.sigmoid(torch.randn((T,), generator=gen, device="cuda"))
            s["dgate"] = torch.randn((T,), generator=gen, device="cuda") * 1e-2
        return s
    K, dt = case["K"], DTYPES[case["dtype"]]
    s["w"], s["scale"], s["zero"] = _weights(gen, case.get("E", 1), case["M"], K, case["G"],
                                             case["zero"], DTYPES[case["sdt"]])
    s["offsets"] = None
    if op == "linear_w4":
        s["x"] = torch.randn((T, K), generator=gen, device="cuda").to(dt)
        return s
    _, ids = _scores(case, gen).topk(TOP_K, dim=1)
    flat = ids.reshape(-1)
    counts = torch.bincount(flat, minlength=case["E"])
    s["offsets"] = torch.zeros(case["E"] + 1, dtype=torch.int32, device="cuda")
    s["offsets"][1:] = counts.cumsum(0)
    order = torch.argsort(flat, stable=True)
    # the plain form's tables: the touched experts, and each row's place among them
    s["touched"] = counts.nonzero()[:, 0]
    expert = flat[order]
    s["group"] = torch.searchsorted(s["touched"], expert)
    s["place"] = torch.arange(T * TOP_K, device="cuda") - s["offsets"].long()[expert]
    s["most"] = int(counts.max())
    if op == "gate_up_w4":
        s["x"] = torch.randn((T, K), generator=gen, device="cuda").to(dt)[order // TOP_K]
    else:  # the rows a SwiGLU gives
        g = torch.randn((T * TOP_K, K), generator=gen, device="cuda")
        u = torch.randn((T * TOP_K, K), generator=gen, device="cuda")
        s["x"] = (g * torch.sigmoid(g) * u).to(dt)
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _swiglu(case):
    return case["op"] == "gate_up_w4" or case.get("swiglu", False)


def _run_own(s):
    from sparse_moe_routing_amd import binding
    c = s["case"]
    if c["op"] == "balance":
        loss, counts, tokens = binding.balance_loss(s["logits"], s["ids"], c["E"], mask=s["mask"])
        dlogits = binding.balance_loss_backward(s["dloss"], s["logits"], counts, tokens,
                                                mask=s["mask"])
        return [loss, counts, tokens, dlogits]
    if c["op"] == "select_grad":
        return binding.route_backward(s["dw"], s["w"], s["ids"], c["E"], dgate=s["dgate"],
                                      gate=s["gate"])
    return binding.matmul_w4(s["x"], s["w"], s["scale"], zero=s["zero"], offsets=s["offsets"],
                             swiglu=_swiglu(c), dtype=DTYPES[c["out"]])


def _spread(w, scale, zero):
    """Weights [E][M][K] in fp32 of codes, scales and zeros."""
    E, M, half = w.shape
    groups = scale.shape[1]
    codes = torch.stack([w & 15, w >> 4], dim=-1).reshape(E, M, groups, 2 * half // groups).float()
    z = 8.0 if zero is None else zero.transpose(1, 2)[..., None].float()
    return ((codes - z) * scale.transpose(1, 2)[..., None].float()).reshape(E, M, 2 * half)


def _half_swiglu(z):
    half = z.shape[-1] // 2
    g, u = z[..., :half], z[..., half:]
    return g / (1.0 + torch.exp(-g)) * u


def _run_plain(s):
    c = s["case"]
    op, T = c["op"], c["T"]
    if op == "balance":
        E, ids, mask = c["E"], s["ids"].long(), s["mask"]
        z = s["logits"][:, :E].float()
        on = torch.ones((T,), dtype=torch.bool, device=z.device) if mask is None else mask
        e = torch.exp(z - z.amax(dim=1, keepdim=True))
        p = torch.where(on[:, None], e / e.sum(dim=1, keepdim=True), 0.0)
        counts = torch.zeros((E,), dtype=torch.int32, device=z.device)
        counts.index_add_(0, ids.reshape(-1), on[:, None].expand(T, TOP_K).reshape(-1).int())
        tokens = on.sum().to(torch.int32)
        n = tokens.double().clamp(min=1.0)
        mean = p.sum(dim=0, dtype=torch.float64) / n
        share = counts.double() / (TOP_K * n)
        loss = (E * (share * mean).sum()).float()
        # sum_e P = 1: taken off the shares, so that what is left of them is not a small difference
        d = (share - 1.0 / E).float()
        dz = p * (d[None, :] - (p * d[None, :]).sum(dim=1, keepdim=True))
        dlogits = torch.zeros_like(s["logits"])
        dlogits[:, :E] = (dz * (s["dloss"] * (E / n)).float()).to(dlogits.dtype)
        return [loss, counts, tokens, dlogits]
    if op == "select_grad":
        w, dw = s["w"], s["dw"]
        v = w * (dw - (w * dw).sum(dim=1, keepdim=True))
        out = torch.zeros((T, c["E"] + (1 if c["gate"] else 0)), device=w.device)
        out.scatter_add_(1, s["ids"].long(), v)
        if c["gate"]:
            out[:, c["E"]] = s["gate"] * (1.0 - s["gate"]) * s["dgate"]
        return out
    x = s["x"].float()
    if op == "linear_w4":
        z = x @ _spread(s["w"], s["scale"], s["zero"])[0].t()
    else:
        t = s["touched"]
        w = _spread(s["w"][t], s["scale"][t], None if s["zero"] is None else s["zero"][t])
        pad = torch.zeros((t.numel(), s["most"], c["K"]), device=x.device)
        pad[s["group"], s["place"]] = x
        z = torch.bmm(pad, w.transpose(1, 2).contiguous())[s["group"], s["place"]]
    return (_half_swiglu(z) if _swiglu(c) else z).to(DTYPES[c["out"]])


def work(case):
    op, T = case["op"], case["T"]
    if op == "balance":
        R, es = case["E"] + (1 if case["gate"] else 0), BYTES[case["dtype"]]
        # the logits are read for the loss and, once all tokens have been counted, for the gradient
        return {"bytes": 3 * T * R * es + 4 * TOP_K * T + (2 * T if case["mask"] else 0),
                "flops": 12 * T * case["E"]}
    if op == "select_grad":
        R = case["E"] + (1 if case["gate"] else 0)
        return {"bytes": 4 * T * R + 12 * TOP_K * T + (8 * T if case["gate"] else 0),
                "flops": 5 * TOP_K * T}
    K, M, E = case["K"], case["M"], case.get("E", 1)
    n = T if op == "linear_w4" else T * TOP_K
    # distinct experts that T tokens touch, routing taken as uniform
    touched = 1 if E == 1 else E * (1.0 - (1.0 - TOP_K / E) ** T)
    per_group = BYTES[case["sdt"]] + (1 if case["zero"] else 0)
    out = M // 2 if _swiglu(case) else M
    read = n * K * BYTES[case["dtype"]] + touched * M * (K / 2 + K // case["G"] * per_group)
    return {"bytes": int(read + n * out * BYTES[case["out"]] + (0 if E == 1 else 4 * (E + 1))),
            "flops": 2 * n * M * K}


def exact(case, seed):
    """The operators' outputs in 64 bits from their definitions: the products expert by expert and
    nibble by nibble, the loss from each token's log probabilities, its gradient and the
    selection's as products with the softmax's Jacobian."""
    s = prepare(case, seed)
    op, T = case["op"], case["T"]
    if op == "balance":
        E, ids = case["E"], s["ids"].long()
        keep = (torch.arange(T, device="cuda") if s["mask"] is None else s["mask"].nonzero()[:, 0])
        n = keep.numel()
        logp = torch.log_softmax(s["logits"][keep, :E].double(), dim=1)
        counts = torch.bincount(ids[keep].reshape(-1), minlength=E)
        f = counts.double() / (TOP_K * max(n, 1))
        loss = E * torch.dot(f, torch.exp(logp).sum(dim=0)) / max(n, 1)
        dlogits = torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda")
        p = torch.exp(logp)
        dlogits[keep, :E] = s["dloss"].double() * E / max(n, 1) * (p * f - p * torch.mv(p, f)[:, None])
        return [loss, counts.int(), torch.tensor(n, dtype=torch.int32, device="cuda"), dlogits]
    if op == "select_grad":
        w, ids = s["w"].double(), s["ids"].long()
        jacobian = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
        d = (jacobian * s["dw"].double()[:, None, :]).sum(dim=2)
        out = torch.zeros((T, case["E"] + (1 if case["gate"] else 0)), dtype=torch.float64,
                          device="cuda")
        token = torch.arange(T, device="cuda")[:, None]
        out.index_put_((token, ids), d, accumulate=True)
        if case["gate"]:
            g = s["gate"].double()
            out[:, case["E"]] = s["dgate"].double() * (g - g * g)
        return out
    K, M, G, E = case["K"], case["M"], case["G"], case.get("E", 1)
    swiglu = _swiglu(case)
    out = torch.empty((s["x"].shape[0], M // 2 if swiglu else M), dtype=torch.float64,
                      device="cuda")
    at = [0, s["x"].shape[0]] if s["offsets"] is None else s["offsets"].tolist()
    for e in range(E):
        if at[e] == at[e + 1]:
            continue
        v = torch.empty((M, K), dtype=torch.float64, device="cuda")
        v[:, 0::2] = s["w"][e].remainder(16).double()
        v[:, 1::2] = s["w"][e].div(16, rounding_mode="floor").double()
        v -= 8.0 if s["zero"] is None else s["zero"][e].double().repeat_interleave(G, dim=0).t()
        v *= s["scale"][e].double().repeat_interleave(G, dim=0).t()
        z = torch.matmul(s["x"][at[e]:at[e + 1]].double(), v.t().contiguous())
        if swiglu:
            z = z[:, :M // 2] * torch.sigmoid(z[:, :M // 2]) * z[:, M // 2:]
        out[at[e]:at[e + 1]] = z
    return out
