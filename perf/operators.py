"""The measured cases of liblora's 4-bit operators: quantisation to MXFP4, the
mixed-adapter linear layer over an MXFP4 base weight, and a mixture-of-experts
layer for a few tokens.

A case is run in one of two forms on the same inputs: with ``own`` true by
the calls a user makes of ``rank_gemm_amd.lora``, otherwise by elementary
torch operations in 32 bits, rounded once at the end. ``exact`` gives the
same outputs from the operators' definitions in 64 bits.

MXFP4 (OCP Microscaling Formats 1.0): 32 consecutive values of a row share a
scale 2^(b - 127), b one byte; each value is E2M1, one of 0, .5, 1, 1.5, 2, 3,
4, 6 with a sign, two to a byte, the earlier one in the low four bits.
Quantising a block takes b - 127 = floor(log2(max |v|)) - 2 and rounds v /
scale to the nearest E2M1 value, ties to the even mantissa, at most 6.
"""
import math

import torch

own = False

# ------------------------------------------------------------------- cases --


def _quant(name, rows, cols, src):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "src": src}


def _lin(name, T, d_in, d_out, act, slots=9, rank=16, mixed=False):
    return {"name": name, "op": "linear", "T": T, "d_in": d_in, "d_out": d_out, "act": act, "slots": slots,
            "rank": rank, "mixed": mixed}


def _moe(name, T, hidden, inner, experts, k, weights, renorm=True):
    return {"name": name, "op": "moe", "T": T, "hidden": hidden, "inner": inner, "experts": experts, "k": k,
            "weights": weights, "renorm": renorm}


def listed():
    return [
        # the activations of one decode step, as the layer quantises them: latency
        _quant("quant_decode_rows", 16, 4096, "bf16"),
        # a whole gate projection brought to 4 bits at load time
        _quant("quant_gate_weight", 14336, 4096, "bf16"),
        # odd rows and a last block that is not full, from 32-bit values
        _quant("quant_ragged_f32", 1021, 1450, "f32"),
        # one user's next token through q_proj: the smallest call
        _lin("lin_decode_t1", 1, 4096, 4096, "bf16"),
        # a full decode batch through the gate projection, 8 adapters
        _lin("lin_decode_t64_gate", 64, 4096, 14336, "bf16"),
        # a short ragged prefill with adapters of several ranks, odd widths
        _lin("lin_ragged_t333", 333, 4088, 1021, "bf16", slots=6, rank=32, mixed=True),
        # prefill of the down projection with the activations kept in 16 bits
        _lin("lin_prefill_down", 2048, 14336, 4096, "bf16", slots=17),
        # prefill of the gate projection, both sides in 4 bits: the largest
        _lin("lin_prefill_gate_a4", 8192, 4096, 14336, "mx4", slots=17),
        # a decode batch with both sides in 4 bits
        _lin("lin_decode_t48_a4", 48, 4096, 4096, "mx4"),
        # one token through a layer of many experts
        _moe("moe_t1", 1, 4096, 1792, 64, 4, "mx4"),
        # a decode batch that reaches almost every expert
        _moe("moe_t32", 32, 4096, 1792, 32, 4, "mx4"),
        # few wide experts in 16 bits, odd inner width, weights not renormalised
        _moe("moe_t7_bf16", 7, 2056, 1000, 8, 2, "bf16", renorm=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "moe"])
    if op == "quantize":
        rows, cols = _log_int(rng, 1, 16384), _log_int(rng, 32, 16384)
        while rows * cols > 14336 * 4096:
            rows = max(1, rows // 2)
        c = _quant("", rows, cols, rng.choice(["bf16", "f32"]))
    elif op == "linear":
        T = _log_int(rng, 1, 8192)
        d_in, d_out = _log_int(rng, 256, 14336), _log_int(rng, 256, 14336)
        if rng.random() < 0.75:  # most models' widths are multiples of 8
            d_in, d_out = d_in // 8 * 8, d_out // 8 * 8
        while T * d_in * d_out > 8192 * 4096 * 14336:
            T = max(1, T // 2)
        c = _lin("", T, d_in, d_out, rng.choice(["bf16", "mx4"]), rng.randint(2, 33),
                 rng.choice([4, 8, 12, 16, 32, 64]), rng.random() < 0.5)
    else:
        experts = _log_int(rng, 4, 64)
        k = rng.randint(1, min(8, experts))
        T = _log_int(rng, 1, 64)
        hidden, inner = _log_int(rng, 256, 4096) // 8 * 8, _log_int(rng, 128, 2048)
        weights = rng.choice(["mx4", "mx4", "bf16"])
        if weights == "bf16":
            inner = inner // 8 * 8
        c = _moe("", T, hidden, inner, experts, k, weights, rng.random() < 0.5)
    del c["name"]
    return c


def work(case):
    """Bytes and operations one pass cannot do without: every input read once,
    every output written once."""
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        blocks = case["rows"] * -(-case["cols"] // 32)
        # the source, the codes and scales written, the bf16 values written
        return {"bytes": n * (2 if case["src"] == "bf16" else 4) + blocks * 17 + n * 2, "flops": 4 * n}
    if case["op"] == "linear":
        T, d_in, d_out = case["T"], case["d_in"], case["d_out"]
        ranks = _ranks(case)
        live = min(T, case["slots"] - 1)  # adapters that can have a token
        per_rank = sum(ranks[1:]) / max(1, len(ranks) - 1)
        on = T * (case["slots"] - 1) / case["slots"]  # tokens on an adapter, on average
        by = d_out * -(-d_in // 32) * 17 + 2 * T * (d_in + d_out) + 2 * live * per_rank * (d_in + d_out)
        return {"bytes": int(by), "flops": int(2 * T * d_in * d_out + 2 * on * per_rank * (d_in + d_out))}
    T, H, N, E, k = (case[n] for n in ("T", "hidden", "inner", "experts", "k"))
    reached = E * (1.0 - (1.0 - k / E) ** T)  # experts that get a token, on average
    if case["weights"] == "mx4":
        expert = (2 * N * -(-H // 32) + H * -(-N // 32)) * 17
    else:
        expert = 3 * N * H * 2
    return {"bytes": int(reached * expert + 2 * E * H + 4 * T * H + 8 * T * k),
            "flops": int(6 * T * k * N * H + 2 * T * E * H)}


# ------------------------------------------------------------------ inputs --


def _ranks(case):
    """Rank of each slot; slot 0 is the zero adapter."""
    r = case["rank"]
    if not case["mixed"]:
        return [0] + [r] * (case["slots"] - 1)
    return [0] + [max(1, r >> (s % 3)) for s in range(1, case["slots"])]


def _quantize_plain(v):
    """(codes, scale bytes) of fp32 rows: whole blocks, zeros behind the row's end."""
    rows, cols = v.shape
    nb = -(-cols // 32)
    if nb * 32 != cols:
        v = torch.nn.functional.pad(v, (0, nb * 32 - cols))
    v = v.view(rows, nb, 32)
    top = v.abs().amax(dim=2)
    byte = ((top.view(torch.int32) >> 23) - 2).clamp_(min=0)  # floor(log2) + 127 - 2, from the exponent field
    inv = ((254 - byte) << 23).view(torch.float32)            # 2^(127 - byte)
    a = v * inv.unsqueeze(2)
    m = a.abs()
    # half-way points to the next E2M1 value; a tie goes to the even mantissa
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = code + 8 * (a.view(torch.int32) < 0)
    code = code.to(torch.uint8).view(rows, nb * 16, 2)
    return code[:, :, 0] | (code[:, :, 1] << 4), byte.to(torch.uint8)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _values_plain(codes, byte, cols):
    """The fp32 values of 4-bit rows."""
    lut = torch.tensor(_E2M1, dtype=torch.float32, device=codes.device)
    rows, nb = byte.shape
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), dim=2).view(rows, nb, 32)
    v = v * (byte.int() << 23).view(torch.float32).unsqueeze(2)
    return v.view(rows, nb * 32)[:, :cols]


def _inputs(case, seed):
    """The case's inputs, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "quantize":
        # rows of different sizes, and a few outlying values, as activations have them
        x = normal(case["rows"], case["cols"]) * torch.exp(normal(case["rows"], 1))
        x = torch.where(torch.rand(x.shape, generator=g, device="cuda") < 1e-3, x * 30.0, x)
        return {"x": x.to(torch.bfloat16) if case["src"] == "bf16" else x}
    if case["op"] == "linear":
        T, d_in, d_out = case["T"], case["d_in"], case["d_out"]
        codes, byte = _quantize_plain(normal(d_out, d_in) * d_in ** -0.5)
        A, B = [None], [None]
        for r in _ranks(case)[1:]:
            A.append((normal(r, d_in) * d_in ** -0.5).to(torch.bfloat16))
            B.append((normal(d_out, r) * 0.25).to(torch.bfloat16))
        ids = torch.randint(0, case["slots"], (T,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
        return {"x": normal(T, d_in).to(torch.bfloat16), "codes": codes, "byte": byte, "A": A, "B": B, "ids": ids,
                "alpha": 2.0 * case["rank"]}
    T, H, N, E = case["T"], case["hidden"], case["inner"], case["experts"]
    s = {"x": normal(T, H).to(torch.bfloat16), "router": (normal(E, H) * H ** -0.5).to(torch.bfloat16)}
    for name, n, c in (("gate", N, H), ("up", N, H), ("down", H, N)):
        if case["weights"] == "mx4":
            parts = [_quantize_plain(normal(n, c) * c ** -0.5) for _ in range(E)]
            s[name] = (torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]))
        else:
            w = torch.empty((E, n, c), dtype=torch.bfloat16, device="cuda")
            for e in range(E):
                w[e] = normal(n, c) * c ** -0.5
            s[name] = w
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = dict(case)
    s["own"] = own
    if not own:
        if case["op"] == "linear":
            # the rows of each adapter, known where the batch is put together
            s["rows"] = [torch.nonzero(s["ids"] == i).flatten().cuda() for i in range(case["slots"])]
        return s
    from rank_gemm_amd import lora

    if case["op"] == "quantize":
        s["q"] = lora.mx4_quantize(s["x"])  # the buffers such a program keeps
    elif case["op"] == "linear":
        s["W"] = lora.mx4_pack(s.pop("codes"), s.pop("byte"), case["d_in"])
        ranks = _ranks(case)
        pool = lora.Pool(case["slots"], max(ranks), case["d_in"], case["d_out"], "bf16")
        for i in range(1, case["slots"]):
            pool.install(i, s["A"][i], s["B"][i], s["alpha"])
        s["pool"], s["plan"] = pool, lora.plan(s["ids"].numpy(), case["slots"])
    elif case["weights"] == "mx4":
        for name, c in (("gate", case["hidden"]), ("up", case["hidden"]), ("down", case["inner"])):
            s[name] = lora.mx4_pack(*s[name], c)
    return s


# --------------------------------------------------------------- one pass --


def _route_plain(x, router, k, renorm):
    """Experts by falling logit, the lower index first among equals; the
    logits in 64 bits, so that no choice hangs on the order of a sum."""
    logits = x.double() @ router.double().t()
    vals, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    vals = vals.float()
    top = torch.exp(vals[:, :k] - vals[:, :1])
    den = top.sum(dim=1, keepdim=True) if renorm else torch.exp(vals - vals[:, :1]).sum(dim=1, keepdim=True)
    return ids[:, :k].to(torch.int32), top / den


def _mlp_plain(x, gate, up, down):
    g = x @ gate.transpose(-1, -2)
    return (g / (1.0 + torch.exp(-g)) * (x @ up.transpose(-1, -2))) @ down.transpose(-1, -2)


def _run_plain(s):
    case = s["case"]
    if case["op"] == "quantize":
        codes, byte = _quantize_plain(s["x"].float())
        return _values_plain(codes, byte, case["cols"]).to(torch.bfloat16)
    if case["op"] == "linear":
        x = s["x"].float()
        xb = x
        if case["act"] == "mx4":
            xb = _values_plain(*_quantize_plain(x), case["d_in"])
        y = xb @ _values_plain(s["codes"], s["byte"], case["d_in"]).t()
        for i, r in enumerate(_ranks(case)):
            rows = s["rows"][i]
            if r and rows.numel():
                h = x[rows] @ s["A"][i].float().t()
                y.index_add_(0, rows, (s["alpha"] / r) * (h @ s["B"][i].float().t()))
        return y.to(torch.bfloat16)
    ids, w = _route_plain(s["x"], s["router"], case["k"], case["renorm"])
    x, T, k, E = s["x"].float(), case["T"], case["k"], case["experts"]

    def weights(name, e):
        cols = case["inner"] if name == "down" else case["hidden"]
        if case["weights"] == "mx4":
            return _values_plain(s[name][0][e], s[name][1][e], cols)
        return s[name][e].float()

    y = torch.zeros_like(x)
    if T * k < E:  # fewer choices than experts: fetch the chosen ones
        def fetched(name, t, j):
            e = ids[t, j:j + 1].long()
            cols = case["inner"] if name == "down" else case["hidden"]
            if case["weights"] == "mx4":
                return _values_plain(s[name][0].index_select(0, e)[0], s[name][1].index_select(0, e)[0], cols)
            return s[name].index_select(0, e)[0].float()

        for t in range(T):
            for j in range(k):
                y[t] += w[t, j] * _mlp_plain(x[t:t + 1], *(fetched(n, t, j) for n in ("gate", "up", "down")))[0]
    else:  # every expert over every token, zero weight where it was not chosen
        for e in range(E):
            we = (w * (ids == e)).sum(dim=1, keepdim=True)
            y += we * _mlp_plain(x, *(weights(n, e) for n in ("gate", "up", "down")))
    return y.to(torch.bfloat16), ids, w


def run(state):
    if not state["own"]:
        return _run_plain(state)
    from rank_gemm_amd import lora

    s, case = state, state["case"]
    if case["op"] == "quantize":
        return lora.mx4_dequantize(lora.mx4_quantize(s["x"], out=s["q"]), "bf16")
    if case["op"] == "linear":
        return lora.linear_mx4(s["x"], s["W"], s["pool"], s["plan"], act=case["act"])
    ids, w = lora.moe_route(s["x"], s["router"], case["k"], renorm=case["renorm"])
    return lora.moe_experts(s["x"], ids, w, s["gate"], s["up"], s["down"]), ids, w


# ------------------------------------------------------------------- exact --


def _pow2_exact(n):
    """2^n of whole numbers n (the exponent field of a 64-bit number)."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _values_exact(codes, byte, cols):
    """4-bit rows in 64 bits, from the fields of each code: sign, two exponent
    bits (bias 1; 0 is subnormal), one mantissa bit."""
    c = torch.stack((torch.remainder(codes, 16), torch.div(codes, 16, rounding_mode="floor")), dim=-1).int()
    c = c.flatten(-2)
    sign = 1.0 - 2.0 * (c // 8).double()
    e, m = (c % 8) // 2, (c % 2).double()
    mag = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * _pow2_exact(e - 1))
    scale = _pow2_exact(byte.int() - 127).repeat_interleave(32, dim=-1)
    return (sign * mag * scale)[..., :cols]


def _nearest_exact(x):
    """The 64-bit values MXFP4 keeps of the rows of x."""
    x = x.double()
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], 32):
        blk = x[:, c:c + 32]
        top = blk.abs().amax(dim=1, keepdim=True)
        ex = torch.frexp(top)[1] - 1 - 2  # floor(log2(top)) - 2
        scale = torch.where(top > 0, _pow2_exact(torch.clamp(ex, min=-127)), torch.ones_like(top))
        v = blk / scale
        step = torch.where(v.abs() < 2.0, 0.5, torch.where(v.abs() < 4.0, 1.0, 2.0))
        out[:, c:c + 32] = torch.clamp(torch.round(v / step) * step, -6.0, 6.0) * scale  # half to even
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "quantize":
        return _nearest_exact(s["x"])
    x = s["x"].double()
    if case["op"] == "linear":
        base = _nearest_exact(x) if case["act"] == "mx4" else x
        y = base @ _values_exact(s["codes"], s["byte"], case["d_in"]).t()
        ids = s["ids"].cuda()
        for i, r in enumerate(_ranks(case)):
            if r:
                on = (ids == i).double().unsqueeze(1)
                y += on * ((x @ s["A"][i].double().t()) @ s["B"][i].double().t()) * (s["alpha"] / r)
        return y
    p = torch.softmax(x @ s["router"].double().t(), dim=1)
    order = torch.argsort(-p, dim=1, stable=True)[:, :case["k"]]
    w = torch.gather(p, 1, order)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    y = torch.zeros_like(x)
    for e in range(case["experts"]):
        hit = (order == e)
        rows = torch.nonzero(hit.any(dim=1)).flatten()
        if rows.numel() == 0:
            continue
        m = []
        for name, cols in (("gate", case["hidden"]), ("up", case["hidden"]), ("down", case["inner"])):
            m.append(_values_exact(s[name][0][e], s[name][1][e], cols) if case["weights"] == "mx4"
                     else s[name][e].double())
        xe = x[rows]
        g = xe @ m[0].t()
        y[rows] += (w * hit).sum(dim=1)[rows].unsqueeze(1) * ((g * torch.sigmoid(g) * (xe @ m[1].t())) @ m[2].t())
    return y, order.to(torch.int32), w
