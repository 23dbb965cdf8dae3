"""The measured cases of liblora's operators around the adapted projections of a
decode step: storing keys and values in a paged cache, attention of one new
token a request over that cache, routing to experts by scores with a bias and
groups, and sampling the next token.

A case is run in one of two forms on the same inputs: with ``own`` true by
the calls a user makes of ``rank_gemm_amd.lora``, otherwise by elementary
torch operations in 32 bits (64 where a choice hangs on the last bits),
rounded once at the end. ``exact`` gives the same outputs from the operators'
definitions in 64 bits.

The cache: pages of ``page`` tokens, [pages, page, kv heads, dim], in bf16 or
in 8 bits (E4M3) with one fp32 scale a kv head; a request's tokens lie in the
pages that its row of the page table names, in order.
"""
import math

import torch

own = False

E4M3_MAX = 448.0

# ------------------------------------------------------------------- cases --


def _attn(name, batch, longest, heads, kv_heads, dim, page, cache, window=0, shortest=1, lse=False):
    return {"name": name, "op": "attn", "batch": batch, "longest": longest, "shortest": shortest, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "cache": cache, "window": window, "lse": lse}


def _append(name, tokens, heads, kv_heads, dim, page, cache):
    return {"name": name, "op": "append", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "cache": cache}


def _route(name, tokens, hidden, experts, k, score, groups=1, top_groups=1, group_best=2, bias=True, renorm=True,
           scale=1.0):
    return {"name": name, "op": "route", "tokens": tokens, "hidden": hidden, "experts": experts, "k": k,
            "score": score, "groups": groups, "top_groups": top_groups, "group_best": group_best, "bias": bias,
            "renorm": renorm, "scale": scale}


def _sample(name, batch, vocab, logits, filters="mixed"):
    return {"name": name, "op": "sample", "batch": batch, "vocab": vocab, "logits": logits, "filters": filters}


def listed():
    return [
        # one user, a short context: the smallest call, all latency
        _attn("attn_one_short", 1, 137, 32, 8, 128, 16, "bf16", shortest=137),
        # a decode batch of requests of very different lengths, small pages
        _attn("attn_batch64", 64, 4096, 32, 8, 128, 16, "bf16"),
        # a full card of long requests: the largest
        _attn("attn_largest", 64, 16384, 32, 8, 128, 64, "bf16", shortest=4096),
        # one request of a very long context over an 8-bit cache
        _attn("attn_long_one", 1, 131072, 32, 8, 128, 64, "f8", shortest=131072, lse=True),
        # odd head dimension, group and page, a sliding window, 8-bit cache
        _attn("attn_odd_window", 23, 3001, 12, 2, 80, 24, "f8", window=1000),
        # the new tokens of a decode batch into an 8-bit cache: latency
        _append("append_decode", 64, 32, 8, 128, 16, "f8"),
        # the keys and values of a long prefill
        _append("append_prefill", 8192, 32, 8, 128, 64, "bf16"),
        # one token over many experts in groups: latency
        _route("route_t1", 1, 4096, 128, 8, "sigmoid", 8, 4, scale=2.5),
        # a decode batch over many experts in groups
        _route("route_t64", 64, 4096, 256, 8, "sigmoid", 8, 4, scale=2.5),
        # one user's next token: latency
        _sample("sample_one", 1, 131072, "bf16"),
        # a decode batch, odd vocabulary, every request with its own filters
        _sample("sample_batch48", 48, 50021, "bf16"),
        # a large batch with 32-bit logits
        _sample("sample_batch256", 256, 131072, "f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "route", "sample", "sample"])
    if op == "attn":
        heads, kv = rng.choice([(32, 8), (32, 8), (40, 8), (28, 4), (16, 16), (12, 2), (16, 1), (64, 2), (3, 3)])
        dim = rng.choice([64, 80, 96, 112, 128, 128, 256])
        page = rng.choice([1, 8, 16, 24, 32, 64, 128, 256])
        batch, longest = _log_int(rng, 1, 256), _log_int(rng, 1, 131072)
        cache = rng.choice(["bf16", "f8"])
        while batch * longest * kv * dim > 64 * 10000 * 8 * 128:
            if batch > 1:
                batch //= 2
            else:
                longest //= 2
        window = rng.choice([0, 0, _log_int(rng, 1, longest)])
        c = _attn("", batch, longest, heads, kv, dim, page, cache, window, rng.choice([1, longest // 2 + 1, longest]),
                  rng.random() < 0.3)
    elif op == "append":
        heads, kv = rng.choice([(32, 8), (40, 8), (28, 4), (12, 2), (16, 16), (3, 3)])
        c = _append("", _log_int(rng, 1, 16384), heads, kv, rng.choice([64, 80, 96, 128, 256]),
                    rng.choice([1, 8, 16, 24, 64, 128]), rng.choice(["bf16", "f8"]))
    elif op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log_int(rng, 4, 512 // groups)
        top = rng.randint(1, groups)
        k = rng.randint(1, min(8, top * (experts // groups)))
        c = _route("", _log_int(rng, 1, 64), _log_int(rng, 256, 8192) // 8 * 8, experts, k,
                   rng.choice(["sigmoid", "softmax"]), groups, top, rng.choice([1, 2]), rng.random() < 0.6,
                   rng.random() < 0.6, rng.choice([1.0, 2.5]))
    else:
        batch, vocab = _log_int(rng, 1, 512), _log_int(rng, 1000, 262144)
        while batch * vocab > 256 * 131072:
            batch //= 2
        c = _sample("", batch, vocab, rng.choice(["bf16", "f32"]), rng.choice(["mixed", "mixed", "none", "top_p", "top_k"]))
    del c["name"]
    return c


def work(case):
    """Bytes and operations one pass cannot do without: every input read once,
    every output written once."""
    if case["op"] == "attn":
        B, D, H, KV = case["batch"], case["dim"], case["heads"], case["kv_heads"]
        mean = (case["shortest"] + case["longest"]) / 2.0
        if case["window"]:
            lo, hi, w = case["shortest"], case["longest"], case["window"]
            mean = sum(min(lo + (hi - lo) * (i + 0.5) / 64, w) for i in range(64)) / 64
        es = 2 if case["cache"] == "bf16" else 1
        return {"bytes": int(B * (mean * KV * D * 2 * es + 4 * H * D + 4 * mean / case["page"])),
                "flops": int(4 * B * mean * H * D)}
    if case["op"] == "append":
        n = 2 * case["tokens"] * case["kv_heads"] * case["dim"]
        return {"bytes": n * (4 if case["cache"] == "bf16" else 3) + 8 * case["tokens"], "flops": n}
    if case["op"] == "route":
        T, H, E = case["tokens"], case["hidden"], case["experts"]
        return {"bytes": 2 * T * H + 2 * E * H + 8 * T * case["k"], "flops": 2 * T * E * H}
    n = case["batch"] * case["vocab"]
    return {"bytes": n * (2 if case["logits"] == "bf16" else 4), "flops": 4 * n}


# ------------------------------------------------------------------ inputs --


def _cache_values(g, case, pages):
    """Keys or values of a cache, and the scales of an 8-bit one."""
    x = torch.randn(pages, case["page"], case["kv_heads"], case["dim"], generator=g, device="cuda",
                    dtype=torch.bfloat16)
    if case["cache"] == "bf16":
        return x, None
    scale = 0.005 + 0.02 * torch.rand(case["kv_heads"], generator=g, device="cuda")
    return (x / scale.view(1, 1, -1, 1)).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _inputs(case, seed):
    """The case's inputs, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    if case["op"] == "attn":
        B, page = case["batch"], case["page"]
        lens = torch.randint(case["shortest"], case["longest"] + 1, (B,), generator=host, dtype=torch.int32)
        lens[0] = case["longest"]
        if B > 8:
            lens[B // 2] = 0  # a place of the batch that no request holds
        width = -(-case["longest"] // page)
        need = (lens + page - 1) // page
        pages = int(need.sum()) + 3
        # the pages in use, in no order, as a server that has run for a while hands them out
        order = torch.randperm(pages, generator=host).to(torch.int32)
        first = torch.cumsum(need, 0) - need
        at = first.unsqueeze(1) + torch.arange(width).unsqueeze(0)
        used = torch.arange(width).unsqueeze(0) < need.unsqueeze(1)
        table = torch.where(used, order[at.clamp(max=pages - 1)], torch.zeros((), dtype=torch.int32))
        # rows of the merged q, k and v projections
        qkv = torch.randn(B, (case["heads"] + 2 * case["kv_heads"]) * case["dim"], generator=g, device="cuda")
        k, ks = _cache_values(g, case, pages)
        v, vs = _cache_values(g, case, pages)
        return {"qkv": (2.0 * qkv).to(torch.bfloat16), "k_cache": k, "v_cache": v, "k_scale": ks, "v_scale": vs,
                "table": table.cuda(), "lens": lens.cuda()}
    if case["op"] == "append":
        T, page = case["tokens"], case["page"]
        pages = -(-2 * T // page) + 1
        rows = torch.randperm(pages * page, generator=host)[:T]
        if T > 8:
            rows[T // 2] = -1  # a padded place of the batch
        qkv = torch.randn(T, (case["heads"] + 2 * case["kv_heads"]) * case["dim"], generator=g, device="cuda")
        k, ks = _cache_values(g, case, pages)
        v, vs = _cache_values(g, case, pages)
        return {"qkv": (1.5 * qkv).to(torch.bfloat16), "k_cache": k, "v_cache": v, "k_scale": ks, "v_scale": vs,
                "rows": rows.cuda()}
    if case["op"] == "route":
        T, H, E = case["tokens"], case["hidden"], case["experts"]
        x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
        r = (1.5 * torch.randn(E, H, generator=g, device="cuda") * H ** -0.5).to(torch.bfloat16)
        return {"x": x, "router": r, "bias": 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None}
    B, V = case["batch"], case["vocab"]
    # most of a vocabulary far down, a few likely tokens
    x = 2.0 * torch.randn(B, V, generator=g, device="cuda") - 4.0
    few = torch.rand(B, V, generator=g, device="cuda") < 40.0 / V
    x = torch.where(few, x + 6.0 + 6.0 * torch.rand(B, V, generator=g, device="cuda"), x)

    def of(values, dtype):
        pick = torch.randint(0, len(values), (B,), generator=host)
        return torch.tensor(values, dtype=dtype)[pick].cuda()

    f = case["filters"]
    return {"logits": x.to(torch.bfloat16) if case["logits"] == "bf16" else x,
            "u": torch.rand(B, generator=host, dtype=torch.float64).cuda(),
            # every request's own; 0 is the likeliest token alone
            "temperature": of([0.6, 0.8, 1.0, 1.3] if f == "top_p" or B == 1 else [0.0, 0.6, 0.8, 1.0, 1.3], torch.float32),
            "top_k": None if f in ("none", "top_p") else of([20, 50, 200] if f == "top_k" else [0, 0, 20, 50, 1000], torch.int32),
            "top_p": None if f in ("none", "top_k") else of([0.8, 0.9, 0.95] if B == 1 or f == "top_p" else [1.0, 0.8, 0.9, 0.95],
                                                            torch.float32),
            "min_p": None if f != "mixed" else of([0.0, 0.0, 0.02, 0.1], torch.float32)}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = dict(case)
    s["own"] = own
    return s


# --------------------------------------------------------------- one pass --


def _split(qkv, case):
    """The q, k and v of merged rows, as views."""
    H, KV, D = case["heads"], case["kv_heads"], case["dim"]
    n = qkv.shape[0]
    return (qkv[:, :H * D].view(n, H, D), qkv[:, H * D:(H + KV) * D].view(n, KV, D),
            qkv[:, (H + KV) * D:].view(n, KV, D))


def _paged(cache, scale, table):
    """[batch, kv heads, tokens, dim] in fp32 of the pages that the table names."""
    got = cache.view(torch.uint8)[table.long()] if scale is not None else cache[table.long()]
    if scale is not None:
        got = got.view(torch.float8_e4m3fn)
    got = got.float().flatten(1, 2).transpose(1, 2)
    return got if scale is None else got * scale.view(1, -1, 1, 1)


def _attn_plain(s, case):
    q = _split(s["qkv"], case)[0].float()
    B, H, D = q.shape
    KV, P = case["kv_heads"], case["page"]
    k, v = _paged(s["k_cache"], s["k_scale"], s["table"]), _paged(s["v_cache"], s["v_scale"], s["table"])
    at = torch.arange(k.shape[2], device=q.device).unsqueeze(0)
    lens = s["lens"].long().unsqueeze(1)
    on = at < lens
    if case["window"]:
        on &= at >= lens - case["window"]
    on = on[:, None, None, :]
    z = (q.view(B, KV, H // KV, D) * D ** -0.5) @ k.transpose(2, 3).contiguous()
    z = torch.where(on, z, -math.inf)
    top = z.amax(dim=3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(z - top)
    den = p.sum(dim=3, keepdim=True)
    out = (p @ v.contiguous()) / torch.where(den == 0, 1.0, den)
    out = out.view(B, H, D).to(torch.bfloat16)
    return (out, (torch.log(den) + top).view(B, H)) if case["lse"] else out


def _append_plain(s, case):
    _, k, v = _split(s["qkv"], case)
    rows = s["rows"]
    keep = torch.nonzero((rows >= 0) & (rows < s["k_cache"].shape[0] * case["page"])).flatten()
    at = rows[keep]

    def store(x, cache, scale):
        x = x[keep]
        if scale is None:
            cache.flatten(0, 1)[at] = x
        else:
            x = (x.float() / scale.view(1, -1, 1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            cache.view(torch.uint8).flatten(0, 1)[at] = x.view(torch.uint8)
        return cache

    return store(k, s["k_cache"], s["k_scale"]), store(v, s["v_cache"], s["v_scale"])


def _route_plain(s, case):
    z = s["x"].double() @ s["router"].double().t()  # in 64 bits, so that no choice hangs on the order of a sum
    T, E = z.shape
    if case["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-z))
    else:
        score = torch.exp(z - z.amax(dim=1, keepdim=True))
        score = score / score.sum(dim=1, keepdim=True)
    c = score if s["bias"] is None else score + s["bias"].double()
    if case["groups"] > 1:
        by = c.view(T, case["groups"], -1)
        best = torch.sort(by, dim=2, descending=True).values[:, :, :case["group_best"]].sum(dim=2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        on = (kept.unsqueeze(2) == torch.arange(case["groups"], device=z.device)).any(dim=1)
        c = torch.where(on.unsqueeze(2), by, -math.inf).view(T, E)
    ids = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :case["k"]]
    w = torch.gather(score, 1, ids)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), (w * case["scale"]).float()


def _sample_plain(s, case):
    x = s["logits"].double()  # in 64 bits, so that no choice hangs on the rounding of a sum
    B, V = x.shape
    t = s["temperature"].double().unsqueeze(1)
    z, idx = torch.sort(x, dim=1, descending=True, stable=True)  # equal logits by index
    w = torch.exp((z - z[:, :1]) / torch.where(t > 0, t, 1.0))
    at = torch.arange(V, device=x.device).unsqueeze(0)
    keep = (t > 0) | (at == 0)
    if s["top_k"] is not None:
        k = s["top_k"].unsqueeze(1)
        keep &= (k <= 0) | (at < k)
    w = torch.where(keep, w, 0.0)
    if s["top_p"] is not None:
        p = s["top_p"].double().unsqueeze(1)
        before = torch.cumsum(w, dim=1) - w
        keep &= (p >= 1) | (at == 0) | (before < p * w.sum(dim=1, keepdim=True))
    if s["min_p"] is not None:
        keep &= (at == 0) | (w >= s["min_p"].double().unsqueeze(1))
    w = torch.zeros_like(w).scatter_(1, idx, torch.where(keep, w, 0.0))  # back in the vocabulary's order
    run = torch.cumsum(w, dim=1)
    ids = (run <= s["u"].unsqueeze(1) * run[:, -1:]).sum(dim=1, keepdim=True).clamp(max=V - 1)
    return ids.flatten().to(torch.int32), (torch.gather(w, 1, ids) / run[:, -1:]).flatten().float()


def run(state):
    s, case = state, state["case"]
    if not s["own"]:
        return {"attn": _attn_plain, "append": _append_plain, "route": _route_plain,
                "sample": _sample_plain}[case["op"]](s, case)
    from rank_gemm_amd import lora

    if case["op"] == "attn":
        return lora.attn_decode(_split(s["qkv"], case)[0], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                window=case["window"], k_scale=s["k_scale"], v_scale=s["v_scale"], lse=case["lse"])
    if case["op"] == "append":
        _, k, v = _split(s["qkv"], case)
        lora.kv_append(k, v, s["k_cache"], s["v_cache"], s["rows"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["k_cache"], s["v_cache"]
    if case["op"] == "route":
        return lora.moe_route_scored(s["x"], s["router"], case["k"], score=case["score"], bias=s["bias"],
                                     groups=case["groups"], top_groups=case["top_groups"],
                                     group_best=case["group_best"], renorm=case["renorm"], scale=case["scale"])
    return lora.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                       min_p=s["min_p"])


# ------------------------------------------------------------------- exact --


def _attn_exact(s, case):
    """A request at a time, over its own tokens alone."""
    q = _split(s["qkv"], case)[0].double()
    B, H, D = q.shape
    KV = case["kv_heads"]
    out = torch.zeros(B, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device=q.device)
    table, page = s["table"].long(), case["page"]
    for b, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n <= lo:
            continue
        at = torch.arange(lo, n, device=q.device)
        where = table[b, torch.div(at, page, rounding_mode="floor")], torch.remainder(at, page)

        def rows(cache, scale):
            if scale is None:
                return cache[where].double()
            return cache.view(torch.uint8)[where].view(torch.float8_e4m3fn).double() * scale.double()[None, :, None]

        k, v = rows(s["k_cache"], s["k_scale"]), rows(s["v_cache"], s["v_scale"])
        for h in range(KV):
            heads = slice(h * (H // KV), (h + 1) * (H // KV))
            z = (q[b, heads] @ k[:, h].t().contiguous()) / math.sqrt(D)
            out[b, heads] = torch.softmax(z, dim=1) @ v[:, h].contiguous()
            lse[b, heads] = torch.logsumexp(z, dim=1)
    return (out, lse) if case["lse"] else out


def _nearest_e4m3(x):
    """The 64-bit values that E4M3 keeps of x: 4 bits of mantissa down to 2^-6, steps of 2^-9 below."""
    x = x.clamp(-E4M3_MAX, E4M3_MAX)
    step = torch.pow(2.0, torch.clamp(torch.frexp(x)[1].double() - 4, min=-9.0))
    return torch.round(x / step) * step  # half to even


def _append_exact(s, case):
    _, k, v = _split(s["qkv"], case)
    found = []
    for x, cache, scale in ((k, s["k_cache"], s["k_scale"]), (v, s["v_cache"], s["v_scale"])):
        flat = cache.double().flatten(0, 1)
        x = x.double()
        if scale is not None:
            # the quotient is taken in 32 bits, as the definition has it
            x = _nearest_e4m3((x.float() / scale.view(1, -1, 1)).double())
        on = s["rows"] >= 0
        flat.index_copy_(0, s["rows"][on], x[on])
        found.append(flat.view(cache.shape))
    return tuple(found)


def _route_exact(s, case):
    z = s["x"].double() @ s["router"].double().t()
    score = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, dim=1)
    c = score.clone()
    if s["bias"] is not None:
        c += s["bias"].double()
    T, E = c.shape
    n = E // case["groups"]
    if case["groups"] > 1:
        value = torch.topk(c.view(T, -1, n), min(case["group_best"], n), dim=2).values.sum(dim=2)
        rank = torch.argsort(torch.argsort(-value, dim=1, stable=True), dim=1)
        c[(rank >= case["top_groups"]).repeat_interleave(n, dim=1)] = -math.inf
    ids = torch.argsort(-c, dim=1, stable=True)[:, :case["k"]]
    w = score.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), w * case["scale"]


def _sample_exact(s, case):
    """A request at a time: its candidates in falling order, then the draw."""
    ids, probs = [], []

    def of(name, off):
        return [off] * case["batch"] if s[name] is None else s[name].tolist()

    for row, u, t, k, p, least in zip(s["logits"], s["u"].tolist(), s["temperature"].tolist(), of("top_k", 0),
                                      of("top_p", 1.0), of("min_p", 0.0)):
        x = row.double()
        order = torch.argsort(-x, stable=True)
        if t <= 0:
            ids.append(int(order[0])), probs.append(1.0)
            continue
        if k > 0:
            order = order[:k]
        w = torch.exp((x[order] - x[order[0]]) / t)
        n = order.numel()
        if p < 1:
            n = min(n, max(1, int(torch.searchsorted(torch.cumsum(w, 0), p * float(w.sum()))) + 1))
        if least > 0:
            n = min(n, max(1, int((w >= least).sum())))
        kept, place = torch.sort(order[:n])
        w = w[:n][place]
        run = torch.cumsum(w, 0)
        i = min(int(torch.searchsorted(run, u * float(run[-1]), right=True)), n - 1)
        ids.append(int(kept[i])), probs.append(float(w[i] / run[-1]))
    return torch.tensor(ids, dtype=torch.int32), torch.tensor(probs, dtype=torch.float64)


def exact(case, seed):
    s = _inputs(case, seed)
    return {"attn": _attn_exact, "append": _append_exact, "route": _route_exact, "sample": _sample_exact}[case["op"]](
        s, case)
