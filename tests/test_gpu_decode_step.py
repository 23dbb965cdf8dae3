"""A decode step over the paged cache as a server runs it, eager and from a
captured graph: q, k, v with adapters, append, attention, output projection,
router, experts, logits, sampling; each step against the one before it redone
in plain torch."""
import numpy as np
import pytest
import torch

from rank_gemm_amd import lora

pytestmark = pytest.mark.gpu

B, HID, HEADS, KV, DIM, PAGE, WIDTH, SLOTS, E, V = 6, 512, 8, 2, 64, 16, 8, 4, 16, 3001


def bf(*shape, scale=1.0, g=None):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


class Model:
    def __init__(self, form):
        g = torch.Generator(device="cuda").manual_seed(11)
        widths = {"q": (HID, HEADS * DIM), "k": (HID, KV * DIM), "v": (HID, KV * DIM), "o": (HEADS * DIM, HID)}
        self.W, self.pool = {}, {}
        for n, (i, o) in widths.items():
            self.W[n] = bf(o, i, scale=i ** -0.5, g=g)
            self.pool[n] = lora.Pool(SLOTS, 8, i, o, "bf16")
            for s in range(1, SLOTS):
                self.pool[n].install(s, bf(8, i, scale=i ** -0.5, g=g), bf(o, 8, scale=0.3, g=g), 16.0)
        self.router = bf(E, HID, scale=HID ** -0.5, g=g)
        self.bias = 0.1 * torch.randn(E, generator=g, device="cuda")
        self.experts = [bf(E, 64, HID, scale=HID ** -0.5, g=g), bf(E, 64, HID, scale=HID ** -0.5, g=g),
                        bf(E, HID, 64, scale=0.125, g=g)]
        self.head = bf(V, HID, scale=4 * HID ** -0.5, g=g)
        pages = B * WIDTH + 3
        dt = torch.bfloat16 if form == "bf16" else torch.float8_e4m3fn
        self.kc, self.vc = (torch.zeros(pages, PAGE, KV, DIM, device="cuda").to(dt) for _ in range(2))
        self.ks = self.vs = None
        if form == "f8":
            self.ks, self.vs = (torch.full((KV,), 0.02, device="cuda") for _ in range(2))
        perm = np.random.default_rng(2).permutation(pages)[:B * WIDTH].reshape(B, WIDTH)
        self.table = torch.from_numpy(perm.astype(np.int32)).cuda()
        self.plan = lora.plan([0, 1, 2, 3, 1, 0], SLOTS)

    def step(self, h, rows, lengths, u, t, p):
        q, k, v = (lora.linear(h, self.W[n], self.pool[n], self.plan) for n in "qkv")
        k, v = k.view(B, KV, DIM), v.view(B, KV, DIM)
        lora.kv_append(k, v, self.kc, self.vc, rows, k_scale=self.ks, v_scale=self.vs)
        a = lora.attn_decode(q.view(B, HEADS, DIM), self.kc, self.vc, self.table, lengths, k_scale=self.ks,
                             v_scale=self.vs)
        x = lora.linear(a.view(B, HEADS * DIM), self.W["o"], self.pool["o"], self.plan)
        ids, w = lora.moe_route_scored(x, self.router, 4, bias=self.bias, groups=4, top_groups=2, scale=1.5)
        y = lora.moe_experts(x, ids, w, *self.experts)
        z = torch.matmul(y, self.head.t())
        tok, prob = lora.sample(z, u, temperature=t, top_p=p)
        return dict(q=q, k=k, v=v, a=a, x=x, ids=ids, w=w, z=z, tok=tok, prob=prob)

    def check(self, r, lengths, u, t, p, history):
        """Each operator's outputs from the ones before them (history: the keys and
        values of earlier steps, per request)."""
        for b in range(B):
            n = int(lengths[b])
            if n == 0:
                assert not r["a"][b].any()
                continue
            kk, vv = (torch.stack([s[b] for s in history[name][-n:]]).float() for name in ("k", "v"))
            if self.ks is not None:  # the values the cache keeps
                kk, vv = ((x / 0.02).clamp(-448, 448).to(torch.float8_e4m3fn).float() * 0.02 for x in (kk, vv))
            q = r["q"][b].view(KV, HEADS // KV, DIM).float()
            s = torch.einsum("hgd,nhd->hgn", q.cpu(), kk.cpu()) * DIM ** -0.5
            ref = torch.einsum("hgn,nhd->hgd", torch.softmax(s, -1), vv.cpu()).reshape(HEADS, DIM)
            err = (r["a"][b].float().cpu() - ref).abs()
            # one rounding to bf16, and fp32 sums of a few dozen positions and 64 products
            assert bool((err <= 2.0 ** -8 * ref.abs() + 2.0 ** -14 * vv.abs().max().cpu()).all())
        z = r["x"].double() @ self.router.double().t()
        s = torch.sigmoid(z)
        c = s + self.bias.double()
        value = torch.topk(c.view(B, 4, -1), 2, dim=2).values.sum(2)
        keep = torch.topk(value, 2, dim=1).indices
        off = torch.ones(B, 4, dtype=torch.bool, device="cuda").scatter_(1, keep, False)
        ids = torch.topk(c.masked_fill(off.repeat_interleave(E // 4, 1), -9.0), 4, dim=1).indices
        assert torch.equal(ids.int(), r["ids"])
        w = s.gather(1, ids)
        np.testing.assert_allclose(r["w"].cpu().numpy(), (1.5 * w / w.sum(1, keepdim=True)).float().cpu().numpy(),
                                   rtol=2.0 ** -23)
        import decode_ref
        for b in range(B):
            want, prob = decode_ref.sample(r["z"][b].float().cpu().numpy(), float(u[b]), float(t[b]), 0, float(p[b]), 0.0)
            assert int(r["tok"][b]) == want
            np.testing.assert_allclose(float(r["prob"][b]), prob, rtol=2.0 ** -23)


def rows_at(m, pos):
    """The cache row of each request's position (-1: a place that no request holds)."""
    page = m.table.gather(1, (pos.clamp(min=0) // PAGE).view(B, 1)).view(B).long()
    return torch.where(pos >= 0, page * PAGE + pos.clamp(min=0) % PAGE, torch.full_like(page, -1))


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("form", ["bf16", "f8"])
def test_decode_steps(form, captured):
    m = Model(form)
    g = torch.Generator(device="cuda").manual_seed(3)
    h = bf(B, HID, g=g)
    rows = torch.full((B,), -1, dtype=torch.int64, device="cuda")
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    u = torch.rand(B, dtype=torch.float64, device="cuda")
    t, p = torch.tensor([0.0, 0.7, 1.0, 1.2, 0.7, 1.0], device="cuda"), torch.full((B,), 0.9, device="cuda")
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            m.step(h, rows, lengths, u, t, p)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r = m.step(h, rows, lengths, u, t, p)
    history = {"k": [], "v": []}
    for step in range(40):
        h.copy_(bf(B, HID, g=g))
        u.copy_(torch.rand(B, generator=g, dtype=torch.float64, device="cuda"))
        pos = torch.full((B,), step, dtype=torch.int64, device="cuda")
        pos[4] = -1  # never a request here
        rows.copy_(rows_at(m, pos))
        lengths.copy_((pos + 1).int())
        if captured:
            graph.replay()
        else:
            r = m.step(h, rows, lengths, u, t, p)
        history["k"].append(r["k"].clone())
        history["v"].append(r["v"].clone())
        if step in (0, 1, 15, 16, 17, 39):
            torch.cuda.synchronize()
            m.check(r, lengths, u, t, p, history)
