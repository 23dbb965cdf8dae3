"""The mixture-of-experts layer for a few tokens against its 64-bit form
(tests/mx4_ref.py). Choices of experts are compared exactly; weights are fp32
(a few steps of 2^-24 each for the exponential, the sum and the quotient);
outputs are one rounding to bf16 (2^-8 of the value) from sums whose loss the
reference bounds."""
import numpy as np
import pytest
import torch

from rank_gemm_amd import lora
from rank_gemm_amd.inputs import bf16_bits, bf16_to_f32
import mx4_ref

pytestmark = pytest.mark.gpu


def dev_bf16(v):
    bits = bf16_bits(np.asarray(v, np.float32))
    return lora.to_device(bits, "bf16"), bf16_to_f32(bits).astype(np.float64)


def as64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Moe:
    def __init__(self, T, H, I, E, k, form, seed=0):
        g = np.random.default_rng(seed)
        self.T, self.H, self.I, self.E, self.k, self.form = T, H, I, E, k, form
        self.x, self.x64 = dev_bf16(g.standard_normal((T, H)))
        self.router, self.router64 = dev_bf16(g.standard_normal((E, H)) * H ** -0.5)
        self.w, self.w64 = [], []
        for n, c in ((I, H), (I, H), (H, I)):
            v = g.standard_normal((E, n, c)) * c ** -0.5
            if form == "bf16":
                d, v64 = dev_bf16(v)
            else:
                d = lora.mx4_quantize(torch.from_numpy(v.astype(np.float32)).cuda())
                v64 = lora.mx4_dequantize(d, "f32").cpu().numpy().astype(np.float64)
            self.w.append(d)
            self.w64.append(v64)

    def experts(self, ids, weights, x=None, y=None):
        n = lora.lib().lora_moe_experts_workspace_bytes(self.T, self.H, self.I, self.k)
        ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")
        return lora.moe_experts(self.x if x is None else x, ids, weights, *self.w, y=y, workspace=ws)

    def check(self, y, ids, weights):
        ref, lost = mx4_ref.experts(self.x64, ids, np.asarray(weights, np.float64), *self.w64)
        err = np.abs(as64(y) - ref)
        bound = 2.0 ** -8 * np.abs(ref) + 1.01 * lost + 1e-30
        worst = float((err / bound).max())
        print(f"T={self.T} H={self.H} I={self.I} E={self.E} k={self.k} {self.form}: worst {worst:.3f} of its bound",
              flush=True)
        assert worst <= 1.0


ROUTES = [(1, 64, 4, 1), (1, 256, 8, 2), (3, 8, 1, 1), (7, 1000, 60, 4), (64, 512, 64, 8), (5, 2056, 130, 16),
          (32, 264, 512, 16), (512, 64, 8, 1), (200, 128, 100, 2)]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,H,E,k", ROUTES)
def test_route(T, H, E, k, renorm):
    g = np.random.default_rng(T + H + E)
    x, x64 = dev_bf16(g.standard_normal((T, H)))
    r, r64 = dev_bf16(g.standard_normal((E, H)) * 2 * H ** -0.5)
    ids, w = lora.moe_route(x, r, k, renorm=renorm)
    ref_ids, ref_w = mx4_ref.route(x64, r64, k, renorm)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)
    # l - max rounded to fp32 (|l - max| 2^-24, at most 16 here), exp and the sum of E of them
    np.testing.assert_allclose(w.cpu().numpy(), ref_w, rtol=(40 + E) * 2.0 ** -24, atol=0)


@pytest.mark.parametrize("E,k", [(6, 4), (130, 8)])
def test_route_ties_go_to_the_lowest_index(E, k):
    x = torch.randn(9, 64, device="cuda").to(torch.bfloat16)
    r = torch.randn(1, 64, device="cuda").to(torch.bfloat16).expand(E, 64).contiguous()
    ids, w = lora.moe_route(x, r, k)
    assert ids.tolist() == [list(range(k))] * 9
    np.testing.assert_allclose(w.cpu().numpy(), 1.0 / k, rtol=2.0 ** -22)
    r[E - 1] = r[2] = 0  # both logits 0, above or below all the others
    ids, _ = lora.moe_route(x, r, k)
    ref, _ = mx4_ref.route(as64(x), as64(r), k, True)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref)


def test_route_nan():
    x = torch.randn(3, 64, device="cuda").to(torch.bfloat16)
    r = torch.randn(70, 64, device="cuda").to(torch.bfloat16)
    x[1, 5] = float("nan")
    ids, w = lora.moe_route(x, r, 5)
    assert ids[1].tolist() == [0, 1, 2, 3, 4] and bool(torch.isnan(w[1]).all())
    assert not bool(torch.isnan(w[[0, 2]]).any())
    x[1, 5] = 0
    r[65] = float("nan")  # one expert: never chosen while others are left
    ids, w = lora.moe_route(x, r, 5)
    assert not bool((ids == 65).any()) and not bool(torch.isnan(w).any())


EXPERTS = [(1, 64, 32, 4, 2), (1, 2056, 1000, 8, 2), (2, 264, 40, 3, 1), (7, 512, 264, 60, 4), (16, 256, 96, 2, 2),
           (20, 256, 72, 4, 3), (32, 512, 512, 16, 4), (64, 128, 64, 8, 8), (40, 8, 8, 5, 4), (512, 64, 32, 6, 1)]


@pytest.mark.parametrize("form", ["bf16", "mx4"])
@pytest.mark.parametrize("T,H,I,E,k", EXPERTS)
def test_layer(T, H, I, E, k, form):
    m = Moe(T, H, I, E, k, form, seed=T + I)
    ids, w = lora.moe_route(m.x, m.router, k)
    y = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    m.check(m.experts(ids, w, y=y), ids.cpu().numpy(), w.cpu().numpy())


@pytest.mark.parametrize("T,H,I,E,k", [(3, 264, 33, 4, 2), (9, 1032, 261, 7, 3)])
def test_odd_inner_width(T, H, I, E, k):
    m = Moe(T, H, I, E, k, "mx4", seed=I)
    ids, w = lora.moe_route(m.x, m.router, k, renorm=False)
    m.check(m.experts(ids, w), ids.cpu().numpy(), w.cpu().numpy())


@pytest.mark.parametrize("form", ["bf16", "mx4"])
def test_callers_choices(form):
    """Ids outside the experts add nothing, an expert may be named twice, and
    one expert may take every token; unreached experts are not read."""
    m = Moe(24, 256, 96, 6, 4, form, seed=4)
    g = np.random.default_rng(4)
    ids = g.integers(0, 3, (24, 4)).astype(np.int32)
    ids[0] = [2, 2, 2, 2]
    ids[1] = [-1, 6, 1 << 30, -(1 << 31)]
    ids[2:12] = 1
    w = g.standard_normal((24, 4)).astype(np.float32)
    for t in m.w:  # experts 3.. hold NaN
        if form == "bf16":
            t[3:] = float("nan")
        else:
            t.scales[3:] = 255
    y = m.experts(torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda())
    assert bool((y[1] == 0).all())
    m.check(y, ids, w)


@pytest.mark.parametrize("form", ["bf16", "mx4"])
def test_no_choice_at_all(form):
    m = Moe(3, 64, 32, 4, 2, form)
    y = torch.full((3, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    m.experts(torch.full((3, 2), -1, dtype=torch.int32, device="cuda"), torch.ones(3, 2, device="cuda"), y=y)
    assert bool((y == 0).all())


def test_nan_token_stays_in_its_row():
    m = Moe(12, 256, 64, 4, 2, "mx4")
    ids, w = lora.moe_route(m.x, m.router, 2)
    clean = m.experts(ids, w)
    x = m.x.clone()
    x[5, 100] = float("inf")
    y = m.experts(ids, w, x=x)
    keep = [t for t in range(12) if t != 5]
    assert torch.equal(y[keep], clean[keep])
    assert not bool(torch.isfinite(y[5]).all())


@pytest.mark.parametrize("form", ["bf16", "mx4"])
@pytest.mark.parametrize("T,H,I", [(1, 8, 8), (5, 40, 24), (70, 72, 40)])
def test_non_finite_weight_stays_in_its_row(T, H, I, form):
    """Rows that end inside a tile: an infinity at the start of a row does not
    reach the row before it."""
    m = Moe(T, H, I, 2, 1, form, seed=H)
    ids, w = torch.zeros((T, 1), dtype=torch.int32, device="cuda"), torch.ones((T, 1), device="cuda")
    clean = m.experts(ids, w)
    v = m.w[2] if form == "bf16" else lora.mx4_dequantize(m.w[2], "f32")
    v = v.clone()
    v[0, 3, 0] = float("inf")
    v[1, 0, 0] = float("inf")  # the row behind the last one of expert 0
    m.w[2] = v if form == "bf16" else lora.mx4_quantize(v)
    y = m.experts(ids, w)
    keep = [n for n in range(H) if n != 3]
    assert not bool(torch.isfinite(y[:, 3]).any())
    assert torch.equal(y[:, keep], clean[:, keep])
    v = (m.w[1] if form == "bf16" else lora.mx4_dequantize(m.w[1], "f32")).clone()
    v[0, 4, 0] = float("inf")  # one inner value: in every output, of expert 0 only
    m.w[1] = v if form == "bf16" else lora.mx4_quantize(v)
    assert not bool(torch.isfinite(m.experts(ids, w)).any())


def test_inner_value_at_the_types_edge():
    """An inner value that rounds past bf16's largest is an infinity, not a NaN."""
    H = I = 8
    x = torch.zeros((1, H), dtype=torch.bfloat16, device="cuda")
    x[0, 0] = 1.0
    gate, up, down = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((1, I, H), (1, I, H), (1, H, I)))
    gate[0, 0, 0] = 2.0 ** 7 * (1 + 2.0 ** -7)  # silu(g) = g: a product just under 2^128
    up[0, 0, 0] = 2.0 ** 120 * (2 - 2.0 ** -6)
    down[0, :, 0] = 1.0
    ids, w = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.ones((1, 1), device="cuda")
    y = lora.moe_experts(x, ids, w, gate, up, down)
    assert bool(torch.isinf(y).all())


def test_two_streams():
    """Layers on two streams at once share no workspace."""
    layers = [Moe(32, 512, 256, 64, 4, "mx4", seed=s) for s in (1, 2)]

    def layer(m):
        ids, w = lora.moe_route(m.x, m.router, 4)
        return lora.moe_experts(m.x, ids, w, *m.w)

    want = [layer(m) for m in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layer(layers[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


@pytest.mark.parametrize("form", ["bf16", "mx4"])
def test_same_bits_every_time(form):
    m = Moe(64, 512, 256, 8, 4, form)
    ids, w = lora.moe_route(m.x, m.router, 4)
    first = m.experts(ids, w)
    for _ in range(5):
        assert torch.equal(m.experts(ids, w), first)


def test_graph_replay():
    m = Moe(16, 512, 256, 16, 4, "mx4")
    x = m.x.clone()
    y = torch.empty_like(x)

    def layer(out=None):
        ids, w = lora.moe_route(x, m.router, 4)
        return lora.moe_experts(x, ids, w, *m.w, y=out)

    layer(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(y)
    for _ in range(4):
        x.copy_(torch.randn(16, 512, device="cuda").to(torch.bfloat16))
        want = layer()
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_refuses():
    m = Moe(4, 64, 32, 4, 2, "mx4")
    ids, w = lora.moe_route(m.x, m.router, 2)
    with pytest.raises(lora.LoraError):
        lora.moe_route(m.x, m.router, 5)
    with pytest.raises(lora.LoraError):
        lora.moe_route(m.x, m.router, 0)
    with pytest.raises(ValueError):
        lora.moe_route(m.x, m.router[:, :32].contiguous(), 2)
    with pytest.raises(ValueError):
        lora.moe_experts(m.x, ids, w, m.w[0], m.w[1], m.w[0])
    with pytest.raises(ValueError):
        lora.moe_experts(m.x, ids, w.double(), *m.w)
    with pytest.raises(ValueError):
        lora.moe_experts(m.x, ids, w, m.w[0], torch.zeros(4, 32, 64, dtype=torch.bfloat16, device="cuda"), m.w[2])
    with pytest.raises(lora.LoraError):
        lora.moe_experts(m.x, ids, w, *m.w, y=m.x)


def test_block_with_adapters():
    """The operators as a decode step runs them: a projection over a 4-bit
    base with each token's adapter, the experts over its output, and the
    layer's own adapters added to theirs."""
    T, H, I, E, k, S = 20, 512, 256, 8, 2, 4
    g = np.random.default_rng(11)
    m = Moe(T, H, I, E, k, "mx4", seed=11)
    ids = g.integers(0, S, T).astype(np.int32)
    plan = lora.plan(ids, S)
    pools, A, B = [], [], []
    for _ in range(2):
        pool = lora.Pool(S, 8, H, H, "bf16")
        As, Bs = [None], [None]
        for s in range(1, S):
            a, a64 = dev_bf16(g.standard_normal((8, H)) * H ** -0.5)
            b, b64 = dev_bf16(g.standard_normal((H, 8)) * 0.3)
            pool.install(s, a, b, 16.0)
            As.append(a64)
            Bs.append(b64)
        pools.append(pool)
        A.append(As)
        B.append(Bs)
    W = lora.mx4_quantize(torch.from_numpy((g.standard_normal((H, H)) * H ** -0.5).astype(np.float32)).cuda())
    W64 = lora.mx4_dequantize(W, "f32").cpu().numpy().astype(np.float64)
    h = lora.linear_mx4(m.x, W, pools[0], plan)
    e, w = lora.moe_route(h, m.router, k)
    moe = lora.moe_experts(h, e, w, *m.w)
    y = lora.correction(h, pools[1], plan, moe.clone())

    ref, lost = mx4_ref.linear(m.x64, W64, ids, A[0], B[0], [16.0] * S)
    assert (np.abs(as64(h) - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * lost).all()
    h64 = as64(h)
    ref_e, _ = mx4_ref.route(h64, m.router64, k, True)
    np.testing.assert_array_equal(e.cpu().numpy(), ref_e)
    ref, lost = mx4_ref.experts(h64, ref_e, as64(w), *m.w64)
    assert (np.abs(as64(moe) - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * lost).all()
    delta, lost = mx4_ref.linear(h64, np.zeros((H, H)), ids, A[1], B[1], [16.0] * S)
    ref = as64(moe) + delta
    assert (np.abs(as64(y) - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * lost).all()


@pytest.mark.parametrize("form", ["bf16", "mx4"])
def test_inner_value_past_the_largest_bf16(form):
    """An inner value of 2^128 - 2^114 (finite in fp32, over every finite bf16)
    times 2^-100 rounds to 2^28; a weight of 0 gives 0."""
    H = I = 8
    x = torch.zeros((1, H), dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[0, 1], x[0, 2] = 1.0, 2.0 ** -7, 2.0 ** -6
    gate, up, down = (torch.zeros(s, device="cuda") for s in ((1, I, H), (1, I, H), (1, H, I)))
    gate[0, 0, 0] = gate[0, 0, 1] = 2.0 ** 7                       # 2^7 (1 + 2^-7)
    up[0, 0, 0], up[0, 0, 2] = 2.0 ** 121, -(2.0 ** 120)           # 2^120 (2 - 2^-6)
    down[0, :4, 0] = 2.0 ** -100
    down[0, 4, 0] = -(2.0 ** -100)
    if form == "mx4":
        w = [lora.mx4_quantize(t) for t in (gate, up, down)]
        assert all(torch.equal(lora.mx4_dequantize(q, "f32"), t) for q, t in zip(w, (gate, up, down)))
    else:
        w = [t.to(torch.bfloat16) for t in (gate, up, down)]
    ids, one = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.ones((1, 1), device="cuda")
    y = lora.moe_experts(x, ids, one, *w)
    assert y[0].tolist() == [2.0 ** 28] * 4 + [-(2.0 ** 28)] + [0.0] * 3


@pytest.mark.parametrize("H", [64, 16384])
def test_route_products_past_fp32(H):
    """Logits whose products leave the range of fp32 on either side: one
    workgroup per token, and (a larger router) one wave per logit."""
    x = torch.zeros(2, H, dtype=torch.bfloat16, device="cuda")
    r = torch.zeros(6, H, dtype=torch.bfloat16, device="cuda")
    x[0, :3] = torch.tensor([2.0 ** 100, 2.0 ** 100, 1.0])
    r[0, :3] = torch.tensor([2.0 ** 100, -(2.0 ** 100), 5.0])  # 5: the first two cancel
    r[1, 2], r[2, 2], r[3, 2] = 7.0, 3.0, -1.0
    x[1, 3] = 2.0 ** -100
    r[4, 3], r[5, 3] = 2.0 ** -60, 2.0 ** -58  # tiny, and not alike
    ids, w = lora.moe_route(x, r, 3)
    assert ids.tolist() == [[1, 0, 2], [5, 4, 0]]
    want = np.exp(np.array([0.0, -2.0, -4.0]))
    np.testing.assert_allclose(w[0].cpu().numpy(), want / want.sum(), rtol=2.0 ** -20)
    np.testing.assert_allclose(w[1].cpu().numpy(), 1 / 3, rtol=2.0 ** -20)


def test_route_nan_logit_in_the_sum():
    """A NaN logit reaches a token's weights through the sum they are divided
    by: over all experts always, over the chosen ones only when it is chosen."""
    x = torch.randn(4, 64, device="cuda").to(torch.bfloat16)
    r = torch.randn(5, 64, device="cuda").to(torch.bfloat16)
    clean = lora.moe_route(x, r, 2)
    r[3] = float("nan")
    ids, w = lora.moe_route(x, r, 2, renorm=False)
    assert bool(torch.isnan(w).all()) and not bool((ids == 3).any())
    ids, w = lora.moe_route(x, r, 5)
    assert bool((ids[:, 4] == 3).all()) and bool(torch.isnan(w).all())
    ids, w = lora.moe_route(x, r, 2)
    assert not bool(torch.isnan(w).any())
    same = (clean[0] != 3).all(dim=1)  # tokens that did not choose it before
    assert torch.equal(ids[same], clean[0][same]) and torch.equal(w[same], clean[1][same])


def test_route_infinite_logit():
    """The largest logit infinite: exp(l - max) has no value. -inf elsewhere is a weight of 0."""
    x = torch.ones(2, 64, dtype=torch.bfloat16, device="cuda")
    x[1, 0] = 0.0
    r = torch.randn(4, 64, device="cuda").to(torch.bfloat16)
    r[2, 0] = float("inf")  # token 1: 0 * inf, a NaN
    ids, w = lora.moe_route(x, r, 4)
    assert ids[0, 0] == 2 and bool(torch.isnan(w).all()) and ids[1, 3] == 2
    x[1, 0] = 1.0
    r[2, 0] = float("-inf")
    ids, w = lora.moe_route(x, r, 4)
    assert bool((ids[:, 3] == 2).all()) and bool((w[:, 3] == 0).all())
    np.testing.assert_allclose(w.sum(dim=1).cpu().numpy(), 1.0, rtol=2.0 ** -20)


@pytest.mark.parametrize("T,k", [(16, 4), (33, 2), (5, 3)])
def test_lists_of_changing_choices(T, k):
    """Calls in a row whose choices change (the kernels' lists of an expert's
    pairs with them), on whole numbers: exact before the rounding of y."""
    H, I, E = 512, 64, 5
    g = torch.Generator(device="cuda").manual_seed(T)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(torch.bfloat16)

    x = ints(-3, 3, T, H)
    x[:, 0] = 2.0
    gate = torch.zeros(E, I, H, dtype=torch.bfloat16, device="cuda")
    gate[:, :, 0] = 64.0  # silu(128) = 128 to the last bit
    up, down = ints(-1, 1, E, I, H), ints(-1, 1, E, H, I)
    out = torch.stack([128.0 * (x.double() @ up[e].double().t()) @ down[e].double().t() for e in range(E)])
    assert float(out.abs().max()) * k < 2 ** 24
    one = torch.ones(T, k, device="cuda")
    for i in range(40):
        ids = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
        want = sum((ids == e).sum(dim=1, keepdim=True).double() * out[e] for e in range(E))
        assert torch.equal(lora.moe_experts(x, ids, one, gate, up, down), want.float().to(torch.bfloat16)), i
