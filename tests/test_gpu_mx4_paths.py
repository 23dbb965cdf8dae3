"""The layer over an MXFP4 base weight and the experts on every path: whole
numbers, whose sums are exact, so that y is compared bit for bit over long K;
scales at the ends of their range; operands past 2 and 4 GiB."""
import numpy as np
import pytest
import torch

from rank_gemm_amd import lora
import mx4_ref

pytestmark = pytest.mark.gpu

# T, d_in, d_out: K split over workgroups (64 and 128 columns), wide and few
# blocks, decoded W (unsplit, split over K), 4-bit tiles of each shape
LONG = [(1, 14336, 4096), (16, 14336, 1000), (40, 14336, 4096), (64, 8200, 14400), (333, 14336, 1021),
        (512, 14336, 4096), (700, 12000, 4096), (1030, 14336, 1100), (2048, 14336, 4096), (2100, 8192, 1300),
        (300, 4099, 700), (1500, 4099, 1300)]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(torch.bfloat16)


class Whole:
    """A layer of whole numbers. x of -3 .. 3 and W of -1 .. 1 are MXFP4 values
    themselves, so both forms of the activations give the same y. Sums stay
    under 2^22 (asserted), corrections are multiples of a quarter: fp32 holds
    every partial sum in any order, and scaled h in bf16 hi + lo."""

    def __init__(self, T, d_in, d_out, ranks, r_max=None, seed=0):
        g = gen(seed)
        self.S = len(ranks)
        self.x, W = ints(g, -3, 3, T, d_in), ints(g, -1, 1, d_out, d_in)
        self.W = lora.mx4_quantize(W)
        self.pool = lora.Pool(self.S, r_max or max(ranks), d_in, d_out, "bf16")
        self.ids = np.random.default_rng(seed).integers(0, self.S, T).astype(np.int32)
        self.A, self.B = [None] * self.S, [None] * self.S
        for s in range(1, self.S):
            if ranks[s]:
                self.A[s], self.B[s] = ints(g, -1, 1, ranks[s], d_in), ints(g, -1, 1, d_out, ranks[s])
                self.pool.install(s, self.A[s], self.B[s], ranks[s] / 4)
        self.W16 = W

    def want(self, rows=None):
        """Exact y of the given rows (or of all), rounded once."""
        rows = torch.arange(len(self.ids), device="cuda") if rows is None else rows
        x = self.x[rows].double()
        ids = torch.from_numpy(self.ids).cuda()[rows]
        y = x @ self.W16.double().t()
        for s in range(1, self.S):
            on = (ids == s).nonzero().flatten()
            if self.A[s] is not None and on.numel():
                h = x[on] @ self.A[s].double().t()
                assert float(h.abs().max()) < 2 ** 16
                y[on] += 0.25 * (h @ self.B[s].double().t())
        assert float(y.abs().max()) < 2 ** 22
        return y.float().to(torch.bfloat16)


@pytest.mark.parametrize("act", ["bf16", "mx4"])
@pytest.mark.parametrize("ranks,r_max", [([0, 16, 0, 32, 8], None), ([0, 12, 4, 9], 12), ([0, 64, 40, 7], 64)])
@pytest.mark.parametrize("T,d_in,d_out", LONG)
def test_whole_numbers_are_exact(T, d_in, d_out, ranks, r_max, act):
    L = Whole(T, d_in, d_out, ranks, r_max, seed=T + d_in)
    want = L.want()
    for plan in (lora.plan(L.ids, L.S), lora.plan_device(torch.from_numpy(L.ids).cuda(), L.S)):
        assert torch.equal(lora.linear_mx4(L.x, L.W, L.pool, plan, act=act), want)


@pytest.mark.parametrize("form", ["bf16", "mx4"])
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (20, 6, 4), (64, 9, 3)])
def test_experts_of_whole_numbers(T, E, k, form):
    """gate of one large column, so that silu(g) = g to the last bit: the inner
    values are whole numbers under 2^16, and y is exact before its rounding."""
    H, I = 4104, 1544
    g = gen(T + E)
    x = ints(g, -3, 3, T, H)
    x[:, 0] = 2.0
    gate = torch.zeros(E, I, H, dtype=torch.bfloat16, device="cuda")
    gate[:, :, 0] = 64.0  # g = 128: expf(-128) is under half a step of 1
    up, down = ints(g, 0, 1, E, I, H), ints(g, -1, 1, E, H, I)
    up[:, :, 1:] *= (torch.rand(E, I, H - 1, generator=g, device="cuda") < 0.02).to(torch.bfloat16)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.ones(T, k, device="cuda") * torch.tensor([1.0, 0.5, 0.25, 2.0], device="cuda")[:k]
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        a = 128.0 * (x.double() @ up[e].double().t())
        assert float((a / 128).abs().max()) < 2 ** 9  # 16 bits of mantissa hold it
        out = a @ down[e].double().t()
        assert float(out.abs().max()) < 2 ** 22
        want += (w * (ids == e)).sum(dim=1, keepdim=True).double() * out
    if form == "mx4":
        gate, up, down = (lora.mx4_quantize(t) for t in (gate, up, down))
    y = lora.moe_experts(x, ids, w, gate, up, down)
    assert torch.equal(y, want.float().to(torch.bfloat16))


# one shape a path: K split, 128 columns a workgroup, decoded W, 4-bit tiles
PATHS = [(3, 520, 200), (40, 520, 200), (1500, 520, 1300)]


@pytest.mark.parametrize("act", ["bf16", "mx4"])
@pytest.mark.parametrize("T,d_in,d_out", PATHS)
def test_scales_at_the_ends_of_their_range(T, d_in, d_out, act):
    """Rows of W whose blocks have a scale byte near 0 or 254 (values within
    bf16's range), rows of x as far on the other side: each y whose terms are
    normal fp32 numbers is one rounding from its exact value."""
    g = np.random.default_rng(T)
    edge = np.array([0, 1, 2, 3, 30, 127, 220, 251, 252, 253, 254])
    byte = np.repeat(edge[g.integers(0, len(edge), (d_out, 1))], -(-d_in // 32), axis=1).astype(np.uint8)
    top = np.where(byte[:, :1] == 254, 4, np.where(byte[:, :1] == 253, 6, 8))  # 1.5 2^127 at most
    c = g.integers(1, 8, (d_out, d_in)) % top
    c += (c == 0) + 8 * g.integers(0, 2, c.shape)
    c = np.pad(c.astype(np.uint8), ((0, 0), (0, byte.shape[1] * 32 - d_in))).reshape(d_out, -1, 2)
    codes = c[:, :, 0] | c[:, :, 1] << 4
    W = mx4_ref.values(codes, byte, d_in)
    q = lora.mx4_pack(torch.from_numpy(codes).cuda(), torch.from_numpy(byte).cuda(), d_in)
    power = np.array([-100, 0, 110, -122, -40, 40, 124])[np.arange(T) % 7][:, None]
    # 1, 1.5, 2 and 3 of one power: MXFP4 values
    x = g.choice([1.0, 1.5, 2.0, 3.0, -1.0, -1.5, -2.0, -3.0], (T, d_in)) * 2.0 ** power
    x[:, ::32] = 3.0 * 2.0 ** power
    pool = lora.Pool(2, 4, d_in, d_out, "bf16")
    xd = torch.from_numpy(x).float().to(torch.bfloat16).cuda()
    np.testing.assert_array_equal(xd.double().cpu().numpy(), x)
    y = lora.linear_mx4(xd, q, pool, lora.plan(np.zeros(T, np.int32), 2), act=act)
    e = power + byte[:, 0].astype(int)[None, :] - 127  # terms lie between 2^(e - 1) and 18 2^e
    fine = (e > -120) & (e < 110)
    assert fine.any(axis=0).all()
    ref = x @ W.T
    # fp32 sums of d_in terms, then one rounding
    bound = 2.0 ** -8 * np.abs(ref) + 2 * (d_in + 64) * 2.0 ** -24 * (np.abs(x) @ np.abs(W).T)
    err = np.abs(y.double().cpu().numpy() - ref)
    bad = fine & ~(err <= bound)
    assert not bad.any(), f"{bad.sum()} of {fine.sum()}, scale bytes {sorted(set(byte[bad.any(axis=0), 0].tolist()))}"


@pytest.mark.parametrize("T,d_in,d_out", PATHS)
def test_weights_past_the_largest_bf16(T, d_in, d_out):
    """Scale bytes 252 .. 254 with every code: with 16-bit activations a value
    past bf16's range is the infinity that dequantising gives, with 4-bit ones
    the product is of the value itself."""
    byte = np.full((d_out, -(-d_in // 32)), 127, np.uint8)
    byte[:, 0] = 254 - np.arange(d_out) // 16 % 3
    codes = np.zeros((d_out, byte.shape[1] * 16), np.uint8)
    codes[:, 0] = np.arange(d_out) % 16  # the first value of each row
    q = lora.mx4_pack(torch.from_numpy(codes).cuda(), torch.from_numpy(byte).cuda(), d_in)
    x = torch.zeros(T, d_in, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 2.0 ** -100
    pool = lora.Pool(2, 4, d_in, d_out, "bf16")
    plan = lora.plan(np.zeros(T, np.int32), 2)
    exact = mx4_ref.values(codes, byte, d_in)[:, 0]
    as_bf16 = lora.mx4_dequantize(q, "bf16")[:, 0].double().cpu().numpy()
    np.testing.assert_array_equal(as_bf16, np.where(np.abs(exact) < 2.0 ** 128, exact, np.copysign(np.inf, exact)))
    for act, w in (("bf16", as_bf16), ("mx4", exact)):
        y = lora.linear_mx4(x, q, pool, plan, act=act).double().cpu().numpy()
        np.testing.assert_array_equal(y, np.broadcast_to(w * 2.0 ** -100, y.shape))


@pytest.mark.parametrize("act", ["bf16", "mx4"])
@pytest.mark.parametrize("T,d_in,d_out", PATHS)
def test_nan_stays_in_its_row_and_column(T, d_in, d_out, act):
    L = Whole(T, d_in, d_out, [0, 16, 8], seed=T)
    plan = lora.plan(L.ids, L.S)
    clean = lora.linear_mx4(L.x, L.W, L.pool, plan, act=act)
    W = L.W16.float()
    W[100, d_in - 1] = float("nan")
    x = L.x.clone()
    x[T // 2, 40] = float("nan")
    y = lora.linear_mx4(x, lora.mx4_quantize(W), L.pool, plan, act=act)
    rows = [t for t in range(T) if t != T // 2]
    cols = [n for n in range(d_out) if n != 100]
    assert bool(torch.isnan(y[T // 2]).all()) and bool(torch.isnan(y[:, 100]).all())
    assert torch.equal(y[rows][:, cols], clean[rows][:, cols])


@pytest.mark.parametrize("act", ["bf16", "mx4"])
def test_rows_past_2_gib(act):
    """x of 8.6 GB, its codes and the expand operand's rows past 2^31 bytes."""
    T, d_in, d_out = (1 << 20) + 35, 4104, 264
    L = Whole(T, d_in, d_out, [0, 16, 8], seed=5)
    rows = torch.cat([torch.arange(70), torch.randint(0, T, (300,), generator=torch.Generator().manual_seed(1)),
                      torch.arange(T - 70, T)]).cuda()
    y = torch.full((T, d_out), float("nan"), dtype=torch.bfloat16, device="cuda")
    lora.linear_mx4(L.x, L.W, L.pool, lora.plan(L.ids, L.S), act=act, y=y)
    assert torch.equal(y[rows], L.want(rows))
    assert not bool(torch.isnan(y).any())


@pytest.mark.parametrize("form", ["bf16", "mx4"])
def test_experts_past_4_gib(form):
    """Batches of experts past 2^32 bytes: the first and the last expert."""
    H = I = 8192
    E = 36 if form == "bf16" else 140
    g = gen(9)
    w, w64 = [], []
    for _ in range(3):
        if form == "bf16":
            t = torch.empty(E, H, H, dtype=torch.bfloat16, device="cuda").normal_(0.0, H ** -0.5, generator=g)
            assert t.numel() * 2 > 1 << 32
            v = t[[0, E - 1]]
        else:
            codes = torch.randint(0, 256, (E, H, H // 2), generator=g, device="cuda", dtype=torch.uint8)
            scales = torch.randint(117, 121, (E, lora.lib().lora_mx4_scale_bytes(H, H)), generator=g, device="cuda",
                                   dtype=torch.uint8)
            assert codes.numel() > 1 << 32
            t = lora.Mx4(codes, scales, H)
            v = lora.mx4_dequantize(lora.Mx4(codes[[0, E - 1]], scales[[0, E - 1]], H), "f32")
        w.append(t)
        w64.append(v.double().cpu().numpy())
    T = 3
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.tensor([[0, E - 1], [E - 1, E], [E - 1, 0]], dtype=torch.int32, device="cuda")
    wt = torch.tensor([[0.5, 0.25], [1.0, 3.0], [0.75, 0.5]], device="cuda")
    y = lora.moe_experts(x, ids, wt, *w).double().cpu().numpy()
    local = np.array([[0, 1], [1, 2], [1, 0]], np.int32)
    ref, lost = mx4_ref.experts(x.double().cpu().numpy(), local, wt.double().cpu().numpy(), *w64)
    assert (np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * lost).all()
