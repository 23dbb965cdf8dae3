"""MXFP4 rows and the mixed-adapter linear layer over an MXFP4 base weight,
against plain 64-bit forms on the same inputs (tests/mx4_ref.py).

Quantisation is exact, so codes and scales are compared bit for bit. An
output of the layer is one rounding to bf16 (2^-8 of the value) away from sums
in fp32, whose loss the reference bounds from the magnitudes it adds up."""
import numpy as np
import pytest
import torch

from rank_gemm_amd import lora
from rank_gemm_amd.inputs import bf16_bits, bf16_to_f32
import mx4_ref

pytestmark = pytest.mark.gpu


def dev_bf16(v):
    """(device bf16 tensor, its fp64 values) of v rounded to bf16."""
    bits = bf16_bits(np.asarray(v, np.float32))
    return lora.to_device(bits, "bf16"), bf16_to_f32(bits).astype(np.float64)


def as64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def poisoned(n):
    """A workspace of n bytes whose every bf16 and fp32 is NaN."""
    return torch.full((max(int(n), 16),), 255, dtype=torch.uint8, device="cuda")


def check_quantized(q, v):
    codes, byte = mx4_ref.quantize(v)
    np.testing.assert_array_equal(q.scales.cpu().numpy(), mx4_ref.tiles(byte))
    np.testing.assert_array_equal(q.codes.cpu().numpy(), codes)
    return codes, byte


# -------------------------------------------------------------- quantise --
def test_quantize_every_bf16_pattern():
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    v = bf16_to_f32(bits)
    bits = bits[np.isfinite(v)]
    # neighbours of like magnitude (every code and tie), then shuffled ones
    order = np.argsort(np.abs(bf16_to_f32(bits)), kind="stable")
    shuffled = np.random.default_rng(0).permutation(len(bits))
    rows = np.concatenate([bits[order], bits[shuffled]])
    rows = rows[:len(rows) // 96 * 96].reshape(-1, 96)
    q = lora.mx4_quantize(lora.to_device(rows, "bf16"))
    codes, byte = check_quantized(q, bf16_to_f32(rows))
    got = lora.mx4_dequantize(q, "f32").cpu().numpy().astype(np.float64)
    np.testing.assert_array_equal(got, mx4_ref.values(codes, byte, 96).astype(np.float32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 32), (3, 31), (16, 33), (63, 64), (64, 255), (65, 256), (130, 257),
                                    (200, 1450), (2, 4096)])
def test_quantize_sizes(dtype, rows, K):
    g = np.random.default_rng(rows * 5000 + K)
    v = (g.standard_normal((rows, K)) * np.exp(g.standard_normal((rows, 1)) * 6)).astype(np.float32)
    v[g.random(v.shape) < 0.05] = 0.0
    if dtype == "bf16":
        src, v = dev_bf16(v)
    else:
        src = torch.from_numpy(v).cuda()
    q = lora.mx4_quantize(src)
    codes, byte = check_quantized(q, v)
    ref = mx4_ref.values(codes, byte, K)
    for out in ("f32", "bf16"):
        np.testing.assert_array_equal(as64(lora.mx4_dequantize(q, out)), ref)


def test_quantize_offset_source():
    """Rows whose storage starts off a 16-byte boundary."""
    buf = torch.randn(5 * 64 + 3, device="cuda").to(torch.bfloat16)
    src = buf[3:].view(5, 64)
    check_quantized(lora.mx4_quantize(src), as64(src))


def test_quantize_batch_and_reuse():
    v = torch.randn(3, 70, 100, device="cuda")
    q = lora.mx4_quantize(v)
    q2 = lora.mx4_quantize(v * 2, out=lora.Mx4.empty(v.shape))
    for b in range(3):
        one = lora.Mx4(q.codes[b].contiguous(), q.scales[b].contiguous(), 100)
        check_quantized(one, v[b].cpu().numpy())
    torch.testing.assert_close(lora.mx4_dequantize(q2, "f32"), 2 * lora.mx4_dequantize(q, "f32"), rtol=0, atol=0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_non_finite_block(dtype):
    v = torch.randn(4, 96, device="cuda").to(dtype)
    v[1, 40], v[2, 95], v[3, 0] = float("inf"), float("nan"), float("-inf")
    q = lora.mx4_quantize(v)
    check_quantized(q, as64(v))
    got = as64(lora.mx4_dequantize(q, "f32"))
    bad = np.zeros((4, 96), bool)
    bad[1, 32:64] = bad[2, 64:] = bad[3, :32] = True
    np.testing.assert_array_equal(np.isnan(got), bad)


def test_dequantize_every_code_and_scale():
    codes = np.tile(np.arange(256, dtype=np.uint8)[:, None] & 0, (1, 16))
    c = np.arange(16)
    codes[:, :8] = (c[0::2] | c[1::2] << 4).astype(np.uint8)
    byte = np.arange(256, dtype=np.uint8)[:, None]
    q = lora.mx4_pack(torch.from_numpy(codes).cuda(), torch.from_numpy(byte.copy()).cuda(), 32)
    ref = mx4_ref.values(codes, byte, 32)
    np.testing.assert_array_equal(q.scales.cpu().numpy(), mx4_ref.tiles(byte))
    np.testing.assert_array_equal(as64(lora.mx4_dequantize(q, "f32")), ref.astype(np.float32))
    want = torch.from_numpy(ref).float().bfloat16()  # exact but at the ends of the range
    np.testing.assert_array_equal(as64(lora.mx4_dequantize(q, "bf16")), as64(want))


def test_pack_equals_quantize():
    v = torch.randn(2, 150, 1000, device="cuda")
    q = lora.mx4_quantize(v)
    byte = np.stack([mx4_ref.quantize(v[b].cpu().numpy())[1] for b in range(2)])
    p = lora.mx4_pack(q.codes, torch.from_numpy(byte).cuda(), 1000)
    assert torch.equal(p.scales, q.scales)


def test_quantize_past_32_bits():
    """4.3 G values: row and element offsets beyond 2^32."""
    rows, K = (1 << 20) + 3, 4104
    src = torch.ones((rows, K), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(70, K, device="cuda").to(torch.bfloat16)
    src[-70:] = tail
    q = lora.mx4_quantize(src)
    del src
    want = lora.mx4_quantize(tail)
    assert torch.equal(q.codes[-70:], want.codes)
    assert bool((q.codes[:5, :K // 2] == 0x66).all())  # 4 * 2^-2
    out = lora.mx4_dequantize(q, "bf16")
    assert torch.equal(out[-70:], lora.mx4_dequantize(want, "bf16"))
    assert bool((out[:-70].amin() == 1) & (out[:-70].amax() == 1))


# ---------------------------------------------------------------- linear --
class Layer:
    """One random layer: pool, 4-bit base weight, and their fp64 values."""

    def __init__(self, T, d_in, d_out, ranks, seed=0, r_max=None, ids=None):
        g = np.random.default_rng(seed)
        self.S = len(ranks)
        self.T, self.d_in, self.d_out = T, d_in, d_out
        self.x, self.x64 = dev_bf16(g.standard_normal((T, d_in)))
        Wv = g.standard_normal((d_out, d_in)) * d_in ** -0.5
        codes, byte = mx4_ref.quantize(Wv.astype(np.float32))
        self.W64 = mx4_ref.values(codes, byte, d_in)
        self.W = lora.mx4_pack(torch.from_numpy(codes).cuda(), torch.from_numpy(byte).cuda(), d_in)
        self.pool = lora.Pool(self.S, r_max or max(max(ranks), 1), d_in, d_out, "bf16")
        self.A, self.B, self.alpha = [None] * self.S, [None] * self.S, [0.0] * self.S
        for s in range(1, self.S):
            if ranks[s] == 0:
                continue
            a, self.A[s] = dev_bf16(g.standard_normal((ranks[s], d_in)) * d_in ** -0.5)
            b, self.B[s] = dev_bf16(g.standard_normal((d_out, ranks[s])) * 0.3)
            self.alpha[s] = 16.0 + s
            self.pool.install(s, a, b, self.alpha[s])
        self.ids = g.integers(0, self.S, T).astype(np.int32) if ids is None else np.asarray(ids, np.int32)

    def run(self, act, plan=None, x=None, y=None):
        plan = plan or lora.plan(self.ids, self.S)
        n = lora.lib().lora_workspace_bytes_mx4(self.pool.handle, self.T, lora._ACT[act])
        return lora.linear_mx4(self.x if x is None else x, self.W, self.pool, plan, act=act, y=y,
                               workspace=poisoned(n))

    def check(self, y, act, ids=None):
        base = None
        if act == "mx4":
            base = mx4_ref.values(*mx4_ref.quantize(self.x64), self.d_in)
        ref, lost = mx4_ref.linear(self.x64, self.W64, self.ids if ids is None else ids, self.A, self.B, self.alpha,
                                   base)
        err = np.abs(as64(y) - ref)
        bound = 2.0 ** -8 * np.abs(ref) + 1.01 * lost
        worst = float((err / bound).max())
        print(f"T={self.T} {self.d_in}->{self.d_out} act={act}: worst error {worst:.3f} of its bound", flush=True)
        assert worst <= 1.0, f"{int((err > bound).sum())} elements out of bound, worst {worst}"


SHAPES = [
    # T, d_in, d_out, ranks, r_max
    (1, 256, 64, [0, 16], None),
    (1, 4096, 1024, [0, 16, 8], None),
    (5, 64, 33, [0, 4, 0, 3], 7),
    (16, 512, 300, [0, 16, 8, 32], None),
    (17, 1000, 129, [0, 8, 8], 12),
    (48, 2048, 1000, [0, 16] * 4, None),
    (64, 288, 640, [0, 64, 16, 1], None),
    (65, 4088, 256, [0, 16, 16, 16], None),
    (100, 33, 50, [0, 8, 5], None),
    (130, 1001, 77, [0, 16, 4], None),
    (300, 768, 1030, [0, 16, 0, 32], None),
    (333, 4088, 1021, [0, 32, 16, 8, 32, 16], None),
    (1000, 512, 2048, [0] + [16] * 16, None),
    (700, 1288, 4096, [0] + [12] * 3, None),
    (520, 320, 8200, [0, 100, 8], None),
    (520, 256, 8200, [0, 16, 8], None),
    (64, 512, 14337, [0, 16, 8, 32, 0, 1], 32),
    (50, 2304, 14336, [0] + [16] * 16, None),
    (250, 512, 8200, [0] + [8, 24, 3] * 20, 24),
    (64, 256, 14336, [0, 16] * 33, None),
    (300, 8200, 300, [0, 16, 0, 8], None),
    (700, 8192, 1100, [0, 8, 24], None),
    (1500, 520, 3100, [0, 16, 64], None),
    (3601, 288, 3500, [0, 16, 8, 0, 64], None),
    (3600, 512, 3591, [0] + [16] * 16, None),
    (3400, 264, 3900, [0, 12, 4], None),
    (768, 520, 1290, [0, 16, 8], None),
    (769, 8200, 1500, [0, 16, 8], None),
    (1030, 14336, 1100, [0, 16, 0, 8], None),
    (1100, 520, 1300, [0, 16] * 40, None),
    (1600, 72, 100, [0, 5, 16], None),
    (4000, 264, 2104, [0, 12, 4, 0, 9], 13),
    (600, 264, 4100, [0, 12, 4, 0, 9], 12),
    (260, 520, 8200, [0, 64, 40, 4, 33], 64),
    (300, 4104, 4096, [0, 44, 20, 3] * 15, 44),
    (64, 320, 14336, [0, 4, 2], 4),
]


@pytest.mark.parametrize("act", ["bf16", "mx4"])
@pytest.mark.parametrize("T,d_in,d_out,ranks,r_max", SHAPES)
def test_linear(T, d_in, d_out, ranks, r_max, act):
    L = Layer(T, d_in, d_out, ranks, seed=T + d_in, r_max=r_max)
    y = torch.full((T, d_out), float("nan"), dtype=torch.bfloat16, device="cuda")
    L.check(L.run(act, y=y), act)


@pytest.mark.parametrize("act", ["bf16", "mx4"])
@pytest.mark.parametrize("T,d_out", [(3, 200), (40, 4096), (400, 1024), (2048, 4096)])
def test_base_rows_equal_base_only(act, T, d_out):
    """Rows on slot 0 or on an empty slot: the bits of a base-only call."""
    L = Layer(T, 512, d_out, [0, 16, 0, 8], seed=T)
    y = L.run(act)
    base = L.run(act, plan=lora.plan(np.zeros(T, np.int32), L.S))
    L.check(base, act, ids=np.zeros(T, np.int32))
    rows = torch.from_numpy(np.flatnonzero((L.ids == 0) | (L.ids == 2))).cuda()
    assert torch.equal(y[rows], base[rows])


@pytest.mark.parametrize("act", ["bf16", "mx4"])
@pytest.mark.parametrize("T", [1, 33, 600])
def test_device_plan(act, T):
    L = Layer(T, 640, 520, [0, 16, 8, 24], seed=T)
    dp = lora.plan_device(torch.from_numpy(L.ids).cuda(), L.S)
    L.check(L.run(act, plan=dp), act)


@pytest.mark.parametrize("act", ["bf16", "mx4"])
@pytest.mark.parametrize("T", [8, 300])
def test_nan_row_stays_in_its_row(act, T):
    L = Layer(T, 320, 96, [0, 8, 8], seed=T)
    clean = L.run(act)
    x = L.x.clone()
    x[T // 2, 17] = float("nan")
    y = L.run(act, x=x)
    assert bool(torch.isnan(y[T // 2]).all())
    keep = [t for t in range(T) if t != T // 2]
    assert torch.equal(y[keep], clean[keep])


def test_nan_scale_of_a_weight_row():
    """A weight block without a scale gives NaN in its column and nowhere else."""
    for T in (4, 300):
        L = Layer(T, 320, 96, [0, 8], seed=1)
        v = lora.mx4_dequantize(L.W, "f32")
        v[40, 33] = float("nan")
        W = lora.mx4_quantize(v)
        clean = {a: L.run(a) for a in ("bf16", "mx4")}
        L.W = W
        for a in ("bf16", "mx4"):
            y = L.run(a)
            assert bool(torch.isnan(y[:, 40]).all())
            keep = [n for n in range(96) if n != 40]
            assert torch.equal(y[:, keep], clean[a][:, keep])


@pytest.mark.parametrize("act", ["bf16", "mx4"])
def test_empty_batch(act):
    L = Layer(0, 64, 32, [0, 8], ids=[])
    assert lora.linear_mx4(L.x, L.W, L.pool, lora.plan(L.ids, L.S), act=act).shape == (0, 32)


@pytest.mark.parametrize("act", ["bf16", "mx4"])
@pytest.mark.parametrize("T", [24, 600])
def test_graph_replay(act, T):
    """Captured once, replayed with other inputs and other slot ids between
    eager work, each replay equal to the eager call."""
    L = Layer(T, 512, 384, [0, 16, 8], seed=T)
    ids = torch.from_numpy(L.ids).cuda()
    x = L.x.clone()
    y = torch.empty((T, 384), dtype=torch.bfloat16, device="cuda")
    lora.linear_mx4(x, L.W, L.pool, lora.plan_device(ids, L.S), act=act, y=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lora.linear_mx4(x, L.W, L.pool, lora.plan_device(ids, L.S), act=act, y=y)
    g = np.random.default_rng(3)
    for _ in range(4):
        x.copy_(torch.randn(T, 512, device="cuda").to(torch.bfloat16))
        ids.copy_(torch.from_numpy(g.integers(0, L.S, T).astype(np.int32)).cuda())
        want = lora.linear_mx4(x, L.W, L.pool, lora.plan_device(ids, L.S), act=act)
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_two_streams():
    """Calls on two streams at once do not share a workspace."""
    layers = [Layer(64, 1024, 2048, [0, 16, 8], seed=s) for s in (1, 2)]
    plans = [lora.plan(L.ids, L.S) for L in layers]
    want = [lora.linear_mx4(L.x, L.W, L.pool, p, act="mx4") for L, p in zip(layers, plans)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(lora.linear_mx4(layers[i].x, layers[i].W, layers[i].pool, plans[i], act="mx4"))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_linear_refuses():
    L = Layer(8, 64, 32, [0, 8])
    p = lora.plan(L.ids, L.S)
    with pytest.raises(ValueError):
        lora.linear_mx4(L.x, L.W, L.pool, p, act="fp8")
    with pytest.raises(ValueError):
        lora.linear_mx4(L.x, lora.Mx4.empty((32, 96)), L.pool, p)
    with pytest.raises(ValueError):
        lora.linear_mx4(L.x.float(), L.W, L.pool, p)
    with pytest.raises(ValueError):
        lora.linear_mx4(L.x, L.W, lora.Pool(2, 4, 64, 32, "f32"), p)
    with pytest.raises(lora.LoraError):  # plan and pool of different S
        lora.linear_mx4(L.x, L.W, L.pool, lora.plan(np.zeros(8, np.int32), 5))
    with pytest.raises(lora.LoraError):
        lora.linear_mx4(L.x, L.W, L.pool, p, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(lora.LoraError):  # rows of x off a 16-byte boundary
        lora.linear_mx4(torch.zeros(8 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(8, 64), L.W, L.pool, p)
    f32 = lora.Pool(2, 4, 64, 32, "f32")
    assert lora.lib().lora_workspace_bytes_mx4(f32.handle, 8, lora.LORA_MX4) == 0
    assert lora.lib().lora_workspace_bytes_mx4(L.pool.handle, 8, 0) == 0


def test_linear_refuses_sizes():
    d_in = 4194248  # a row past what the scale tiles' grid takes
    pool = lora.Pool(2, 1, d_in, 8, "bf16")
    for act in ("bf16", "mx4"):
        assert lora.lib().lora_workspace_bytes_mx4(pool.handle, 1, lora._ACT[act]) == 0
        with pytest.raises(lora.LoraError):
            lora.linear_mx4(torch.zeros(1, d_in, dtype=torch.bfloat16, device="cuda"), lora.Mx4.empty((8, d_in)), pool,
                            lora.plan(np.zeros(1, np.int32), 2), act=act)


@pytest.mark.parametrize("act", ["bf16", "mx4"])
@pytest.mark.parametrize("T", [3, 40, 1500])
def test_scales_on_an_8_byte_boundary(act, T):
    L = Layer(T, 520, 1100, [0, 16, 8], seed=T)
    clean = L.run(act)
    n = L.W.scales.numel()
    moved = torch.empty(n + 8, dtype=torch.uint8, device="cuda")[8:]
    moved.copy_(L.W.scales)
    assert moved.data_ptr() % 16 == 8
    L.W = lora.Mx4(L.W.codes, moved, 520)
    assert torch.equal(L.run(act), clean)


@pytest.mark.parametrize("T", [20, 700])
def test_two_graphs_with_a_workspace_each(T):
    """Two captured calls, replayed in turn and after one another, with the
    eager call between them."""
    L = [Layer(T, 512, 768, [0, 16, 8], seed=s) for s in (3, 4)]
    plans = [lora.plan(m.ids, m.S) for m in L]
    ys = [torch.empty((T, 768), dtype=torch.bfloat16, device="cuda") for _ in L]
    graphs = []
    for m, p, y in zip(L, plans, ys):
        lora.linear_mx4(m.x, m.W, m.pool, p, act="mx4", y=y)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            lora.linear_mx4(m.x, m.W, m.pool, p, act="mx4", y=y)
    want = [lora.linear_mx4(m.x, m.W, m.pool, p, act="mx4") for m, p in zip(L, plans)]
    for _ in range(3):
        for y in ys:
            y.fill_(float("nan"))
        for g in graphs:
            g.replay()
        assert torch.equal(lora.linear_mx4(L[0].x, L[0].W, L[0].pool, plans[0], act="mx4"), want[0])
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for y, w in zip(ys, want))
