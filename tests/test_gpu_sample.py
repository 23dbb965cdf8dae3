"""Sampling against its 64-bit form (tests/decode_ref.py): tokens exactly,
probabilities within one fp32 rounding (2^-24) and what weights held as whole
numbers of 2^-shift lose of their sum (V 2^-(shift + 1), under 2^-26)."""
import numpy as np
import pytest
import torch

from rank_gemm_amd import lora
import decode_ref

pytestmark = pytest.mark.gpu

RTOL = 2.0 ** -24 + 2.0 ** -26


def own(values, dtype):
    return None if values is None else torch.tensor(values, dtype=dtype, device="cuda")


def check(x, u, t=None, k=None, p=None, least=None):
    B = x.shape[0]
    ids, probs = lora.sample(x, own(u, torch.float64), own(t, torch.float32), own(k, torch.int32),
                             own(p, torch.float32), own(least, torch.float32))
    rows = x.detach().float().cpu().numpy()
    f32 = np.float32

    def of(v, i, off):
        return off if v is None else float(f32(v[i]))

    for b in range(B):
        want, prob = decode_ref.sample(rows[b], u[b], of(t, b, 1.0), 0 if k is None else k[b], of(p, b, 1.0),
                                       of(least, b, 0.0))
        assert (int(ids[b]), b) == (want, b)
        np.testing.assert_allclose(float(probs[b]), prob, rtol=RTOL, atol=1e-37)
    return ids, probs


def logits(B, V, dtype, seed=0, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = spread * torch.randn(B, V, generator=g, device="cuda")
    return (x + 8.0 * (torch.rand(B, V, generator=g, device="cuda") < 8.0 / V)).to(dtype)


SIZES = [(1, 1), (3, 2), (2, 7), (5, 63), (4, 64), (4, 65), (3, 1000), (9, 1024), (2, 4097), (7, 50021), (2, 131072),
         (1, 262144)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,V", SIZES)
def test_filters(B, V, dtype):
    g = np.random.default_rng(B + V)
    x = logits(B, V, dtype, B)
    u = g.random(B).tolist()
    t = g.choice([0.5, 0.8, 1.0, 1.7], B).tolist()
    k = g.choice([1, 2, 5, 40, V // 2 + 1, V], B).tolist()
    p = g.choice([0.05, 0.5, 0.9, 0.99], B).tolist()
    least = g.choice([0.0, 1e-4, 0.02, 0.5], B).tolist()
    check(x, u)
    check(x, u, t=t)
    check(x, u, t=t, k=k)
    check(x, u, t=t, p=p)
    check(x, u, t=t, least=least)
    check(x, u, k=k, p=p)
    check(x, u, t=t, k=k, p=p, least=least)


def test_largest_vocabulary():
    """Sums over 8192 tiles, and borders among millions of equal logits."""
    V = 4194304
    x = logits(4, V, torch.bfloat16, 30)
    x[2] = 1.5
    x[3, ::2] = -2.0
    check(x, [0.3, 0.9, 0.5, 0.999], k=[0, 100, 3000001, 0], p=[0.7, 0.9, 0.5, 0.99], t=[1.0, 0.7, 1.0, 2.0])
    check(x, [0.1, 0.6, 0.7, 0.2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_rows_of_few_numbers(dtype):
    """Infinite logits, the type's lowest value and many close ones, over more
    tokens than one workgroup ranks."""
    V = 20001
    g = torch.Generator(device="cuda").manual_seed(31)
    x = torch.randn(6, V, generator=g, device="cuda")
    x[0, ::3] = float("inf")
    x[1] = torch.finfo(dtype).min
    x[1, 5::7] = x[2, 5::7]
    x[2] = x[2] * 1e-4 + 3.0
    x[3, 100:] = torch.finfo(dtype).min
    x[4] = torch.where(x[4] > 0, 2.0, -float("inf"))
    x[5] *= 1e30
    x = x.to(dtype)
    u = [0.1, 0.35, 0.6, 0.85, 0.999, 0.5]
    check(x, u)
    check(x, u, k=[5000, 1500, 9000, 150, 4000, 3])
    check(x, u, p=[0.2, 0.9, 0.6, 0.95, 0.5, 0.9])
    check(x, u, k=[5000, 1500, 9000, 150, 4000, 3], p=[0.2, 0.9, 0.6, 0.95, 0.5, 0.9], t=[1.0, 0.5, 1.0, 2.0, 1.0, 1e30])
    check(x, u, least=[0.5, 0.1, 0.9, 0.3, 1.0, 0.5])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [5, 700, 30000])
def test_equal_logits(V, dtype):
    """All logits equal, and few different values: the borders of the filters
    fall among equal logits, where the lower indices stay."""
    B = 6
    g = np.random.default_rng(V)
    u = [0.0, 0.2, 0.5, 0.9, 0.999999, 1.0 - 2.0 ** -53]
    flat = torch.full((B, V), -3.5, dtype=dtype, device="cuda")
    steps = torch.from_numpy(g.integers(0, 4, (B, V)).astype(np.float32)).cuda().to(dtype)
    for x in (flat, steps):
        check(x, u)
        check(x, u, k=[1, 2, 3, V // 3 + 1, V - 1, V])
        check(x, u, p=[0.1, 0.25, 0.5, 0.75, 0.9, 0.999])
        check(x, u, k=[3, 3, V // 2 + 1, V - 1, V, V + 5], p=[0.3, 0.9, 0.4, 0.6, 0.7, 0.2], t=[0.3, 1.0, 2.0, 9.0, 1.0, 0.1])
        check(x, u, least=[0.0, 0.1, 0.3, 0.5, 1.0, 2.0], t=[1.0, 0.7, 1.0, 1.0, 1.0, 1.0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ends_of_the_parameters(dtype):
    x = logits(12, 900, dtype, 3)
    inf, nan = float("inf"), float("nan")
    u = np.random.default_rng(0).random(12).tolist()
    check(x, u, t=[0.0, -1.0, nan, 1e-30, 1e-45, 1e30, 3e38, inf, 1e-3, 1.0, 1.0, 1.0])
    check(x, u, k=[0, -1, -2 ** 31, 2 ** 31 - 1, 900, 899, 1, 2, 901, 3, 4, 5])
    check(x, u, p=[0.0, -1.0, 1.0, 1.5, nan, inf, -inf, 1e-30, 0.9999999, 0.5, 0.5, 0.5])
    check(x, u, least=[0.0, -1.0, 1.0, 1.5, nan, inf, -inf, 1e-30, 0.9999999, 0.5, 0.5, 0.5])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_logits(dtype):
    """Masks as servers write them: -infinity, the type's lowest value, NaN;
    rows of nothing else; infinite logits."""
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(dtype).min
    x = logits(12, 700, dtype, 4)
    x[0, 5:] = -inf
    x[1] = -inf
    x[2] = nan
    x[3, ::2] = nan
    x[4, 1:] = low
    x[5] = low
    x[6, 100] = inf
    x[7, 100:300:50] = inf
    x[7, 3] = nan
    x[8, :699] = -inf
    x[9, :699] = nan
    x[10, 10:] = low
    x[11] = torch.finfo(dtype).max
    u = np.random.default_rng(1).random(12).tolist()
    for kw in ({}, dict(k=[3] * 12), dict(p=[0.9] * 12), dict(least=[0.01] * 12), dict(t=[0.0] * 12),
               dict(t=[2.0] * 12, k=[4] * 12, p=[0.7] * 12)):
        check(x, u, **kw)
    ids, probs = lora.sample(x, own(u, torch.float64))
    assert ids[1] == -1 and ids[2] == -1 and probs[1] == 0 and probs[2] == 0 and ids[6] == 100 and ids[8] == 699


def test_zeros_of_both_signs_are_equal():
    x = torch.zeros(2, 50, device="cuda")
    x[0, ::2] = -0.0
    x[1, 1::2] = -0.0
    check(x, [0.3, 0.3], k=[5, 5])
    assert lora.sample(x, own([0.5, 0.5], torch.float64), own([0.0, 0.0], torch.float32))[0].tolist() == [0, 0]


def test_random_numbers_at_their_ends():
    x = logits(6, 333, torch.float32, 5)
    u = [0.0, 5e-324, 1.0 - 2.0 ** -53, 0.5, 0.25, 0.75]
    check(x, u)
    # outside [0, 1) as the nearest in it
    ids, _ = lora.sample(x[:4], own([-1.0, float("nan"), 1.0, 7.0], torch.float64))
    want = [decode_ref.sample(x[i].cpu().numpy(), v, 1.0, 0, 1.0, 0.0)[0] for i, v in
            enumerate((0.0, 0.0, 1.0 - 2.0 ** -53, 1.0 - 2.0 ** -53))]
    assert ids.tolist() == want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 1, 3, 8])
def test_rows_of_any_stride(pad, dtype):
    """Rows that start anywhere, as slices of padded ones; the padding is not read."""
    B, V = 5, 1003
    wide = torch.full((B, V + pad), float("inf"), dtype=dtype, device="cuda")
    wide[:, :V] = logits(B, V, dtype, 6)
    u = np.random.default_rng(pad).random(B).tolist()
    check(wide[:, :V], u, k=[7] * B, p=[0.8] * B)
    check(wide[1:, :V], u[1:])
    if pad:
        wide[:, 0] = float("inf")
        check(wide[:, 1:V + 1][:, :V - 1], u, p=[0.95] * B)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_spread_out_and_peaked(dtype):
    """A flat vocabulary, where a filter keeps a large part of it, and one token far above the rest."""
    u = np.random.default_rng(7).random(4).tolist()
    flat = logits(4, 40000, dtype, 8, spread=0.05)
    check(flat, u, p=[0.1, 0.5, 0.9, 0.99])
    check(flat, u, k=[100, 5000, 20000, 39999], p=[0.9] * 4)
    peak = logits(4, 40000, dtype, 9)
    peak[:, 777] = 60.0
    check(peak, u, p=[0.1, 0.5, 0.9, 0.99999])
    check(peak, u, k=[1, 2, 300, 0], least=[0.1, 1e-20, 0.0, 1e-30])


def test_frequencies():
    """Over evenly spread random numbers the tokens come as often as their
    probabilities say, to one draw a border."""
    x = torch.tensor([[1.0, 0.0, 2.0, -1.0, 0.5]], device="cuda")
    n = 4000
    u = (torch.arange(n, dtype=torch.float64, device="cuda") + 0.5) / n
    ids, probs = lora.sample(x.expand(n, 5).contiguous(), u)
    want = torch.softmax(x[0].double(), 0)
    for i in range(5):
        assert abs(int((ids == i).sum()) - n * float(want[i])) <= 2
    np.testing.assert_allclose(probs.cpu().numpy(), want[ids.long()].cpu().numpy(), rtol=RTOL)


def test_captured_and_repeated():
    """Two captured graphs replayed in turn against eager calls; equal calls give equal bits."""
    x, u = logits(20, 30011, torch.bfloat16, 10), torch.rand(20, dtype=torch.float64, device="cuda")
    k, p = own([0, 7, 50, 1000] * 5, torch.int32), own([1.0, 0.9, 0.5, 0.99] * 5, torch.float32)
    t = own([0.0, 0.7, 1.0, 1.3, 2.0] * 4, torch.float32)
    args = [dict(), dict(temperature=t, top_k=k, top_p=p)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = [lora.sample(x, u, **a) for a in args]
    torch.cuda.synchronize()
    for a, f in zip(args, first):
        for _ in range(3):
            got = lora.sample(x, u, **a)
            assert torch.equal(got[0], f[0]) and torch.equal(got[1], f[1])
    graphs = []
    for a in args:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = lora.sample(x, u, **a)
        graphs.append((gr, out, a))
    for step in range(4):
        x.copy_(logits(20, 30011, torch.bfloat16, 20 + step))
        u.copy_(torch.rand(20, dtype=torch.float64, device="cuda"))
        for gr, _, _ in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for _, out, a in graphs:
            want = lora.sample(x, u, **a)
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_binding_refuses():
    x, u = torch.zeros(2, 9, device="cuda"), torch.zeros(2, dtype=torch.float64, device="cuda")
    with pytest.raises(ValueError):
        lora.sample(x.half(), u)
    with pytest.raises(ValueError):
        lora.sample(x, u.float())
    with pytest.raises(ValueError):
        lora.sample(x, u[:1])
    with pytest.raises(ValueError):
        lora.sample(x.t(), torch.zeros(9, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError):
        lora.sample(x, u, top_k=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        lora.sample(x, u, temperature=torch.zeros(2))
    with pytest.raises(lora.LoraError):
        lora.sample(torch.zeros(2, 0, device="cuda"), u)
    ids, probs = lora.sample(torch.zeros(0, 9, device="cuda"), u[:0])
    assert ids.shape == (0,) and probs.shape == (0,)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_few_rows_and_many(dtype):
    """Rows of a small batch, whose passes are spread over the chip, and of one that
    takes a workgroup a row give the same bits: rows of every kind, filters of
    every kind."""
    V, kinds = 40000, 8
    x = logits(kinds, V, dtype, seed=2)
    x[1] = 1.5  # all equal
    x[2] = torch.randint(0, 3, (V,), device="cuda").to(dtype)  # many of few values
    x[3, 5:] = -float("inf")
    x[4] = float("nan")
    x[5, ::7] = float("inf")
    x[6, 1::2] = float("nan")
    x[7] = torch.linspace(-300.0, 300.0, V, device="cuda").to(dtype)
    g = np.random.default_rng(11)
    for n in range(12):
        u = torch.from_numpy(g.random(kinds)).cuda()
        t = torch.from_numpy(g.choice([0.0, 0.3, 1.0, 40.0], kinds).astype(np.float32)).cuda()
        k = torch.from_numpy(g.choice([0, 1, 30, 3000, V - 1], kinds).astype(np.int32)).cuda()
        p = torch.from_numpy(g.choice([0.0, 0.1, 0.9, 0.9999, 1.0], kinds).astype(np.float32)).cuda()
        least = torch.from_numpy(g.choice([0.0, 0.01, 2.0], kinds).astype(np.float32)).cuda()
        for use in (dict(), dict(temperature=t), dict(temperature=t, top_k=k), dict(top_p=p),
                    dict(temperature=t, top_k=k, top_p=p, min_p=least)):
            ids, probs = lora.sample(x, u, **use)
            many = {name: v.repeat(4) for name, v in use.items()}
            ids4, probs4 = lora.sample(x.repeat(4, 1), u.repeat(4), **many)
            assert torch.equal(ids.repeat(4), ids4) and torch.equal(probs.repeat(4), probs4), (n, sorted(use))
    L = lora.lib()  # the two ways: with a workspace and without
    assert L.lora_sample_workspace_bytes(kinds, V) > 0 and L.lora_sample_workspace_bytes(4 * kinds, V) == 0
