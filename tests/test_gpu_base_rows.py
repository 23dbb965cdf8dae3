"""Rows on slot 0, or on a slot of rank 0, keep the bits of a base-only call,
also where the tiled GEMM's plan splits K: whether it runs split goes by the
sizes and the pool (its ranks, its slots), not by the adapters of the batch."""
import numpy as np
import pytest
import torch

from rank_gemm_amd import lora

pytestmark = pytest.mark.gpu

# T, d_in, d_out, S, r_max, rank: sizes whose plan splits K
CASES = [
    (1030, 14336, 1100, 4, 12, 12),     # ranks that are no multiple of 8: unsplit
    (769, 8200, 1500, 4, 12, 9),
    (1024, 14336, 4096, 3, 12, 12),
    (1030, 14336, 1100, 1100, 8, 8),    # more slots than the slot metadata holds: unsplit
    (769, 8200, 1500, 400, 64, 64),     # more extra steps than a split takes: unsplit
    (769, 8200, 1500, 4, 1023, 1023),
    (769, 8200, 1500, 4, 1024, 1000),
    (512, 14336, 4096, 17, 16, 16),     # split
    (769, 8200, 1500, 128, 16, 16),
    (512, 14336, 4096, 64, 32, 32),
]
# of the slots, how many a batch uses
USED = [2, 6, None]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(g, lo, hi, *shape):
    """Whole numbers lo .. hi in bf16."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(torch.bfloat16)


def slot_ids(T, S, seed, used=None):
    """Mixed slots, a fifth of the rows on slot 0; slot 1 stays empty."""
    r = np.random.default_rng(seed)
    ids = r.integers(0, min(S, used or S), T).astype(np.int32)
    ids[r.random(T) < 0.2] = 0
    ids[T // 2] = 2
    return ids


def install(pool, A, B, rank):
    """Slots 2 .. of the pool; the scale alpha / rank is a quarter."""
    for s in range(2, pool.S):
        pool.install(s, A[s], B[s], rank / 4)


def call(op, x, W, pool, plan):
    if op == "linear":
        return lora.linear(x, W, pool, plan)
    return lora.linear_mx4(x, W, pool, plan, act="bf16")


@pytest.mark.parametrize("op", ["linear", "linear_mx4"])
@pytest.mark.parametrize("T,d_in,d_out,S,r_max,rank", CASES)
def test_base_rows_keep_their_bits(T, d_in, d_out, S, r_max, rank, op):
    g = gen(T + S)
    x = torch.randn(T, d_in, generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randn(d_out, d_in, generator=g, device="cuda").to(torch.bfloat16)
    if op == "linear_mx4":
        W = lora.mx4_quantize(W)
    pool = lora.Pool(S, r_max, d_in, d_out, "bf16")
    A = (torch.randn(S, rank, d_in, generator=g, device="cuda") * d_in ** -0.5).to(torch.bfloat16)
    B = torch.randn(S, d_out, rank, generator=g, device="cuda").to(torch.bfloat16)
    install(pool, A, B, rank)
    base = call(op, x, W, pool, lora.plan(np.zeros(T, np.int32), S))
    for used in USED:
        ids = slot_ids(T, S, T, used)
        rows = torch.from_numpy(np.flatnonzero(ids < 2)).cuda()
        for plan in (lora.plan(ids, S), lora.plan_device(torch.from_numpy(ids).cuda(), S)):
            y = call(op, x, W, pool, plan)
            assert torch.equal(y[rows], base[rows])
            assert not torch.equal(y, base)


@pytest.mark.parametrize("op", ["linear", "linear_mx4"])
@pytest.mark.parametrize("T,d_in,d_out,S,r_max,rank", CASES)
def test_whole_numbers_are_exact(T, d_in, d_out, S, r_max, rank, op):
    """Whole numbers whose products and sums stay under 2^24 (scaled ones are
    multiples of a quarter under 2^22): fp32 sums are exact in any order, h
    keeps its 16 bits, and y is the exact value rounded once."""
    g = gen(T + rank)
    x, W = ints(g, -3, 3, T, d_in), ints(g, -1, 1, d_out, d_in)
    pool = lora.Pool(S, r_max, d_in, d_out, "bf16")
    A, B = ints(g, -1, 1, S, rank, d_in), ints(g, -1, 1, S, d_out, rank)
    install(pool, A, B, rank)
    ids = slot_ids(T, S, T)
    want = x.double() @ W.double().t()
    for s in range(2, S):
        rows = torch.from_numpy(np.flatnonzero(ids == s)).cuda()
        if rows.numel():
            h = x[rows].double() @ A[s].double().t()
            assert float(h.abs().max()) < 2 ** 16
            want[rows] += 0.25 * (h @ B[s].double().t())
    assert float(want.abs().max()) < 2 ** 22
    want = want.float().to(torch.bfloat16)
    Wq = lora.mx4_quantize(W) if op == "linear_mx4" else W
    for plan in (lora.plan(ids, S), lora.plan_device(torch.from_numpy(ids).cuda(), S)):
        assert torch.equal(call(op, x, Wq, pool, plan), want)
