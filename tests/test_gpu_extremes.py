"""Values at the ends of the types' ranges: a scaled h that rounds past bf16's
largest value, or is infinite, on every path of the layer."""
import numpy as np
import pytest
import torch

from rank_gemm_amd import lora

pytestmark = pytest.mark.gpu

# T, d_in, d_out, S, r_max, call: what carries the expand
EXPANDS = [
    (5, 256, 200, 3, 16, "linear"),          # split K, matrix cores
    (5, 256, 200, 3, 64, "linear"),
    (70, 256, 200, 70, 16, "linear"),        # dot products per lane
    (5, 256, 200, 3, 7, "linear"),
    (2100, 256, 1300, 3, 16, "linear"),      # extra K steps; the shrink split over K
    (9000, 256, 300, 3, 16, "linear"),       # its full K range
    (2100, 256, 1300, 3, 12, "linear"),      # the tile's epilogue
    (512, 14336, 4096, 3, 16, "linear"),     # a tiled split's extra steps
    (1030, 14336, 1100, 3, 12, "linear"),    # ... and unsplit, in the epilogue
    (9000, 256, 300, 3, 16, "multi"),        # several slices, one shrink
    (5, 256, 200, 3, 16, "bf16"),            # over a 4-bit base: kernel 2 of the bf16 path
    (64, 256, 14400, 3, 16, "bf16"),         # its own
    (64, 256, 14400, 3, 12, "bf16"),
    (64, 256, 14400, 3, 64, "mx4"),
    (2100, 256, 1300, 3, 16, "bf16"),        # the shrink beside the decoding
    (2100, 256, 1300, 3, 12, "bf16"),
    (2100, 256, 1300, 3, 16, "mx4"),         # ... beside the quantisation
    (2100, 256, 1300, 3, 12, "mx4"),
    (2100, 8192, 1300, 3, 16, "mx4"),        # planes joined in a launch of their own
    (1030, 14336, 1100, 3, 12, "bf16"),
]


def run(call, x, W, pool, plan):
    if call == "linear":
        return lora.linear(x, W, pool, plan)
    if call == "multi":
        ys = lora.linear_multi(x, [W, W], [pool, pool], plan)
        assert torch.equal(ys[0].view(torch.int16), ys[1].view(torch.int16))
        return ys[0]
    return lora.linear_mx4(x, lora.mx4_quantize(W), pool, plan, act=call)


def layer(T, d_in, d_out, S, r_max, alpha):
    """Base weight 0. Row 0 of A makes h = 2^128 - 2^113 of the rows of slot 1
    (finite in fp32, over every finite bf16), rank min(r_max, 5); B is 2^-100 in
    its first rank, 0 in the others, and every fourth column of it is -2^-100."""
    x = torch.zeros(T, d_in, dtype=torch.bfloat16, device="cuda")
    x[:, :2] = 2.0 ** 63
    rank = min(r_max, 5)
    A = torch.zeros(rank, d_in, dtype=torch.bfloat16, device="cuda")
    A[0, 0], A[0, 1] = 2.0 ** 64 * (2 - 2.0 ** -7), 2.0 ** 56 * (2 - 2.0 ** -6)
    B = torch.zeros(d_out, rank, dtype=torch.bfloat16, device="cuda")
    B[:, 0] = 2.0 ** -100
    B[::4, 0] = -(2.0 ** -100)
    pool = lora.Pool(S, r_max, d_in, d_out, "bf16")
    pool.install(1, A, B, alpha * rank)
    # one row of the slot among rows of slot 0 and the empty slot 2, and a run of it
    ids = np.zeros(T, np.int32)
    ids[1] = 1
    ids[T // 2:T // 2 + T // 4] = 1
    ids[-1] = 2
    sign = torch.ones(d_out, device="cuda")
    sign[::4] = -1
    return x, torch.zeros(d_out, d_in, dtype=torch.bfloat16, device="cuda"), pool, lora.plan(ids, S), ids, sign


@pytest.mark.parametrize("T,d_in,d_out,S,r_max,call", EXPANDS)
def test_h_past_the_largest_bf16(T, d_in, d_out, S, r_max, call):
    """h B = (2^128 - 2^113) 2^-100, which rounds to 2^28."""
    x, W, pool, plan, ids, sign = layer(T, d_in, d_out, S, r_max, 1.0)
    y = run(call, x, W, pool, plan)
    on = torch.from_numpy(ids == 1).cuda()
    assert bool((y[on] == 2.0 ** 28 * sign).all())
    assert bool((y[~on] == 0).all())


@pytest.mark.parametrize("T,d_in,d_out,S,r_max,call", EXPANDS)
def test_infinite_scaled_h(T, d_in, d_out, S, r_max, call):
    """scale h is past fp32's range: an infinity of the product's sign, or the
    product itself where the scale is applied after the sum over ranks."""
    x, W, pool, plan, ids, sign = layer(T, d_in, d_out, S, r_max, 4.0)
    y = run(call, x, W, pool, plan)
    on = torch.from_numpy(ids == 1).cuda()
    got = y[on].float() * sign
    assert bool(((got == float("inf")) | (got == 2.0 ** 30)).all())
    assert bool((y[~on] == 0).all())
