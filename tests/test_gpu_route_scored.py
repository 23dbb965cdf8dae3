"""Routing by scores with a bias and groups against its 64-bit form
(tests/decode_ref.py): experts exactly, weights within the one rounding to fp32
(2^-24) and the last places of 64-bit sums."""
import numpy as np
import pytest
import torch

from rank_gemm_amd import lora
from rank_gemm_amd.inputs import bf16_bits, bf16_to_f32
import decode_ref

pytestmark = pytest.mark.gpu

RTOL = 2.0 ** -24 + 2.0 ** -40


def dev_bf16(v):
    bits = bf16_bits(np.asarray(v, np.float32))
    return lora.to_device(bits, "bf16"), bf16_to_f32(bits).astype(np.float64)


SIZES = [  # T, H, E, k, groups, top_groups
    (1, 8, 1, 1, 1, 1), (3, 64, 8, 2, 4, 2), (1, 256, 64, 6, 8, 3), (7, 1000, 60, 4, 1, 1), (64, 512, 256, 8, 8, 4),
    (5, 2056, 130, 16, 10, 4), (32, 264, 512, 16, 2, 1), (512, 64, 12, 1, 3, 1), (200, 128, 100, 2, 1, 1),
    (13, 4096, 96, 8, 96, 8), (64, 4096, 256, 8, 8, 4), (2, 8192, 512, 4, 512, 4), (1, 4096, 128, 8, 8, 4)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,H,E,k,groups,top", SIZES)
def test_route(T, H, E, k, groups, top, score):
    g = np.random.default_rng(T + H + E)
    x, x64 = dev_bf16(g.standard_normal((T, H)))
    r, r64 = dev_bf16(g.standard_normal((E, H)) * 2 * H ** -0.5)
    bias = (0.2 * g.standard_normal(E)).astype(np.float32)
    for b, best, renorm, scale in ((bias, 2, True, 2.5), (bias, 1, False, 1.0), (None, 2, False, 0.7), (None, 1, True, 1.0)):
        ids, w = lora.moe_route_scored(x, r, k, score=score, bias=None if b is None else torch.from_numpy(b).cuda(),
                                       groups=groups, top_groups=top, group_best=best, renorm=renorm, scale=scale)
        ref, rw = decode_ref.route(x64, r64, k, score, None if b is None else b.astype(np.float64), groups, top, best,
                                   renorm, float(np.float32(scale)))
        np.testing.assert_array_equal(ids.cpu().numpy(), ref)
        np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=RTOL, atol=0)


@pytest.mark.parametrize("T,H,E", [(4, 64, 16), (4, 8192, 64)])
def test_without_bias_and_groups_it_is_moe_route(T, H, E):
    """Both routers read the same logits: softmax scores choose the same experts
    and give its weights, to fp32's rounding."""
    g = np.random.default_rng(H)
    x, _ = dev_bf16(g.standard_normal((T, H)))
    r, _ = dev_bf16(g.standard_normal((E, H)) * H ** -0.5)
    for renorm in (True, False):
        ids, w = lora.moe_route(x, r, 4, renorm=renorm)
        ids2, w2 = lora.moe_route_scored(x, r, 4, score="softmax", renorm=renorm)
        assert torch.equal(ids, ids2)
        # moe_route's exponentials and sum are fp32 (tests of its own bound them)
        np.testing.assert_allclose(w.cpu().numpy(), w2.cpu().numpy(), rtol=(40 + E) * 2.0 ** -24)


@pytest.mark.parametrize("H", [64, 8192])
def test_ties_go_to_the_lowest_index(H):
    E, k = 64, 6
    x = torch.randn(9, H, device="cuda").to(torch.bfloat16)
    r = torch.randn(1, H, device="cuda").to(torch.bfloat16).expand(E, H).contiguous()
    for groups, top, best in ((1, 1, 1), (8, 3, 1), (8, 3, 2), (16, 2, 2)):
        ids, w = lora.moe_route_scored(x, r, k, groups=groups, top_groups=top, group_best=best)
        assert ids.tolist() == [list(range(k))] * 9
        np.testing.assert_allclose(w.cpu().numpy(), 1.0 / k, rtol=2.0 ** -23)
    # a bias moves the choice and not the weights: the last group, backwards
    bias = torch.zeros(E, device="cuda")
    bias[56:] = torch.arange(8, 16, device="cuda").float()
    ids, w = lora.moe_route_scored(x, r, k, bias=bias, groups=8, top_groups=1, renorm=True, scale=3.0)
    assert ids.tolist() == [[63, 62, 61, 60, 59, 58]] * 9
    np.testing.assert_allclose(w.cpu().numpy(), 3.0 / k, rtol=2.0 ** -23)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_masked_experts_and_nan(score):
    g = np.random.default_rng(5)
    x, x64 = dev_bf16(g.standard_normal((6, 64)))
    r, r64 = dev_bf16(g.standard_normal((32, 64)))
    bias = np.zeros(32, np.float32)
    bias[:8] = -np.inf  # a group that is switched off
    bias[9] = np.finfo(np.float32).min
    bias[30] = np.nan  # never chosen while others are left
    bias[20] = np.inf
    ids, w = lora.moe_route_scored(x, r, 5, score=score, bias=torch.from_numpy(bias).cuda(), groups=4, top_groups=2)
    ref, rw = decode_ref.route(x64, r64, 5, score, bias.astype(np.float64), 4, 2, 2, True, 1.0)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=RTOL)
    # a NaN token: valid, distinct experts, NaN weights
    x[2, 3] = float("nan")
    ids, w = lora.moe_route_scored(x, r, 5, score=score, groups=4, top_groups=2)
    assert ids[2].tolist() == [0, 1, 2, 3, 4] and bool(w[2].isnan().all())
    assert not bool(w[[0, 1, 3, 4, 5]].isnan().any())


def test_saturated_scores():
    """Logits far out: sigmoid of -1000 is 0 and does not divide by zero where another is chosen."""
    x, x64 = dev_bf16(np.ones((1, 8)))
    r = np.zeros((6, 8))
    r[:, 0] = [-1000, 1000, -1000, 30, 38, 0]
    rd, r64 = dev_bf16(r)
    ids, w = lora.moe_route_scored(x, rd, 4)
    ref, rw = decode_ref.route(x64, r64, 4, "sigmoid", None, 1, 1, 2, True, 1.0)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=RTOL)


def test_captured():
    x = torch.randn(16, 4096, device="cuda").to(torch.bfloat16)
    r = (torch.randn(128, 4096, device="cuda") / 64).to(torch.bfloat16)
    bias = torch.randn(128, device="cuda") * 0.1
    kw = dict(bias=bias, groups=8, top_groups=4, scale=2.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lora.moe_route_scored(x, r, 8, **kw)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        ids, w = lora.moe_route_scored(x, r, 8, **kw)
    for _ in range(4):
        x.copy_(torch.randn(16, 4096, device="cuda"))
        gr.replay()
        torch.cuda.synchronize()
        want = lora.moe_route_scored(x, r, 8, **kw)
        assert torch.equal(ids, want[0]) and torch.equal(w, want[1])
