"""Renormalised weights where a bias, or groups, choose experts whose scores are at
the end of 64 bits or past it: against the ratios of their logarithms. The logits
are exact (one product each), a weight is off by its rounding to fp32 (2^-24, and
half the smallest fp32 step, 2^-150) and the last places of 64-bit exponentials."""
import numpy as np
import pytest
import torch

from rank_gemm_amd import lora

pytestmark = pytest.mark.gpu

RTOL, ATOL = 2.0 ** -24 + 2.0 ** -40, 2.0 ** -150

CHOSEN = [[-800.0, -801.0, -2000.0, -799.5],  # all of them 0 in 64 bits
          [-730.0, -731.0, -732.0, -733.0],   # in its last few places
          [-665.0, -666.0, -665.5, -667.0],   # 2^-960 lies among them
          [-664.0, -680.0, -700.0, -900.0], [-1000.0, -5.0, -900.0, -3.0], [-65536.0, -65280.0, -3e5, -1e6],
          [-1e30, -1e30, -1e30, -1e38], [-746.0] * 4]


def logs(l, score, every):
    l = np.asarray(l, np.float64)
    return -np.logaddexp(0.0, -l) if score == "sigmoid" else l - (every.max() + np.log(np.exp(every - every.max()).sum()))


@pytest.mark.parametrize("H", [8, 8192])  # one launch, two
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("chosen", CHOSEN)
def test_small_scores(chosen, score, H):
    E = 16
    r = torch.zeros(E, H, dtype=torch.bfloat16)
    r[:, 3] = torch.linspace(-4.0, 2.0, E)
    at = [2, 5, 11, 14]
    r[at, 3] = torch.tensor(chosen).to(torch.bfloat16)
    x = torch.zeros(2, H, dtype=torch.bfloat16)
    x[:, 3] = 1.0
    l = r[:, 3].double().numpy()
    bias = torch.zeros(E)
    bias[at] = torch.tensor([7.0, 6.0, 5.0, 4.0])
    log = logs(l[at], score, l)
    want = 2.5 * np.exp(log - log.max()) / np.exp(log - log.max()).sum()
    call = dict(score=score, bias=bias.cuda(), scale=2.5)
    ids, w = lora.moe_route_scored(x.cuda(), r.cuda(), 4, **call)
    assert ids.tolist() == [at, at]
    for t in range(2):
        np.testing.assert_allclose(w[t].double().cpu().numpy(), want, rtol=RTOL, atol=ATOL)
    _, w = lora.moe_route_scored(x.cuda(), r.cuda(), 4, renorm=False, **call)
    with np.errstate(under="ignore"):
        np.testing.assert_allclose(w[0].double().cpu().numpy(), 2.5 * np.exp(log), rtol=RTOL, atol=ATOL)


def test_small_scores_by_groups():
    """A group that is chosen for two large experts brings two that are far down."""
    r = torch.zeros(8, 8, dtype=torch.bfloat16)
    r[:, 0] = torch.tensor([3.0, 2.0, -900.0, -1000.0, 1.0, 1.0, 1.0, 1.0])
    x = torch.zeros(1, 8, dtype=torch.bfloat16)
    x[0, 0] = 1.0
    bias = torch.tensor([-5.0, -5.0, 4.0, 3.0, 0.0, 0.0, 0.0, 0.0])
    ids, w = lora.moe_route_scored(x.cuda(), r.cuda(), 2, bias=bias.cuda(), groups=2, top_groups=1)
    assert ids.tolist() == [[2, 3]]
    e = np.exp(float(r[3, 0]) - float(r[2, 0]))
    np.testing.assert_allclose(w[0].double().cpu().numpy(), [1 / (1 + e), e / (1 + e)], rtol=RTOL, atol=ATOL)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_logits_of_minus_infinity(score):
    """A chosen logit of -infinity weighs 0 next to others; of nothing else the weights are NaN."""
    r = torch.zeros(8, 8, dtype=torch.bfloat16)
    r[:, 0] = torch.tensor([-float("inf"), -800.0, -float("inf"), -801.0, 0.0, 0.0, 0.0, 0.0])
    x = torch.zeros(1, 8, dtype=torch.bfloat16)
    x[0, 0] = 1.0
    bias = torch.tensor([9.0, 8.0, 7.0, 6.0, 0.0, 0.0, 0.0, 0.0])
    ids, w = lora.moe_route_scored(x.cuda(), r.cuda(), 4, score=score, bias=bias.cuda())
    assert ids.tolist() == [[0, 1, 2, 3]]
    e = np.exp(float(r[3, 0]) - float(r[1, 0]))  # of the values that bf16 keeps
    np.testing.assert_allclose(w[0].double().cpu().numpy(), [0.0, 1 / (1 + e), 0.0, e / (1 + e)], rtol=RTOL)
    bias = torch.tensor([9.0, 0.0, 7.0, 0.0, 0.0, 0.0, 0.0, 0.0])
    ids, w = lora.moe_route_scored(x.cuda(), r.cuda(), 2, score=score, bias=bias.cuda())
    assert ids.tolist() == [[0, 2]] and bool(w.isnan().all())
