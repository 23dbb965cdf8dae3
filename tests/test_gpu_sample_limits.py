"""Sampling at the limits between a workgroup a row and rows spread over the chip
(32768 logits, 40960 of 32 rows, 65536 of 192), and at the end of the weights'
whole numbers."""
import numpy as np
import pytest
import torch

from rank_gemm_amd import lora
from test_gpu_sample import check, logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("few,many,V", [(8, 32, 32769), (8, 32, 40960), (24, 192, 40961), (8, 192, 65536)])
def test_both_ways_give_the_same_bits(few, many, V, dtype):
    L = lora.lib()
    assert L.lora_sample_workspace_bytes(few, V) > 0 and L.lora_sample_workspace_bytes(many, V) == 0
    assert L.lora_sample_workspace_bytes(1, 32768) == 0 and L.lora_sample_workspace_bytes(many, 65537) > 0
    x = logits(few, V, dtype, seed=V)
    x[1] = 1.5
    x[2] = torch.randint(0, 3, (V,), device="cuda").to(dtype)
    x[3, 5:] = -float("inf")
    x[4, 1::2] = float("nan")
    g = np.random.default_rng(V)

    def own(values, kind):
        return torch.from_numpy(g.choice(values, few).astype(kind)).cuda()

    n = many // few
    for _ in range(4):
        u = torch.from_numpy(g.random(few)).cuda()
        kw = dict(temperature=own([0.0, 0.5, 1.0, 30.0], np.float32), top_k=own([0, 1, 40, 2000, V - 1], np.int32),
                  top_p=own([0.1, 0.9, 0.999, 1.0], np.float32), min_p=own([0.0, 0.01, 1.0], np.float32))
        for use in (dict(), dict(top_p=kw["top_p"]), kw):
            ids, probs = lora.sample(x, u, **use)
            ids2, probs2 = lora.sample(x.repeat(n, 1), u.repeat(n), **{k: v.repeat(n) for k, v in use.items()})
            assert torch.equal(ids.repeat(n), ids2) and torch.equal(probs.repeat(n), probs2)


@pytest.mark.parametrize("B,V", [(16, 32768), (16, 32769), (32, 40960), (40, 40961), (192, 41000), (2, 65537)])
def test_beside_the_limits(B, V):
    x = logits(B, V, torch.bfloat16, seed=B)
    g = np.random.default_rng(B + V)
    check(x, g.random(B).tolist(), t=g.choice([0.5, 1.0], B).tolist(), k=g.choice([0, 3, 300], B).tolist(),
          p=g.choice([0.6, 0.95, 1.0], B).tolist(), least=g.choice([0.0, 0.05], B).tolist())


@pytest.mark.parametrize("V", [300, 70000])
def test_weights_that_round_to_nothing(V):
    """Up to 65536 tokens a weight is a whole number of 2^-46, of 70000 one of 2^-45:
    at a quarter of that a token is not drawn, whatever u, and at three quarters it is."""
    one = 2.0 ** -46 if V <= 65536 else 2.0 ** -45
    x = torch.full((2, V), -1000.0, device="cuda")
    x[:, 100] = 0.0
    x[0, 7] = float(np.log(one / 4))
    x[1, 7] = float(np.log(one * 3 / 4))
    ids, probs = lora.sample(x, torch.zeros(2, dtype=torch.float64, device="cuda"))
    assert ids.tolist() == [100, 7]
    # of a token that weighs w the probability is w over the sum, itself not rounded to whole numbers
    np.testing.assert_allclose(probs.cpu().numpy(), [1.0, float(np.exp(np.float64(np.float32(x[1, 7].item()))))],
                               rtol=2.0 ** -24 + 2.0 ** -40)
