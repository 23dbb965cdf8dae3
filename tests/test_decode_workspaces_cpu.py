"""Workspaces of attention and sampling at sizes that need one and at sizes that do
not: a size that is said to be 0 is 0 for the call too, and one above 0 is
insisted on. Nothing is launched: a call whose workspace passes is refused for an
output that is an input, which is looked at later."""
import pytest

from rank_gemm_amd import lora
from test_decode_cpu import P16, Q16, attend, cache, draw


@pytest.mark.parametrize("B,V", [(2, 100), (1, 1), (1, 32768), (600, 32768)])
def test_sampling_without_a_workspace(B, V):
    assert lora.lib().lora_sample_workspace_bytes(B, V) == 0
    bad = dict(B=B, V=V, stride=V, ids=P16)  # the logits
    assert draw(ws=None, wsb=0, **bad) == lora.LORA_EINVAL
    assert draw(ws=P16 + 16392, **bad) == lora.LORA_EINVAL
    # a workspace that is not used may be anything
    assert draw(ws=Q16, wsb=0, B=B, V=V, stride=V, probs=Q16) == lora.LORA_EINVAL


@pytest.mark.parametrize("B,V", [(1, 65537), (2, 200000), (300, 65537), (4, 4194304)])
def test_sampling_with_a_workspace(B, V):
    n = lora.lib().lora_sample_workspace_bytes(B, V)
    assert n > 0
    kw = dict(B=B, V=V, stride=V)
    assert draw(ws=None, **kw) == lora.LORA_ESPACE
    assert draw(wsb=n - 1, **kw) == lora.LORA_ESPACE
    assert draw(ws=P16 + 16392, **kw) == lora.LORA_ESPACE
    assert draw(ws=P16 + 8192, **kw) == lora.LORA_EINVAL  # ids
    assert draw(wsb=n, ids=P16, **kw) == lora.LORA_EINVAL


def test_attention_with_a_workspace():
    n = lora.lib().lora_attn_decode_workspace_bytes(2, 4, 2, 64, 1 << 16, 16)
    assert n > 0
    kw = dict(width=1 << 16, ts=1 << 16)
    assert attend(cache(), ws=None, **kw) == lora.LORA_ESPACE
    assert attend(cache(), wsb=n - 1, **kw) == lora.LORA_ESPACE
    assert attend(cache(), ws=P16 + 8, **kw) == lora.LORA_ESPACE
    assert attend(cache(), ws=P16 + 32768, **kw) == lora.LORA_EINVAL  # out
    assert attend(cache(), wsb=n, out=P16, **kw) == lora.LORA_EINVAL


def test_attention_without_a_workspace():
    assert lora.lib().lora_attn_decode_workspace_bytes(2, 4, 2, 64, 8, 16) == 0
    for window in (0, 1, 113, 120, 127, 128):
        assert attend(cache(), ws=None, wsb=0, window=window, out=P16) == lora.LORA_EINVAL
