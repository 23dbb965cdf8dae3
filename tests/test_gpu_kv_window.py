"""Windows near the size of the page table, beside the limits at which attention
goes from a workgroup a row to work that is split and joined (512, 1536 and 2048
positions): parity, and nothing written outside the workspace that was asked for."""
import pytest
import torch

from rank_gemm_amd import lora
from test_gpu_kv import Cache, check

pytestmark = pytest.mark.gpu

# requests, heads, kv heads, dim, page, positions of the table, form
LIMITS = [(16, 32, 8, 128, 16, 2048, "bf16"), (16, 32, 8, 128, 16, 2064, "bf16"), (1, 32, 8, 128, 16, 1536, "f8"),
          (1, 32, 8, 128, 24, 1536, "bf16"), (1, 16, 4, 256, 16, 512, "bf16"), (1, 64, 2, 128, 32, 512, "f8"),
          (2, 6, 2, 80, 10, 1530, "bf16"), (40, 8, 8, 64, 16, 2048, "f8"), (3, 8, 4, 32, 8, 1536, "bf16"),
          (70, 4, 4, 32, 1, 2040, "bf16"), (1, 130, 2, 128, 1, 505, "bf16")]


@pytest.mark.parametrize("B,heads,kv,dim,page,most,form", LIMITS)
def test_window_near_the_table(B, heads, kv, dim, page, most, form):
    lengths = [most, most - 1, 0, most - 17, 3][:B] + [5] * max(0, B - 5)
    c = Cache(lengths, kv, dim, page, form, width=most // page, seed=most)
    for window in (most - 16, most - 15, most - 14, most - 1, most, most + 1):
        check(c, heads, window=window)


@pytest.mark.parametrize("B,heads,kv,dim,page,most,form", LIMITS)
def test_workspace_ends_where_it_was_asked_to(B, heads, kv, dim, page, most, form):
    lengths = [most] + [most // 2] * (B - 1)
    c = Cache(lengths, kv, dim, page, form, width=most // page, seed=most)
    table, n = c.tensors()
    q = torch.randn(B, heads, dim, device="cuda").to(torch.bfloat16)
    asked = lora.lib().lora_attn_decode_workspace_bytes(B, heads, kv, dim, c.width, page)
    room = torch.full((asked + (64 << 20),), 171, dtype=torch.uint8, device="cuda")
    for window in (0, 7, most - 15, most - 8, most - 1):
        lora.attn_decode(q, c.k, c.v, table, n, window=window, k_scale=c.ks, v_scale=c.vs,
                         workspace=room[:asked] if asked else None)
        assert bool((room[asked:] == 171).all())
