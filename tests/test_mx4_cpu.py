"""MXFP4 and mixture-of-experts entry points on the CPU: sizes, and the
argument checks that return before anything is launched."""
import ctypes

import numpy as np
import pytest

from rank_gemm_amd import lora
import mx4_ref

P16 = 1 << 20  # a 16-byte aligned address that is never read


@pytest.mark.parametrize("K,bytes_", [(0, 0), (1, 16), (32, 16), (33, 32), (4096, 2048)])
def test_row_bytes(K, bytes_):
    assert lora.lib().lora_mx4_row_bytes(K) == bytes_


@pytest.mark.parametrize("rows,K,bytes_", [(0, 32, 0), (1, 1, 512), (64, 256, 512), (65, 256, 1024), (64, 257, 1024),
                                           (14336, 4096, 224 * 16 * 512)])
def test_scale_bytes(rows, K, bytes_):
    assert lora.lib().lora_mx4_scale_bytes(rows, K) == bytes_


def test_reference_rounding():
    # half-way points go to the even mantissa, past 6 saturates, both signs
    v = np.zeros((1, 32))
    v[0, :12] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.25, -5.0, 0.2500001, 4.0]
    codes, byte = mx4_ref.quantize(v)
    assert byte[0, 0] == 127
    assert mx4_ref.values(codes, byte, 32)[0, :12].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 0, -4, 0.5, 4]


def q_args(**kw):
    a = dict(dtype=lora.LORA_BF16, src=P16, batch=1, rows=4, K=64, codes=P16, scales=P16)
    a.update(kw)
    return [a[n] for n in ("dtype", "src", "batch", "rows", "K", "codes", "scales")] + [None]


@pytest.mark.parametrize("bad", [dict(dtype=2), dict(K=0), dict(rows=-1), dict(batch=-1), dict(batch=65536),
                                 dict(rows=4194241), dict(src=None), dict(codes=None), dict(scales=None),
                                 dict(codes=P16 + 8), dict(scales=P16 + 4), dict(src=P16 + 1)])
def test_quantize_refuses(bad):
    assert lora.lib().lora_mx4_quantize(*q_args(**bad)) == lora.LORA_EINVAL


def test_empty_quantize():
    L = lora.lib()
    assert L.lora_mx4_quantize(*q_args(rows=0, src=None, codes=None, scales=None)) == lora.LORA_OK
    assert L.lora_mx4_dequantize(None, None, 0, 4, 64, lora.LORA_F32, None, None) == lora.LORA_OK
    assert L.lora_mx4_pack_scales(None, 1, 0, 64, None, None) == lora.LORA_OK


@pytest.mark.parametrize("bad", [dict(dtype=7), dict(dst=None), dict(dst=P16 + 2), dict(codes=P16 + 1), dict(K=-1)])
def test_dequantize_refuses(bad):
    a = dict(codes=P16, scales=P16, batch=1, rows=4, K=64, dtype=lora.LORA_F32, dst=P16)
    a.update(bad)
    args = [a[n] for n in ("codes", "scales", "batch", "rows", "K", "dtype", "dst")]
    assert lora.lib().lora_mx4_dequantize(*args, None) == lora.LORA_EINVAL


def test_pack_refuses():
    L = lora.lib()
    assert L.lora_mx4_pack_scales(None, 1, 4, 64, P16, None) == lora.LORA_EINVAL
    assert L.lora_mx4_pack_scales(P16, 1, 4, 64, P16 + 4, None) == lora.LORA_EINVAL
    assert L.lora_mx4_pack_scales(P16, 1, 4, 0, P16, None) == lora.LORA_EINVAL


def test_linear_refuses_without_pool():
    info = lora.PlanInfo(T=1, S=2, chunk=16)
    L = lora.lib()
    assert L.lora_linear_mx4(None, P16, P16, P16, 1, P16, P16, None, ctypes.byref(info), P16, P16, 1 << 20,
                             None) == lora.LORA_EINVAL
    assert L.lora_linear_mx4_device_plan(None, P16, P16, P16, 1, P16, 4, P16, P16, 1 << 20, None) == lora.LORA_EINVAL
    assert L.lora_workspace_bytes_mx4(None, 4, 1) == 0


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), -1), (dict(H=60), -1), (dict(H=0), -1), (dict(E=0), -1), (dict(E=513), -1), (dict(k=0), -1),
    (dict(k=17, E=64), -1), (dict(k=9), -1), (dict(T=257), -1), (dict(x=None), -1), (dict(x=P16 + 2), -1),
    (dict(router=None), -1), (dict(ids=None), -1), (dict(weights=None), -1), (dict(H=8192, E=64, ws=None), -6),
    (dict(H=8192, E=64, wsb=10), -6)])
def test_route_refuses(bad, want):
    a = dict(x=P16, router=P16, T=4, H=64, E=8, k=2, renorm=1, ids=P16, weights=P16, ws=P16, wsb=1 << 20)
    a.update(bad)
    args = [a[n] for n in ("x", "router", "T", "H", "E", "k", "renorm", "ids", "weights", "ws", "wsb")]
    assert lora.lib().lora_moe_route(*args, None) == want


@pytest.mark.parametrize("bad,want", [
    (dict(form=0), -1), (dict(T=257), -1), (dict(H=60), -1), (dict(I=0), -1), (dict(form=1, I=60), -1),
    (dict(x=None), -1), (dict(ids=None), -1), (dict(weights=None), -1), (dict(y=None), -1), (dict(y=P16), -1),
    (dict(gate=None), -1), (dict(down=P16 + 8), -1), (dict(up_scales=None), -1), (dict(ws=None), -6),
    (dict(wsb=100), -6), (dict(ws=P16 + 8), -6)])
def test_experts_refuses(bad, want):
    a = dict(form=lora.LORA_MX4, x=P16, ids=P16, weights=P16, T=4, H=64, I=64, E=8, k=2, y=P16 + 4096, ws=P16,
             wsb=1 << 20)
    w = dict(gate=P16, up=P16, down=P16, gate_scales=P16, up_scales=P16, down_scales=P16)
    w.update({n: v for n, v in bad.items() if n in w})
    a.update({n: v for n, v in bad.items() if n not in w})
    d = lora.MoeWeightsDesc(**w)
    rc = lora.lib().lora_moe_experts(a["form"], a["x"], a["ids"], a["weights"], ctypes.byref(d), a["T"], a["H"],
                                     a["I"], a["E"], a["k"], a["y"], a["ws"], a["wsb"], None)
    assert rc == want


def test_moe_empty():
    L = lora.lib()
    assert L.lora_moe_route(None, None, 0, 64, 8, 2, 1, None, None, None, 0, None) == lora.LORA_OK
    d = lora.MoeWeightsDesc()
    assert L.lora_moe_experts(lora.LORA_MX4, None, None, None, ctypes.byref(d), 0, 64, 64, 8, 2, None, None, 0,
                              None) == lora.LORA_OK
    assert L.lora_moe_experts(lora.LORA_MX4, None, None, None, None, 0, 64, 64, 8, 2, None, None, 0,
                              None) == lora.LORA_EINVAL


def test_binding_refuses_host_tensors():
    import torch
    with pytest.raises(ValueError):
        lora.mx4_quantize(torch.zeros(4, 64))
    with pytest.raises(ValueError):
        lora.mx4_quantize(torch.zeros(4, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        lora.Mx4.empty((4,), device="cpu")
    q = lora.Mx4.empty((2, 70, 33), device="cpu")
    assert q.shape == (2, 70, 33) and q.codes.shape == (2, 70, 32) and q.scales.shape == (2, 1024)
    with pytest.raises(ValueError):
        lora.mx4_dequantize(q)
    with pytest.raises(ValueError):
        lora.moe_route(torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16), 2)


@pytest.mark.parametrize("form,H,I", [(lora.LORA_BF16, 32768, 32768), (lora.LORA_MX4, 65536, 65536),
                                      (lora.LORA_MX4, 4194248, 8), (lora.LORA_MX4, 8, 4194241)])
def test_experts_refuses_sizes(form, H, I):
    """One expert's matrix of 2 GiB, and a side past LORA_MX4_MAX_ROWS."""
    d = lora.MoeWeightsDesc(*[P16] * 6)
    assert lora.lib().lora_moe_experts(form, P16, P16, P16, ctypes.byref(d), 1, H, I, 2, 1, P16 + 4096, P16, 1 << 60,
                                       None) == lora.LORA_EINVAL


def test_outputs_alias_nothing():
    """Buffers that would be read and written, or written twice, in one call."""
    L, Q = lora.lib(), P16 + 4096
    for a, b, c in ((P16, P16, Q), (P16, Q, P16), (P16, Q, Q)):
        assert L.lora_mx4_quantize(*q_args(src=a, codes=b, scales=c)) == lora.LORA_EINVAL
    for dst in (P16, Q):
        assert L.lora_mx4_dequantize(P16, Q, 1, 4, 64, lora.LORA_F32, dst, None) == lora.LORA_EINVAL
    assert L.lora_mx4_pack_scales(P16, 1, 4, 64, P16, None) == lora.LORA_EINVAL
    for ids, weights in ((P16, Q + 512), (Q, Q + 512), (Q + 512, P16), (Q + 512, Q), (Q + 512, Q + 512)):
        assert L.lora_moe_route(P16, Q, 4, 64, 8, 2, 1, ids, weights, None, 0, None) == lora.LORA_EINVAL
    d = lora.MoeWeightsDesc(*[P16 + 8192] * 6)
    for y in (P16, Q, Q + 512, P16 + 8192):
        assert L.lora_moe_experts(lora.LORA_MX4, P16, Q, Q + 512, ctypes.byref(d), 4, 64, 64, 8, 2, y, P16 + 16384,
                                  1 << 20, None) == lora.LORA_EINVAL
