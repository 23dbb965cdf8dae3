"""The paged cache, decode attention, routing by scores and sampling on the
CPU: argument checks that return before anything is launched, and the 64-bit
forms the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

from rank_gemm_amd import lora
import decode_ref

P16 = 1 << 20  # a 16-byte aligned address that is never read
Q16 = P16 + 4096


def cache(**kw):
    a = dict(k=P16, v=Q16, k_scale=None, v_scale=None, page_stride=16 * 2 * 64, row_stride=2 * 64, head_stride=64,
             form=lora.LORA_BF16, n_pages=4, page_rows=16, kv_heads=2, dim=64)
    a.update(kw)
    return lora.KvCacheDesc(**a)


BAD_CACHES = [dict(k=None), dict(v=None), dict(k=P16 + 8), dict(v=P16), dict(form=0), dict(form=2), dict(n_pages=0),
              dict(page_rows=0), dict(kv_heads=0), dict(dim=0), dict(dim=60), dict(dim=264), dict(page_stride=0),
              dict(row_stride=4), dict(head_stride=68), dict(form=lora.LORA_F8),
              dict(form=lora.LORA_F8, k_scale=P16 + 64), dict(form=lora.LORA_F8, k_scale=P16 + 64, v_scale=P16 + 66),
              dict(form=lora.LORA_F8, k_scale=P16 + 64, v_scale=P16 + 64, dim=40)]


def append(c, **kw):
    a = dict(k=P16 + 8192, v=P16 + 16384, ks=128, vs=128, rows=P16 + 32768, T=3)
    a.update(kw)
    return lora.lib().lora_kv_append(ctypes.byref(c) if c else None, *(a[n] for n in ("k", "v", "ks", "vs", "rows", "T")),
                                     None)


def attend(c, **kw):
    a = dict(q=P16 + 8192, qs=4 * 64, heads=4, table=P16 + 16384, ts=8, width=8, lengths=P16 + 20480, B=2, scale=0.125,
             window=0, out=P16 + 32768, lse=None, ws=P16 + 65536, wsb=1 << 40)
    a.update(kw)
    return lora.lib().lora_attn_decode(ctypes.byref(c) if c else None, *(a[n] for n in (
        "q", "qs", "heads", "table", "ts", "width", "lengths", "B", "scale", "window", "out", "lse", "ws", "wsb")), None)


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_cache_refuses(bad):
    assert append(cache(**bad)) == lora.LORA_EINVAL
    assert attend(cache(**bad)) == lora.LORA_EINVAL


@pytest.mark.parametrize("bad", [dict(T=-1), dict(k=None), dict(v=None), dict(rows=None), dict(k=P16 + 8200),
                                 dict(v=P16 + 8), dict(rows=P16 + 4), dict(ks=120), dict(vs=132), dict(k=P16),
                                 dict(v=Q16), dict(rows=P16), dict(T=2 ** 31 - 1)])
def test_append_refuses(bad):
    assert append(cache(), **bad) == lora.LORA_EINVAL


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(B=65536), dict(heads=3), dict(heads=0), dict(heads=65536), dict(width=0), dict(width=1 << 27),
    dict(ts=7), dict(qs=200), dict(qs=260), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1),
    dict(B=40000, heads=128, qs=128 * 64), dict(scale=3e38),
    dict(q=None), dict(q=P16 + 8200), dict(table=None), dict(table=P16 + 2), dict(lengths=None), dict(out=None),
    dict(out=P16 + 8), dict(lse=P16 + 2), dict(out=P16), dict(out=Q16), dict(out=P16 + 8192), dict(lse=P16 + 16384),
    dict(lse=P16 + 20480), dict(lse=P16 + 32768)])
def test_attend_refuses(bad):
    assert attend(cache(), **bad) == lora.LORA_EINVAL


def test_empty_calls():
    assert append(cache(), T=0, k=None, v=None, rows=None) == lora.LORA_OK
    assert attend(cache(), B=0, q=None, table=None, lengths=None, out=None, ws=None) == lora.LORA_OK
    assert append(None) == lora.LORA_EINVAL and attend(None) == lora.LORA_EINVAL
    assert lora.lib().lora_sample(lora.LORA_F32, None, 8, 0, 8, None, None, None, None, None, None, None, None, 0,
                                  None) == lora.LORA_OK


def test_attend_workspace():
    L = lora.lib()
    for sizes in ((-1, 4, 2, 64, 8, 16), (2, 3, 2, 64, 8, 16), (2, 4, 2, 0, 8, 16), (2, 4, 2, 64, 0, 16)):
        assert L.lora_attn_decode_workspace_bytes(*sizes) == 0
    n = L.lora_attn_decode_workspace_bytes(2, 4, 2, 64, 1 << 16, 16)
    if n:
        assert attend(cache(), width=1 << 16, ts=1 << 16, ws=None) == lora.LORA_ESPACE
        assert attend(cache(), width=1 << 16, ts=1 << 16, wsb=n - 1) == lora.LORA_ESPACE
        assert attend(cache(), width=1 << 16, ts=1 << 16, ws=P16 + 8) == lora.LORA_ESPACE
        assert attend(cache(), width=1 << 16, ts=1 << 16, ws=P16 + 32768) == lora.LORA_EINVAL


def route(scores=None, **kw):
    a = dict(x=P16, router=Q16, T=4, H=64, E=8, k=2, ids=P16 + 8192, weights=P16 + 12288, ws=None, wsb=0)
    s = dict(bias=None, score=1, groups=2, top_groups=1, group_best=2, renorm=1, scale=1.0)
    s.update({n: v for n, v in kw.items() if n in s})
    a.update({n: v for n, v in kw.items() if n not in s})
    d = lora.RouteScoresDesc(*(s[n] for n in ("bias", "score", "groups", "top_groups", "group_best", "renorm",
                                              "scale")))
    return lora.lib().lora_moe_route_scored(*(a[n] for n in ("x", "router", "T", "H", "E", "k")), ctypes.byref(d),
                                            *(a[n] for n in ("ids", "weights", "ws", "wsb")), None)


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), -1), (dict(H=60), -1), (dict(E=513), -1), (dict(k=0), -1), (dict(T=257), -1), (dict(x=None), -1),
    (dict(router=Q16 + 2), -1), (dict(ids=None), -1), (dict(weights=None), -1), (dict(score=2), -1),
    (dict(groups=0), -1), (dict(groups=3), -1), (dict(top_groups=0), -1), (dict(top_groups=3), -1), (dict(k=5), -1),
    (dict(group_best=0), -1), (dict(group_best=3), -1), (dict(scale=float("inf")), -1), (dict(ids=P16), -1),
    (dict(ids=P16 + 12288), -1), (dict(bias=P16 + 12288), -1), (dict(bias=P16 + 2), -1),
    (dict(H=8192, E=64), -6), (dict(H=8192, E=64, ws=P16 + 8192, wsb=1 << 20), -1),
    (dict(H=8192, E=64, ws=P16, wsb=8), -6)])
def test_route_refuses(bad, want):
    assert route(**bad) == want


def test_route_empty():
    assert route(T=0, x=None, router=None, ids=None, weights=None) == lora.LORA_OK


def draw(**kw):
    a = dict(dtype=lora.LORA_BF16, logits=P16, stride=100, B=2, V=100, u=Q16, temperature=None, top_k=None, top_p=None,
             min_p=None, ids=P16 + 8192, probs=P16 + 12288, ws=P16 + 16384, wsb=1 << 40)
    a.update(kw)
    return lora.lib().lora_sample(*(a[n] for n in ("dtype", "logits", "stride", "B", "V", "u", "temperature", "top_k",
                                                   "top_p", "min_p", "ids", "probs", "ws", "wsb")), None)


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(B=-1), dict(B=65536), dict(V=0), dict(V=4194305, stride=4194305), dict(stride=99),
    dict(logits=None), dict(logits=P16 + 1), dict(u=None), dict(u=Q16 + 4), dict(ids=None), dict(ids=P16 + 8194),
    dict(probs=None), dict(probs=P16 + 8194), dict(ids=P16), dict(probs=Q16), dict(ids=P16 + 12288),
    dict(temperature=P16 + 2), dict(top_k=P16 + 1),
    dict(temperature=P16 + 8192), dict(top_k=P16 + 8192), dict(top_p=P16 + 12288), dict(min_p=P16 + 12288)])
def test_sample_refuses(bad):
    assert draw(**bad) == lora.LORA_EINVAL


def test_sample_workspace():
    L = lora.lib()
    for B, V in ((-1, 8), (65536, 8), (2, 0), (2, 4194305)):
        assert L.lora_sample_workspace_bytes(B, V) == 0
    n = L.lora_sample_workspace_bytes(2, 100)
    if n:
        assert draw(ws=None) == lora.LORA_ESPACE and draw(wsb=n - 1) == lora.LORA_ESPACE
        assert draw(ws=P16 + 16392) == lora.LORA_ESPACE and draw(ws=P16 + 8192) == lora.LORA_EINVAL
    big = dict(V=200000, stride=200000)
    n = L.lora_sample_workspace_bytes(2, 200000)
    assert n > 0 and draw(ws=None, **big) == lora.LORA_ESPACE and draw(wsb=n - 1, **big) == lora.LORA_ESPACE
    assert draw(ws=P16 + 16392, **big) == lora.LORA_ESPACE and draw(ws=P16 + 8192, **big) == lora.LORA_EINVAL


def test_binding_refuses_host_tensors():
    b, f = torch.bfloat16, torch.float32
    k = torch.zeros(4, 16, 2, 64, dtype=b)
    with pytest.raises(ValueError):
        lora.attn_decode(torch.zeros(1, 4, 64, dtype=b), k, k, torch.zeros(1, 4, dtype=torch.int32),
                         torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        lora.kv_append(torch.zeros(1, 2, 64, dtype=b), torch.zeros(1, 2, 64, dtype=b), k, k,
                       torch.zeros(1, dtype=torch.int64))
    for bad in (None, k.float()):
        with pytest.raises(ValueError):
            lora.kv_append(k[0], k[0], k, bad, torch.zeros(16, dtype=torch.int64))
        with pytest.raises(ValueError):
            lora.attn_decode(k[0], bad, k, torch.zeros(16, 4, dtype=torch.int32), torch.zeros(16, dtype=torch.int32))
    with pytest.raises(ValueError):
        lora.moe_route_scored(torch.zeros(4, 64, dtype=b), torch.zeros(8, 64, dtype=b), 2)
    with pytest.raises(ValueError):
        lora.moe_route_scored(torch.zeros(4, 64, dtype=b), torch.zeros(8, 64, dtype=b), 2, score="tanh")
    with pytest.raises(ValueError):
        lora.sample(torch.zeros(2, 9, dtype=f), torch.zeros(2, dtype=torch.float64))


def test_e4m3_rule():
    """Rounding to E4M3 against the code whose value is nearest, over both signs,
    half-way points included (to the even code)."""
    v = decode_ref.e4m3_values()[:127]
    mid = (v[1:] + v[:-1]) / 2
    for i, m in enumerate(mid):
        even = v[i] if i % 2 == 0 else v[i + 1]
        assert decode_ref.e4m3_nearest(m) == even and decode_ref.e4m3_nearest(-m) == -even
        assert decode_ref.e4m3_nearest(m * (1 + 1e-12)) == v[i + 1]
    assert decode_ref.e4m3_nearest([500.0, -1e9, np.inf]).tolist() == [448.0, -448.0, 448.0]
    x = torch.from_numpy(np.concatenate([v, mid, -mid]).astype(np.float32))
    np.testing.assert_array_equal(x.to(torch.float8_e4m3fn).double().numpy(), decode_ref.e4m3_nearest(x.numpy()))


def test_attention_form():
    """The 64-bit form against sums written out, and a request of one position."""
    g = np.random.default_rng(0)
    q, k, v = g.standard_normal((4, 8)), g.standard_normal((5, 2, 8)), g.standard_normal((5, 2, 8))
    out, lse, bound, lb = decode_ref.attention(q, k, v, 0.3)
    for h in range(4):
        e = [np.exp(0.3 * sum(q[h, d] * k[j, h // 2, d] for d in range(8))) for j in range(5)]
        np.testing.assert_allclose(lse[h], np.log(sum(e)), rtol=1e-12)
        np.testing.assert_allclose(out[h], sum(e[j] * v[j, h // 2] for j in range(5)) / sum(e), rtol=1e-12)
    np.testing.assert_allclose(decode_ref.attention(q, k[:1], v[:1], 0.3)[0], v[0].repeat(2, axis=0), rtol=1e-15)


def test_route_form():
    x, r = np.eye(1, 8), np.zeros((8, 8))
    r[:, 0] = [0, 3, 1, 1, 4, -5, 2, 2.5]  # the logits
    s = 1 / (1 + np.exp(-r[:, 0]))
    ids, w = decode_ref.route(x, r, 2, "sigmoid", None, 1, 1, 2, False, 1.0)
    assert ids.tolist() == [[4, 1]] and np.allclose(w, s[[4, 1]])
    # groups of two: sums .5 + .95, .73 + .73, .98 + .007, .88 + .92
    assert decode_ref.route(x, r, 2, "sigmoid", None, 4, 1, 2, True, 1.0)[0].tolist() == [[7, 6]]
    assert decode_ref.route(x, r, 2, "sigmoid", None, 4, 1, 1, True, 1.0)[0].tolist() == [[4, 5]]
    ids, w = decode_ref.route(x, r, 3, "sigmoid", np.array([1.0, 0, 0, 0, 0, 0, 0, 0]), 4, 2, 2, True, 2.5)
    assert ids.tolist() == [[0, 1, 7]] and np.isclose(w.sum(), 2.5)
    np.testing.assert_allclose(decode_ref.route(x, r, 8, "softmax", None, 1, 1, 2, False, 1.0)[1].sum(), 1.0)


def test_sample_form():
    x = np.log([0.1, 0.4, 0.2, 0.2, 0.1])
    assert decode_ref.sample(x, 0.05, 1.0, 0, 1.0, 0.0)[0] == 0
    assert [decode_ref.sample(x, u, 1.0, 0, 1.0, 0.0)[0] for u in (0.11, 0.49, 0.51, 0.71, 0.95)] == [1, 1, 2, 3, 4]
    assert decode_ref.sample(x, 0.99, 0.0, 0, 1.0, 0.0) == (1, 1.0)
    # the two largest; equal ones by index
    assert [decode_ref.sample(x, u, 1.0, 2, 1.0, 0.0)[0] for u in (0.0, 0.66, 0.67, 0.99)] == [1, 1, 2, 2]
    assert decode_ref.sample(x, 0.99, 1.0, 0, 0.7, 0.0)[0] == 3 and decode_ref.sample(x, 0.99, 1.0, 0, 0.55, 0.0)[0] == 2
    assert decode_ref.sample(x, 0.99, 1.0, 0, 1.0, 0.49)[0] == 3
    assert decode_ref.sample(x, 0.5, 1.0, 0, 0.0, 0.0) == (1, 1.0)
    assert decode_ref.sample([np.nan, -np.inf], 0.5, 1.0, 0, 1.0, 0.0) == (-1, 0.0)
    assert decode_ref.sample([0.0, np.inf, np.inf], 0.7, 1.0, 0, 1.0, 0.0) == (2, 0.5)
