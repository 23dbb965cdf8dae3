"""The paged cache and decode attention against their 64-bit forms
(tests/decode_ref.py). Stored rows are compared exactly; an output of attention
is one rounding to bf16 (2^-8 of the value) from fp32 sums whose loss the form
bounds."""
import numpy as np
import pytest
import torch

from rank_gemm_amd import lora
import decode_ref

pytestmark = pytest.mark.gpu


def as64(t):
    return t.detach().cpu().double().numpy()


class Cache:
    """A cache whose pages lie in no order, with requests of given lengths.
    `order`: "rows" [page][row][head], "heads" [page][head][row], or "both" (k
    and v of a page side by side)."""

    def __init__(self, lengths, kv, dim, page, form="bf16", order="rows", spare=2, seed=0, width=None):
        g = np.random.default_rng(seed)
        self.lengths, self.kv, self.dim, self.page, self.form = list(lengths), kv, dim, page, form
        need = [-(-n // page) for n in self.lengths]
        self.pages = sum(need) + spare
        self.width = max([1, *need]) if width is None else width
        names = g.permutation(self.pages)
        self.table = np.full((len(need), self.width), -7, np.int32)  # past a request's pages nothing is read
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = names[at:at + n]
            at += n
        gen = torch.Generator(device="cuda").manual_seed(seed)
        dt = torch.bfloat16 if form == "bf16" else torch.float8_e4m3fn
        shape = {"rows": (2, self.pages, page, kv, dim), "heads": (2, self.pages, kv, page, dim),
                 "both": (self.pages, 2, page, kv, dim)}[order]
        x = torch.randn(shape, generator=gen, device="cuda")
        x = (x if form == "bf16" else x * 40).to(dt)
        self.store = x
        two = x if order != "both" else x.transpose(0, 1)
        self.k, self.v = (two[0], two[1]) if order != "heads" else (two[0].transpose(1, 2), two[1].transpose(1, 2))
        self.ks = self.vs = None
        if form == "f8":
            self.ks = (0.01 + 0.02 * torch.rand(kv, generator=gen, device="cuda"))
            self.vs = (0.01 + 0.02 * torch.rand(kv, generator=gen, device="cuda"))

    def tensors(self):
        return (torch.from_numpy(self.table).cuda(), torch.tensor(self.lengths, dtype=torch.int32, device="cuda"))

    def rows(self, b, lo, hi):
        """k and v [hi - lo, kv, dim] of a request's positions, in 64 bits."""
        at = np.arange(lo, hi)
        page = torch.from_numpy(self.table[b, at // self.page].astype(np.int64)).cuda()
        where = page, torch.from_numpy(at % self.page).cuda()
        found = []
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            y = x[where] if s is None else x.view(torch.uint8)[where].view(torch.float8_e4m3fn).float() * 1.0
            y = as64(y)
            found.append(y if s is None else y * as64(s)[None, :, None])
        return found


def check(c, heads, window=0, scale=None, q=None, seed=1, skip=(), **kw):
    """One call against the form; skip: {(b, position)} that the table leaves out."""
    B = len(c.lengths)
    g = torch.Generator(device="cuda").manual_seed(seed)
    if q is None:
        q = torch.randn(B, heads, c.dim, generator=g, device="cuda").to(torch.bfloat16)
    table, lengths = c.tensors()
    out = torch.full((B, heads, c.dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    n = lora.lib().lora_attn_decode_workspace_bytes(B, heads, c.kv, c.dim, c.width, c.page)
    ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")
    got, lse = lora.attn_decode(q, c.k, c.v, table, lengths, scale=scale, window=window, k_scale=c.ks, v_scale=c.vs,
                                out=out, lse=True, workspace=ws, **kw)
    assert got is out
    sc = c.dim ** -0.5 if scale is None else scale
    worst = worst_lse = 0.0
    for b, n in enumerate(c.lengths):
        n = min(max(n, 0), c.width * c.page)
        lo = max(0, n - window) if window else 0
        k, v = c.rows(b, lo, n)
        keep = [j - lo for j in range(lo, n) if (b, j) not in skip]
        ref, rl, bound, lb = decode_ref.attention(as64(q[b]), k[keep], v[keep], sc)
        o, s = as64(out[b]), as64(lse[b])
        if not keep:
            assert not o.any() and np.isneginf(s).all()
            continue
        worst = max(worst, float((np.abs(o - ref) / (2.0 ** -8 * np.abs(ref) + bound + 1e-30)).max()))
        worst_lse = max(worst_lse, float((np.abs(s - rl) / (lb + 2.0 ** -24 * np.abs(rl))).max()))
    print(f"B={B} heads={heads}/{c.kv} dim={c.dim} page={c.page} {c.form} longest={max(c.lengths)}: worst {worst:.3f}, "
          f"lse {worst_lse:.3f} of the bounds", flush=True)
    assert worst <= 1.0 and worst_lse <= 1.0
    return out, lse


# ------------------------------------------------------------------ append --


@pytest.mark.parametrize("order", ["rows", "heads", "both"])
@pytest.mark.parametrize("form", ["bf16", "f8"])
@pytest.mark.parametrize("T,kv,dim,page", [(1, 1, 16, 1), (7, 2, 80, 24), (64, 8, 128, 16), (300, 3, 256, 5),
                                           (1000, 4, 64, 128)])
def test_append(T, kv, dim, page, form, order):
    c = Cache([T], kv, dim, page, form, order, spare=3)
    before = c.store.clone()
    g = np.random.default_rng(T)
    rows = g.permutation(c.pages * page)[:T]
    rows[T // 2:T // 2 + 1] = -1
    rows[T // 3:T // 3 + 1] = c.pages * page  # just outside
    qkv = torch.randn(T, (1 + 2 * kv) * dim, device="cuda").to(torch.bfloat16) * 4
    k, v = qkv[:, dim:(1 + kv) * dim].view(T, kv, dim), qkv[:, (1 + kv) * dim:].view(T, kv, dim)
    k[0, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38], dtype=torch.bfloat16)
    lora.kv_append(k, v, c.k, c.v, torch.from_numpy(rows).cuda(), k_scale=c.ks, v_scale=c.vs)
    for x, cache, s in ((k, c.k, c.ks), (v, c.v, c.vs)):
        old = before if order != "both" else before.transpose(0, 1)
        old = old[0 if cache is c.k else 1]
        want = as64(old.transpose(1, 2) if order == "heads" else old).copy()
        y = x.float().cpu().numpy() if s is None else x.float().cpu().numpy() / s.cpu().numpy()[None, :, None]
        y = y.astype(np.float64) if s is None else decode_ref.e4m3_nearest(y)
        for t, r in enumerate(rows):
            if 0 <= r < c.pages * page:
                want[r // page, r % page] = y[t]
        np.testing.assert_array_equal(as64(cache), want)


def test_append_every_e4m3_border():
    """Every value between two codes, the half-way points and both sides of them."""
    v = decode_ref.e4m3_values()[:127]
    pts = np.concatenate([v, (v[1:] + v[:-1]) / 2, [464.0, 500.0]])
    x = torch.from_numpy(pts.astype(np.float32)).to(torch.bfloat16)  # exact: 5 bits of mantissa
    x = torch.cat([x, -x, torch.nextafter(x, torch.full_like(x, 1e4)), torch.nextafter(x, torch.full_like(x, -1.0))])
    x = torch.nn.functional.pad(x, (0, -len(x) % 128)).view(-1, 1, 128).cuda()
    T = x.shape[0]
    k, v8 = (torch.zeros(1, T, 1, 128, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    one = torch.ones(1, device="cuda")
    lora.kv_append(x, x, k, v8, torch.arange(T, device="cuda"), k_scale=one, v_scale=one)
    want = decode_ref.e4m3_nearest(as64(x).reshape(T, 128))
    np.testing.assert_array_equal(as64(k).reshape(T, 128), want)
    np.testing.assert_array_equal(as64(v8).reshape(T, 128), want)


def test_append_nothing():
    c = Cache([3], 2, 64, 4)
    before = c.store.clone()
    k = torch.randn(0, 2, 64, device="cuda").to(torch.bfloat16)
    lora.kv_append(k, k, c.k, c.v, torch.zeros(0, dtype=torch.int64, device="cuda"))
    k = torch.randn(5, 2, 64, device="cuda").to(torch.bfloat16)
    lora.kv_append(k, k, c.k, c.v, torch.tensor([-1, -2 ** 62, 2 ** 62, c.pages * 4, 2 ** 33], device="cuda"))
    assert torch.equal(before, c.store)


# --------------------------------------------------------------- attention --

SHAPES = [  # lengths, heads, kv heads, dim, page
    ([1], 1, 1, 64, 16), ([0, 5, 0], 4, 2, 64, 8), ([137], 32, 8, 128, 16), ([1, 2, 31, 32, 33, 63, 64, 65], 8, 2, 128, 16),
    ([127, 128, 129, 255, 256, 257, 0, 1], 6, 3, 64, 32), ([700, 1, 1500], 12, 2, 80, 24), ([300, 4097], 5, 1, 96, 1),
    ([1000, 513], 16, 1, 128, 7), ([40, 2000], 64, 2, 64, 64), ([900], 3, 3, 256, 48), ([777, 10], 40, 1, 112, 16),
    ([257, 64], 130, 2, 128, 16), ([600, 50], 70, 1, 256, 32), ([90] * 33, 4, 4, 16, 16), ([33, 1025], 28, 4, 176, 128),
    ([2049], 17, 17, 128, 3), ([300, 70], 100, 2, 64, 16), ([900, 5, 1600], 96, 2, 48, 16), ([1300] + [9] * 63, 40, 2, 128, 16),
    ([700] + [20] * 63, 4, 2, 256, 16), ([2000, 0] + [30] * 150, 2, 2, 64, 16), ([1536, 1000], 8, 2, 128, 16),
    ([1537, 600], 8, 2, 128, 16), ([512], 32, 2, 256, 32), ([513, 100], 24, 1, 128, 16), ([3000, 77, 1], 8, 4, 64, 16),
    ([2500, 2501], 16, 2, 64, 24), ([2100, 0, 5], 6, 6, 32, 16), ([1999], 4, 2, 48, 5), ([2222, 1700], 12, 2, 16, 64),
    ([300, 0, 1] + [7] * 150, 8, 4, 64, 16), ([1900] + [20] * 255, 4, 2, 32, 10)]


@pytest.mark.parametrize("form", ["bf16", "f8"])
@pytest.mark.parametrize("lengths,heads,kv,dim,page", SHAPES)
def test_attention(lengths, heads, kv, dim, page, form):
    check(Cache(lengths, kv, dim, page, form, seed=heads), heads)


@pytest.mark.parametrize("form", ["bf16", "f8"])
@pytest.mark.parametrize("order", ["heads", "both"])
@pytest.mark.parametrize("dim,page", [(128, 16), (64, 6), (48, 32)])
def test_layouts(dim, page, order, form):
    check(Cache([300, 17, 0, 1], 2, dim, page, form, order), 8)


@pytest.mark.parametrize("window", [1, 2, 31, 100, 128, 129, 1000, 5000])
def test_window(window):
    check(Cache([1, 99, 100, 101, 128, 1000, 3333, 0], 2, 128, 16), 8, window=window)
    check(Cache([40, 257, 1999], 2, 80, 24, "f8"), 6, window=window)


@pytest.mark.parametrize("window", [17, 1700, 2300])
@pytest.mark.parametrize("dim,form,page", [(64, "f8", 16), (64, "f8", 24), (32, "bf16", 16)])
def test_window_over_pairs(dim, form, page, window):
    """Kv heads that share a line of memory, in long rows and in many."""
    check(Cache([40, 2600, 0, 1999], 4, dim, page, form), 12, window=window)
    check(Cache([2100] + [30] * 64, 4, dim, page, form), 8, window=window)


@pytest.mark.parametrize("n,heads,kv,dim,page,form", [(40000, 8, 2, 128, 64, "bf16"), (70001, 4, 1, 64, 16, "f8"),
                                                      (33333, 32, 8, 128, 16, "f8"), (20011, 2, 1, 256, 11, "bf16")])
def test_long(n, heads, kv, dim, page, form):
    check(Cache([n, 7, n // 3], kv, dim, page, form), heads)


def test_many_requests():
    g = np.random.default_rng(3)
    check(Cache(g.integers(0, 300, 700).tolist(), 2, 64, 16), 8)


def test_scale_and_large_scores():
    """Scores far apart: the softmax is nearly one position; a negative scale."""
    c = Cache([500, 90], 2, 128, 16)
    q = (torch.randn(2, 8, 128, device="cuda") * 30).to(torch.bfloat16)
    check(c, 8, q=q, scale=1.0)
    check(c, 8, q=q, scale=-0.3)
    check(c, 8, q=q, scale=0.0)


def test_wide_table_and_strided_rows():
    """A table much wider than the requests, as a slice of a wider one, q as a
    slice of merged rows: the same bits as from tensors of their own."""
    c = Cache([100, 333, 0], 2, 128, 16, width=21)
    table, lengths = c.tensors()
    wide = torch.full((3, 70), 10 ** 9, dtype=torch.int32, device="cuda")
    wide[:, :21] = table
    qkv = torch.randn(3, 12 * 128, device="cuda").to(torch.bfloat16)
    q = qkv[:, :1024].view(3, 8, 128)
    a = lora.attn_decode(q, c.k, c.v, wide[:, :21], lengths)
    assert torch.equal(a, lora.attn_decode(q.contiguous(), c.k, c.v, table, lengths))
    full = lora.attn_decode(q, c.k, c.v, wide, lengths)  # its sums may be made in another order
    assert float((full.float() - a.float()).abs().max()) <= 2.0 ** -7 * float(a.float().abs().max())


def test_lengths_past_the_table():
    """Lengths below 0 and past the table's positions."""
    c = Cache([48, 48, 48], 2, 64, 16)
    c.lengths = [-5, 49, 2 ** 31 - 1]
    check(c, 4)


def test_pages_outside_the_cache():
    """Positions of pages that are not there are left out; a request of nothing
    else gets zeros."""
    c = Cache([100, 64, 40, 1], 2, 64, 16)
    good = c.table.copy()
    skip = set()
    for b, p, bad in ((0, 2, -1), (0, 6, c.pages), (1, 0, 2 ** 31 - 1), (2, 0, -2 ** 31), (2, 1, c.pages), (2, 2, -9),
                      (3, 0, -1)):
        c.table[b, p] = bad
        skip |= {(b, j) for j in range(16 * p, min(16 * p + 16, c.lengths[b]))}
    table, lengths = c.tensors()
    q = torch.randn(4, 4, 64, device="cuda").to(torch.bfloat16)
    out, lse = lora.attn_decode(q, c.k, c.v, table, lengths, lse=True)
    c.table = good
    for b, n in enumerate(c.lengths):
        k, v = c.rows(b, 0, n)
        keep = [j for j in range(n) if (b, j) not in skip]
        ref, rl, bound, lb = decode_ref.attention(as64(q[b]), k[keep], v[keep], 0.125)
        if not keep:
            assert not as64(out[b]).any() and np.isneginf(as64(lse[b])).all()
        else:
            assert (np.abs(as64(out[b]) - ref) <= 2.0 ** -8 * np.abs(ref) + bound).all()
            assert (np.abs(as64(lse[b]) - rl) <= lb + 2.0 ** -24 * np.abs(rl)).all()


def test_rows_past_the_length_are_not_read():
    """NaN and infinity in the rest of a request's last page, in other pages and
    before the window change nothing; at an attended position they show."""
    c = Cache([70, 9, 200], 2, 128, 16, spare=4)
    table, lengths = c.tensors()
    q = torch.randn(3, 8, 128, device="cuda").to(torch.bfloat16)
    want = lora.attn_decode(q, c.k, c.v, table, lengths, window=60)
    keep = torch.zeros(c.pages, 16, dtype=torch.bool)
    for b, n in enumerate(c.lengths):
        for j in range(max(0, n - 60), n):
            keep[c.table[b, j // 16], j % 16] = True
    for bad in (float("nan"), float("inf"), -float("inf")):
        c.k[~keep.cuda()] = bad
        c.v[~keep.cuda()] = bad
        assert torch.equal(want, lora.attn_decode(q, c.k, c.v, table, lengths, window=60))
    c.v[c.table[0, 69 // 16], 69 % 16, 1, 5] = float("nan")
    got = lora.attn_decode(q, c.k, c.v, table, lengths, window=60)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[0, 4:, 5] = True
    assert bool(got[hit].isnan().all()) and torch.equal(got[~hit], want[~hit])


def test_infinite_keys():
    """A score of -infinity weighs nothing (all of them: as a request without a
    position), one of +infinity gives NaN, to the heads that meet it."""
    c = Cache([300, 40], 2, 128, 16)
    table, lengths = c.tensors()
    q = torch.randn(2, 8, 128, device="cuda").to(torch.bfloat16)
    q[..., 7] = 1.5
    c.k[c.table[0, 100 // 16], 100 % 16, :, 7] = -float("inf")
    for j in range(40):
        c.k[c.table[1, j // 16], j % 16, 1, 7] = -float("inf")
    out, lse = lora.attn_decode(q, c.k, c.v, table, lengths, lse=True)
    k, v = c.rows(0, 0, 300)
    keep = [j for j in range(300) if j != 100]
    ref, rl, bound, lb = decode_ref.attention(as64(q[0]), k[keep], v[keep], 128 ** -0.5)
    assert (np.abs(as64(out[0]) - ref) <= 2.0 ** -8 * np.abs(ref) + bound).all()
    assert (np.abs(as64(lse[0]) - rl) <= lb + 2.0 ** -24 * np.abs(rl)).all()
    assert not as64(out[1, 4:]).any() and np.isneginf(as64(lse[1, 4:])).all()
    assert bool(out[1, :4].isfinite().all())
    c.k[c.table[0, 17], 3, 0, 7] = float("inf")
    got = lora.attn_decode(q, c.k, c.v, table, lengths)
    assert bool(got[0, :4].isnan().all()) and torch.equal(got[0, 4:], out[0, 4:]) and torch.equal(got[1], out[1])


@pytest.mark.parametrize("lengths", [[2500], [300] * 130])
@pytest.mark.parametrize("dim,form", [(64, "f8"), (32, "bf16")])
def test_neighbouring_kv_heads_are_apart(dim, form, lengths):
    """A NaN (and an infinity) in the rows of one kv head reaches its heads alone,
    also where two kv heads share a line of memory."""
    c = Cache(lengths, 4, dim, 16, form)
    table, n = c.tensors()
    B = len(lengths)
    q = torch.randn(B, 8, dim, device="cuda").to(torch.bfloat16)
    call = lambda: lora.attn_decode(q, c.k, c.v, table, n, k_scale=c.ks, v_scale=c.vs)
    want = call()
    for bad in (float("nan"),) if form == "f8" else (float("nan"), float("inf")):
        for head in range(4):
            for x in (c.k, c.v):
                at = (int(c.table[0, 7]), 5, head)
                raw = x[at].clone()
                x[at] = torch.full((dim,), bad, device="cuda").to(x.dtype)
                got = call()
                hit = torch.zeros_like(got, dtype=torch.bool)
                hit[0, 2 * head:2 * head + 2] = True
                assert not bool(got[hit].isfinite().any()) and torch.equal(got[~hit], want[~hit])
                x[at] = raw
    assert torch.equal(want, call())


def test_shared_pages():
    """A page that several requests read, or one request several times."""
    c = Cache([100, 200, 64], 2, 128, 16)
    c.table[1, :3] = c.table[0, 2:5]
    c.table[2, :4] = c.table[1, 5]
    check(c, 8)


def test_rows_far_apart():
    """Rows 2^24 elements apart, heads and pages between them."""
    x = torch.randn(2, 16, 1 << 24, device="cuda", dtype=torch.bfloat16)
    c = Cache([40], 2, 128, 16, spare=0)
    c.k, c.v = (y.as_strided((3, 16, 2, 128), (1024, 1 << 24, 256, 1), y.storage_offset()) for y in (x[0], x[1]))
    check(c, 8)
    new = torch.randn(2, 2, 128, device="cuda").to(torch.bfloat16)
    lora.kv_append(new, -new, c.k, c.v, torch.tensor([47, 0], device="cuda"))
    assert torch.equal(c.k[2, 15], new[0]) and torch.equal(c.v[0, 0], -new[1])
    check(c, 8)


def test_offsets_past_4_gib():
    """The first and the last page of a cache of over 4 GiB, and of its rows."""
    page, kv, dim = 16, 8, 128
    pages = (5 << 30) // (page * kv * dim * 2)
    k, v = (torch.empty(pages, page, kv, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c = Cache([40], kv, dim, page)
    c.table = np.array([[pages - 1, 0, pages // 2 + 3]], np.int32)
    for x in (k, v):
        x[torch.from_numpy(c.table[0].astype(np.int64)).cuda()] = 0
    c.k, c.v, c.pages = k, v, pages
    rows = np.array([(pages - 1) * page + j for j in range(16)] + list(range(16)) +
                    [(pages // 2 + 3) * page + j for j in range(8)])
    new = torch.randn(40, kv, dim, device="cuda").to(torch.bfloat16)
    lora.kv_append(new, -new, k, v, torch.from_numpy(rows).cuda())
    assert torch.equal(k[pages - 1], new[:16]) and torch.equal(v[0], -new[16:32])
    check(c, 32)


def test_streams_and_repeats():
    """Equal calls give equal bits, on a stream of their own too, and calls of
    two streams do not disturb one another."""
    c, d = Cache([5000, 3, 900], 2, 128, 16), Cache([4000, 4001], 2, 64, 16, seed=5)
    qc = torch.randn(3, 8, 128, device="cuda").to(torch.bfloat16)
    qd = torch.randn(2, 8, 64, device="cuda").to(torch.bfloat16)
    tc, td = c.tensors(), d.tensors()
    a, b = lora.attn_decode(qc, c.k, c.v, *tc), lora.attn_decode(qd, d.k, d.v, *td)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        with torch.cuda.stream(s1):
            x = lora.attn_decode(qc, c.k, c.v, *tc)
        with torch.cuda.stream(s2):
            y = lora.attn_decode(qd, d.k, d.v, *td)
        got.append((x, y))
    torch.cuda.synchronize()
    assert all(torch.equal(a, x) and torch.equal(b, y) for x, y in got)


def test_captured():
    """Two captured graphs, replayed in turn over growing lengths, with eager
    calls between the replays."""
    c = Cache([3000, 40, 700], 2, 128, 16)
    table, full = c.tensors()
    lengths = full.clone()
    q = torch.randn(3, 8, 128, device="cuda").to(torch.bfloat16)
    graphs = []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        lora.attn_decode(q, c.k, c.v, table, lengths)
    torch.cuda.synchronize()
    for window in (0, 500):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = lora.attn_decode(q, c.k, c.v, table, lengths, window=window)
        graphs.append((gr, out, window))
    for step in range(4):
        lengths.copy_(torch.clamp(full - 3 * step * step, min=0))
        q.copy_(torch.randn(3, 8, 128, device="cuda"))
        for gr, out, window in graphs:
            gr.replay()
        for gr, out, window in graphs:
            torch.cuda.synchronize()
            assert torch.equal(out, lora.attn_decode(q, c.k, c.v, table, lengths, window=window))


def test_binding_refuses():
    c = Cache([20], 2, 64, 16)
    t, n = c.tensors()
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        lora.attn_decode(q.float(), c.k, c.v, t, n)
    with pytest.raises(ValueError):
        lora.attn_decode(q, c.k, c.v.float(), t, n)
    with pytest.raises(ValueError):
        lora.attn_decode(q, c.k, c.v, t.long(), n)
    with pytest.raises(ValueError):
        lora.attn_decode(q, c.k, c.v, t, n.long())
    with pytest.raises(ValueError):
        lora.attn_decode(q, c.k, c.v, t.cpu(), n)
    with pytest.raises(ValueError):
        lora.attn_decode(q, c.k, c.v, t, n, k_scale=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError):
        lora.attn_decode(q, c.k.transpose(1, 3), c.v.transpose(1, 3), t, n)
    with pytest.raises(ValueError):
        lora.attn_decode(q, c.k[:1].expand(9, -1, -1, -1), c.v[:1].expand(9, -1, -1, -1), t, n)
    with pytest.raises(ValueError):
        lora.attn_decode(q[:, :, :32], c.k, c.v, t, n)
    with pytest.raises(lora.LoraError):
        lora.attn_decode(q[:, :3].contiguous(), c.k, c.v, t, n)
    with pytest.raises(lora.LoraError):
        lora.attn_decode(q, c.k, c.v, t, n, out=q)
    f = Cache([20], 2, 64, 16, "f8")
    with pytest.raises(ValueError):
        lora.attn_decode(q, f.k, f.v, t, n)
    kv = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        lora.kv_append(kv, kv, c.k, c.v, torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        lora.kv_append(kv, kv[:2], c.k, c.v, torch.zeros(3, dtype=torch.int64, device="cuda"))
