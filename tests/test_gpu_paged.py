"""GPU parity of the paged cache calls against plain 64-bit references.

Cache write: the pool bytes equal the blocks that the generator's quantiser
makes of the same fp32 values.  Read-back: exact.  Head norm with rotation:
|diff| <= 2e-6 * (|w| r |x|) of the pair, from the fp32 steps: the sum of
squares is off by at most log2-depth-plus-lane-steps 2^-24 (<= 16 of them, half
of that through the root), division, root, two products, then cos and sin
rounded to fp32 and three operations, at most 20 half-steps of 2^-24 in all
(1.2e-6).  Attention: with e = 2^-23,
  |diff| <= (2 ds + (n/16 + 64) e) sum_p p_p |v_p| + (n 2^-35 + 2^-29) max|v|,
  ds = (D + 8) e max_p (scale sum_i |q_i k_i|) + 4 e max_p |s_p|
(ds: a score's error with every one of its D products and sums off by a step,
and the scaling and the exponential's argument; a probability moves by at most
2 ds relative, numerator and sum together; the weighted sums take at most one
rounding for every 16 positions and 64 for the joins).  The last term: p enters the
products 2^10 fold as a sum of two fp16 numbers (2^14 fold for F16); the second
is rounded to the nearest multiple of 2^-24 where it is subnormal, an error of
at most 2^-25 whatever p, 2^-35 of the largest weight, for each of the n
positions.  A value block's scale enters times a power of two that puts the
chunk's largest at 2^4 or more, rounded to a multiple of 2^-24 below 2^-14: at
most 2^-25 / 2^4 = 2^-29 of the largest, weighted with p, whose sum is 1.  Where
all scales are subnormal (below 2^-14) p is scaled by up to 2^14 and the largest
product is at least 2^5: 2^-25 / 2^5 = 2^-30 instead of 2^-35.
(Where one position takes all and its value is zero, that is all
there is: without the term, 4-bit values of exactly zero would demand an output
right to 2^-15 of a weight of 1e-10.)"""
import numpy as np
import pytest

import quantized_weight_gemv_dequant_b200 as ntx
import synthgen as sg
from helpers import CANARY

pytestmark = pytest.mark.gpu

F16, Q8, Q4 = ntx.NTX_F16, ntx.NTX_Q8_0, ntx.NTX_Q4_0
TYPES = [F16, Q8, Q4]
ROW = {F16: lambda d: 2 * d, Q8: lambda d: d + d // 16, Q4: lambda d: d // 2 + d // 16}
STEP = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    from quantized_weight_gemv_dequant_b200 import build
    build.build()
    torch.cuda.init()
    yield
    torch.cuda.synchronize()
    assert ntx.ntx_device_status() == 0


def _t():
    import torch
    return torch


# ------------------------------------------------------------------ reference
def blocks_of(kind, w):
    """(codes, scales) that the cache holds for rows w [..., D], by the generator's quantiser."""
    d = w.shape[-1]
    if kind == F16:
        with np.errstate(over="ignore"):
            return w.astype(np.float16).view(np.uint8), None
    raw = sg.quantize(kind, w).reshape(*w.shape[:-1], d // 32, -1)
    return np.ascontiguousarray(raw[..., 2:]).reshape(*w.shape[:-1], -1), \
        np.ascontiguousarray(raw[..., :2]).view(np.float16)[..., 0]


def values_of(kind, codes, scales):
    """What the cache's rows stand for, in 64 bits."""
    if kind == F16:
        return np.ascontiguousarray(codes).view(np.float16).astype(np.float64)
    if kind == Q8:
        q = codes.view(np.int8).astype(np.float64)
    else:
        c = codes.reshape(*scales.shape, 16)
        q = np.concatenate([c & 15, c >> 4], -1).reshape(*codes.shape[:-1], -1).astype(np.float64) - 8
    return (q.reshape(*scales.shape, 32) * scales.astype(np.float64)[..., None]).reshape(q.shape)


class Cache:
    """Pools with a canary in every byte, a shuffled table (-1 behind each sequence's pages), and host views."""

    def __init__(self, kind, hkv, d, ps, lens, seed, spare=2, max_pages=None):
        torch = _t()
        self.kind, self.hkv, self.d, self.ps = kind, hkv, d, ps
        used = [-(-n // ps) for n in lens]
        self.n_pages = sum(used) + spare
        self.max_pages = max_pages or max(1, max(used))
        order = np.random.RandomState(seed).permutation(self.n_pages)
        table = np.full((len(lens), self.max_pages), -1, np.int32)
        i = 0
        for s, u in enumerate(used):
            table[s, :u] = order[i:i + u]
            i += u
        self.table_h = table
        size = ntx.ntx_paged_kv_bytes(kind, hkv, d, ps, self.n_pages)
        assert size == self.n_pages * hkv * ps * ROW[kind](d)
        self.pools = [torch.full((size,), 0xAB, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.table = torch.from_numpy(table).cuda()
        self.kv = ntx.make_paged_kv(kind, hkv, d, ps, self.n_pages, *self.pools, self.table, len(lens), self.max_pages)

    def host(self, which):
        """(codes [pages, heads, ps, bytes], scales [pages, heads, ps, D/32] or None) of a pool."""
        raw = self.pools[which].cpu().numpy().reshape(self.n_pages, self.hkv, -1)
        cb = {F16: 2 * self.d, Q8: self.d, Q4: self.d // 2}[self.kind]
        codes = raw[:, :, :self.ps * cb].reshape(self.n_pages, self.hkv, self.ps, cb)
        if self.kind == F16:
            return codes, None
        return codes, np.ascontiguousarray(raw[:, :, self.ps * cb:]).view(np.float16).reshape(
            self.n_pages, self.hkv, self.ps, -1)

    def place(self, seq, pos):
        return self.table_h[seq, pos // self.ps], pos % self.ps

    def fill(self, seed, sigma=1.0):
        """Random valid contents everywhere; returns the [which] values [pages, heads, ps, D] in 64 bits."""
        torch = _t()
        rs = np.random.RandomState(seed)
        self.val = []
        for which in range(2):
            w = (rs.standard_normal((self.n_pages, self.hkv, self.ps, self.d)) * sigma).astype(np.float32)
            codes, scales = blocks_of(self.kind, w)
            parts = [codes.reshape(self.n_pages, self.hkv, -1)]
            if scales is not None:
                parts.append(scales.reshape(self.n_pages, self.hkv, -1).view(np.uint8))
            self.pools[which].copy_(torch.from_numpy(np.concatenate(parts, -1).ravel()))
            self.val.append(values_of(self.kind, codes, scales))
        return self

    def seq_values(self, which, s, n):
        """[heads, n, D] of a sequence."""
        p = np.arange(n)
        return self.val[which][self.table_h[s, p // self.ps], :, p % self.ps].transpose(1, 0, 2)


def attention_ref(cache, q, lens, hq, scale):
    """(out, bound) in 64 bits; q fp32 [seqs, hq, D]."""
    g = hq // cache.hkv
    out = np.zeros(q.shape)
    bound = np.zeros(q.shape)
    for s, n in enumerate(lens):
        if n == 0:
            continue
        k, v = cache.seq_values(0, s, n), cache.seq_values(1, s, n)
        top_scale = np.abs(v).max() / {F16: 1e-9, Q8: 127, Q4: 8}[cache.kind]
        tiny = 2.0 ** (-30 if top_scale < 2.0 ** -14 else -35)
        for h in range(hq):
            a = q[s, h].astype(np.float64)
            x = scale * (k[h // g] @ a)
            p = np.exp(x - x.max())
            p /= p.sum()
            out[s, h] = p @ v[h // g]
            ds = (cache.d + 8) * STEP * abs(scale) * (np.abs(k[h // g]) @ np.abs(a)).max() + 4 * STEP * np.abs(x).max()
            bound[s, h] = (2 * ds + (n / 16 + 64) * STEP) * (p @ np.abs(v[h // g])) \
                + (n * tiny + 2.0 ** -29) * np.abs(v[h // g]).max()
    return out, bound


def attend(cache, q, lens, hq, scale, ws=None, stream=None, q_stride=None, out=None):
    """q: device fp32 rows.  Returns the device output [seqs, hq, D]."""
    torch = _t()
    n = ntx.ntx_attn_paged_workspace_bytes(cache.kv, hq)
    if ws is None:
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN everywhere: scratch on entry
    if out is None:
        out = torch.full((len(lens), hq, cache.d), float("nan"), device="cuda")
    ntx.ntx_attn_decode_paged(cache.kv, q, q_stride or hq * cache.d, out, hq,
                              torch.tensor(lens, dtype=torch.int32, device="cuda"), scale, ws, n, stream)
    return out


def check_attention(kind, hq, hkv, d, ps, lens, seed, q_sigma=1.0, scale=None, max_pages=None):
    torch = _t()
    c = Cache(kind, hkv, d, ps, lens, seed, max_pages=max_pages).fill(seed + 1)
    q = (np.random.RandomState(seed + 2).standard_normal((len(lens), hq, d)) * q_sigma).astype(np.float32)
    scale = np.float32(d ** -0.5 if scale is None else scale).item()
    got = attend(c, torch.from_numpy(q).cuda(), lens, hq, scale).cpu().numpy().astype(np.float64)
    ref, bound = attention_ref(c, q, lens, hq, scale)
    assert np.all(np.isfinite(got))
    over = np.abs(got - ref) - bound
    assert np.all(over <= 0), (float(over.max()), np.unravel_index(over.argmax(), over.shape))
    for s, n in enumerate(lens):
        if n == 0:
            assert np.all(got[s] == 0)


# ------------------------------------------------------------------ write and read
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hkv,d,ps,lens", [(8, 128, 64, [1]), (1, 64, 16, [33, 1, 0, 16]), (3, 256, 48, [5, 97]),
                                           (2, 128, 16, [17, 31, 32, 64, 1]), (40, 64, 32, [40])])
def test_append_bytes_and_read_back(kind, hkv, d, ps, lens):
    """Every written block is the quantiser's, every other byte stays; the read-back is exact and leaves the
    rows of unused tokens as they were."""
    torch = _t()
    c = Cache(kind, hkv, d, ps, lens, 11)
    seq = np.array([s for s, n in enumerate(lens) for _ in range(n)] + [0, 0], np.int32)
    pos = np.array([p for n in lens for p in range(n)] + [-1, -2 ** 31], np.int32)
    mix = np.random.RandomState(12).permutation(len(seq))
    seq, pos = seq[mix], pos[mix]
    n, width = len(seq), hkv * d
    size = np.exp2(np.arange(n) % 12).astype(np.float32)[:, None, None]
    w = [sg.fill_f32(13, name, n * width).reshape(n, hkv, d) * size for name in ("pk", "pv")]
    dev = [torch.from_numpy(x).cuda() for x in w]
    sd, pd = torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda()
    ntx.ntx_kv_append(c.kv, *dev, width, width, sd, pd, n)
    want = [[np.full_like(a, 0xAB) if a.dtype == np.uint8 else np.full(a.shape, 0xABAB, np.uint16).view(np.float16)
             for a in c.host(i) if a is not None] for i in range(2)]
    back = np.zeros((2, n, hkv, d))
    for i in range(2):
        codes, scales = blocks_of(kind, w[i])
        back[i] = values_of(kind, codes, scales)
        for t in range(n):
            if pos[t] >= 0:
                page, row = c.place(seq[t], pos[t])
                want[i][0][page, :, row] = codes[t]
                if scales is not None:
                    want[i][1][page, :, row] = scales[t]
    for i in range(2):
        got = [a for a in c.host(i) if a is not None]
        assert np.array_equal(got[0], want[i][0])
        if kind != F16:
            assert np.array_equal(got[1].view(np.uint16), want[i][1].view(np.uint16))
    rows = [torch.full((n, width + 4), CANARY, dtype=torch.int32, device="cuda") for _ in range(2)]
    ntx.ntx_kv_read(c.kv, *rows, width + 4, width + 4, sd, pd, n)
    one = torch.full((n, width), CANARY, dtype=torch.int32, device="cuda")
    ntx.ntx_kv_read(c.kv, None, one, 0, width, sd, pd, n)
    for i in range(2):
        h = rows[i].cpu().numpy()
        assert np.all(h[:, width:].view(np.uint32) == CANARY)
        assert np.all(h[pos < 0].view(np.uint32) == CANARY)
        assert np.array_equal(h[pos >= 0, :width].view(np.float32), back[i].reshape(n, -1)[pos >= 0].astype(np.float32))
    assert np.array_equal(one.cpu().numpy()[pos >= 0].view(np.float32), back[1].reshape(n, -1)[pos >= 0].astype(np.float32))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shift,pad", [(1, 0), (0, 3), (2, 5)])
def test_append_and_read_rows_of_any_alignment(kind, shift, pad):
    """Rows inside wider rows, at addresses and strides that are multiples of 4 bytes only; no seq_ids."""
    torch = _t()
    hkv, d, ps, n = 2, 64, 16, 7
    c = Cache(kind, hkv, d, ps, [40] * n, 21)
    width, stride = hkv * d, hkv * d + pad
    buf = [torch.from_numpy(sg.fill_f32(22, nm, n * stride + 8)).cuda() for nm in ("a", "b")]
    view = [b[shift:] for b in buf]
    pos = torch.arange(n, dtype=torch.int32, device="cuda") * 6
    ntx.ntx_kv_append(c.kv, *view, stride, stride, None, pos, n)
    out = [torch.full((n * stride + 8,), CANARY, dtype=torch.int32, device="cuda") for _ in range(2)]
    ntx.ntx_kv_read(c.kv, out[0][shift:], out[1][shift:], stride, stride, None, pos, n)
    for i in range(2):
        src, got = buf[i].cpu().numpy(), out[i].cpu().numpy()
        mask = np.zeros(got.shape, bool)
        for t in range(n):
            lo = shift + t * stride
            codes, scales = blocks_of(kind, src[lo:lo + width].reshape(1, hkv, d).copy())
            assert np.array_equal(got[lo:lo + width].view(np.float32),
                                  values_of(kind, codes, scales).ravel().astype(np.float32))
            mask[lo:lo + width] = True
        assert np.all(got[~mask].view(np.uint32) == CANARY)


@pytest.mark.parametrize("kind", [Q8, Q4])
def test_append_odd_blocks(kind):
    """Zeros of both signs, subnormals, tiny and huge blocks, ties of sign and of rounding: the quantiser's bytes."""
    torch = _t()
    d = 128
    rs = np.random.RandomState(5)
    rows = [np.zeros(d), -np.zeros(d), np.full(d, 1e-40), np.full(d, -3e-39), np.full(d, 1e-7), np.full(d, 65504 * 3.9),
            np.where(np.arange(d) % 2, 1.0, -1.0), np.where(np.arange(d) % 2, -1.0, 1.0),
            np.arange(d) % 32 * 0.5 - 7.75, np.r_[np.full(64, 127.0), np.arange(64) + 0.5],
            np.arange(d) % 32 * 0.25 - 4, rs.standard_normal(d) * 1e-6, rs.standard_normal(d) * 1e5,
            np.r_[np.zeros(31), 5.0, np.zeros(96)], rs.standard_cauchy(d), np.exp2(rs.uniform(-30, 15, d))]
    rows += [rs.standard_normal(d) * np.exp2(e) for e in range(-30, 14)]
    w = np.array(rows, np.float32).reshape(-1, 1, d)
    n = len(w)
    c = Cache(kind, 1, d, 16, [n], 31)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    x = torch.from_numpy(w).cuda()
    ntx.ntx_kv_append(c.kv, x, -x, d, d, ids, pos, n)
    for i, src in ((0, w), (1, -w)):
        codes, scales = blocks_of(kind, src)
        hc, hs = c.host(i)
        for t in range(n):
            page, row = c.place(0, t)
            assert np.array_equal(hc[page, :, row], codes[t]), t
            assert np.array_equal(hs[page, :, row].view(np.uint16), scales[t].view(np.uint16)), t


def test_append_infinities_and_nans():
    """A block with an infinity or a NaN reads back as NaN, its neighbours are untouched; fp16 keeps the element."""
    torch = _t()
    d, n = 64, 6
    w = np.random.RandomState(6).standard_normal((n, d)).astype(np.float32)
    for t, bad in enumerate((np.inf, -np.inf, np.nan, -np.nan, np.inf, np.nan)):
        w[t, 32 + 5 * t] = bad
    w[4, 40] = np.nan
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    for kind in TYPES:
        c = Cache(kind, 1, d, 16, [n], 41)
        x = torch.from_numpy(w).cuda()
        ntx.ntx_kv_append(c.kv, x, x, d, d, ids, pos, n)
        out = torch.zeros(2, n, d, device="cuda")
        ntx.ntx_kv_read(c.kv, out[0], out[1], d, d, ids, pos, n)
        for got in out.cpu().numpy():
            if kind == F16:
                assert np.array_equal(got, w.astype(np.float16).astype(np.float32), equal_nan=True)
            else:
                codes, scales = blocks_of(kind, w[:, :32].copy())
                assert np.array_equal(got[:, :32], values_of(kind, codes, scales).astype(np.float32))
                assert np.all(np.isnan(got[:, 32:]))


@pytest.mark.parametrize("kind", TYPES)
def test_places_outside_the_cache_are_skipped_and_reported(kind):
    torch = _t()
    hkv, d, ps = 2, 64, 16
    good = [(0, 3), (1, 20)]
    for bad in ((2, 0), (-1, 0), (0, 32), (0, 2 ** 31 - 1), (1, 5), (1, 16)):
        c = Cache(kind, hkv, d, ps, [32, 32], 51)
        t = c.table_h.copy()
        t[1, 0] = c.n_pages  # the page of (1, 5): one past the pool
        if bad == (1, 16):
            t[1, 1] = -1
        c.table.copy_(torch.from_numpy(t))
        places = [p for p in good if not (bad == (1, 16) and p == (1, 20))] + [bad]
        seq = torch.tensor([p[0] for p in places], dtype=torch.int32, device="cuda")
        pos = torch.tensor([p[1] for p in places], dtype=torch.int32, device="cuda")
        x = torch.from_numpy(sg.fill_f32(52, "x", len(places) * hkv * d)).cuda()
        ntx.ntx_kv_append(c.kv, x, x, hkv * d, hkv * d, seq, pos, len(places))
        assert ntx.ntx_device_status() == 5
        touched = (c.host(0)[0] != 0xAB).any(-1).any(1)
        assert touched.sum() == len(places) - 1
        for s, p in places[:-1]:
            assert touched[t[s, p // ps], p % ps]
        out = torch.full((len(places), hkv * d), CANARY, dtype=torch.int32, device="cuda")
        ntx.ntx_kv_read(c.kv, out, None, hkv * d, 0, seq, pos, len(places))
        assert ntx.ntx_device_status() == 5
        h = out.cpu().numpy().view(np.uint32)
        assert np.all(h[-1] == CANARY) and not np.any(h[:-1] == CANARY)


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 1), (15, 3), (24, 2)])
@pytest.mark.parametrize("max_pages", [None, 40])
def test_attention_types_and_heads(kind, d, hq, hkv, max_pages):
    """In a table for 224 positions a sequence (one CTA to an item) and in one for 1280 (parts and their join)."""
    check_attention(kind, hq, hkv, d, 32, [1, 77, 200], 100 + d + hq, max_pages=max_pages)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("ps", [16, 48, 256])
def test_attention_lengths(kind, ps):
    """Empty and single-token sequences, and both sides of every tile, page and chunk border."""
    check_attention(kind, 8, 2, 128, ps, [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 127, 128, 129, 0,
                                          255, 256, 257, 1000, 3, 0], 200 + ps)


@pytest.mark.parametrize("kind,hq,hkv,d,ps,lens", [
    (F16, 32, 8, 128, 64, [5001]), (Q8, 64, 8, 128, 64, [2049]), (Q4, 32, 2, 256, 16, [4099, 17]),
    (Q8, 64, 1, 128, 32, [700, 1]), (F16, 12, 12, 64, 16, [1999, 0, 513]), (Q4, 6, 1, 64, 112, [3001]),
    (F16, 4, 2, 256, 16, [2500, 31])])
def test_attention_long_and_wide(kind, hq, hkv, d, ps, lens):
    check_attention(kind, hq, hkv, d, ps, lens, 300 + hq)


@pytest.mark.parametrize("kind", TYPES)
def test_attention_many_sequences(kind):
    rs = np.random.RandomState(9)
    lens = [int(x) for x in rs.randint(0, 90, 300)]
    check_attention(kind, 8, 2, 64, 16, lens, 400)
    check_attention(kind, 8, 2, 64, 16, lens, 403, max_pages=50)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("d,hq,hkv", [(64, 12, 2), (128, 8, 2), (128, 40, 1), (256, 24, 3)])
def test_attention_up_to_both_sides_of_one_cta(kind, d, hq, hkv):
    """Every number of chunks a CTA's warps can have, to the longest table that one CTA to an item takes; then one
    page more."""
    lens = [0, 1, 16, 17, 31, 32, 33, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300, 400, 511, 512, 767, 768]
    check_attention(kind, hq, hkv, d, 16, lens, 410 + d, max_pages=48)
    check_attention(kind, hq, hkv, d, 16, lens, 410 + d, max_pages=49)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("d,hq,hkv", [(64, 16, 1), (128, 4, 1), (256, 8, 1)])
@pytest.mark.parametrize("top", [128, 256, 272, 512, 528, 1024, 1040, 2048, 2064, 6144, 6160])
def test_attention_clusters(kind, d, hq, hkv, top):
    """Few items: one CTA to eight for each, by the positions a table can hold, and parts beyond; a full sequence, an
    empty one, and one that leaves most warps without a chunk."""
    check_attention(kind, hq, hkv, d, 16, [top, 0, 35], 430 + top, max_pages=top // 16)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hq,hkv,d", [(64, 8, 128), (18, 3, 64), (33, 3, 128), (32, 2, 256)])
@pytest.mark.parametrize("top", [300, 700, 1090, 1500, 1800, 2049])
def test_attention_clusters_of_any_size_and_tiles_of_four(kind, hq, hkv, d, top):
    """Groups of 6 to 16 query heads, cut into tiles of four or not; clusters of 2 to 8 CTAs."""
    check_attention(kind, hq, hkv, d, 16, [top], top + d)
    check_attention(kind, hq, hkv, d, 16, [5, 0, top], top + d)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("top", [8192, 8193])
def test_attention_both_sides_of_the_longest_cluster(kind, top):
    check_attention(kind, 8, 1, 128, 16, [top], top)
    check_attention(kind, 4, 1, 64, 16, [top], top)


@pytest.mark.parametrize("kind", TYPES)
def test_attention_one_cta_for_many_items(kind):
    """80 items (more than half of the SMs), tables of 1024 positions and of a page more."""
    lens = [1024, 1000, 0, 1, 33, 700, 513, 1023] + [5] * 32
    check_attention(kind, 6, 2, 64, 32, lens, 420, max_pages=32)
    check_attention(kind, 6, 2, 64, 32, lens, 420, max_pages=33)


def test_attention_most_sequences():
    lens = [0] * 1024
    for i, n in ((0, 40), (500, 3), (1023, 65)):
        lens[i] = n
    check_attention(Q8, 2, 1, 64, 16, lens, 401)
    check_attention(F16, 1, 1, 64, 16, [0] * 1024, 402)


@pytest.mark.parametrize("kind", TYPES)
def test_attention_peaked_and_flat_scores(kind):
    check_attention(kind, 8, 2, 128, 32, [300, 90], 500, q_sigma=30.0)  # scores of +-100: one position takes all
    check_attention(kind, 8, 2, 128, 32, [300, 90], 501, q_sigma=1e-6)  # uniform weights
    check_attention(kind, 8, 2, 128, 32, [300, 90], 502, q_sigma=1e5, scale=1e-6)
    check_attention(kind, 8, 2, 128, 32, [300, 90], 503, q_sigma=1e-30, scale=1e29)
    check_attention(kind, 8, 2, 128, 32, [300, 90], 504, scale=-0.1)
    check_attention(kind, 8, 2, 128, 32, [300, 90], 505, scale=0.0)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("sigma", [1e-5, 1e-3, 100.0])
def test_attention_value_magnitudes(kind, sigma):
    """Small and large values: the relative bound holds whatever the scale of the cache's numbers."""
    torch = _t()
    lens, hq, hkv, d = [333, 64], 8, 2, 128
    c = Cache(kind, hkv, d, 16, lens, 61).fill(62, sigma=sigma)
    q = (np.random.RandomState(63).standard_normal((2, hq, d)) / sigma).astype(np.float32)
    scale = np.float32(0.088).item()
    got = attend(c, torch.from_numpy(q).cuda(), lens, hq, scale).cpu().numpy().astype(np.float64)
    ref, bound = attention_ref(c, q, lens, hq, scale)
    assert np.all(np.abs(got - ref) <= bound)


@pytest.mark.parametrize("kind", TYPES)
def test_attention_uneven_values(kind):
    """Rows and blocks whose magnitudes differ by powers of two up to 2^12, in keys and values."""
    torch = _t()
    lens, hq, hkv, d, ps = [210, 95], 8, 2, 64, 16
    c = Cache(kind, hkv, d, ps, lens, 71)
    rs = np.random.RandomState(72)
    n = sum(lens)
    seq = np.repeat(np.arange(2), lens).astype(np.int32)
    pos = np.concatenate([np.arange(m) for m in lens]).astype(np.int32)
    w = [(rs.standard_normal((n, hkv, d)) * np.exp2(rs.randint(-6, 7, (n, 1, 1)))
          * np.exp2(rs.randint(-3, 4, (n, hkv, d // 32))).repeat(32, -1)).astype(np.float32) for _ in range(2)]
    w[0] /= 64
    ntx.ntx_kv_append(c.kv, *[torch.from_numpy(x).cuda() for x in w], hkv * d, hkv * d,
                      torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda(), n)
    c.val = [values_of(kind, *c.host(i)) for i in range(2)]
    q = rs.standard_normal((2, hq, d)).astype(np.float32)
    got = attend(c, torch.from_numpy(q).cuda(), lens, hq, 0.125).cpu().numpy().astype(np.float64)
    ref, bound = attention_ref(c, q, lens, hq, 0.125)
    assert np.all(np.abs(got - ref) <= bound)


@pytest.mark.parametrize("kind", TYPES)
def test_attention_ignores_what_lies_behind_a_sequence(kind):
    """NaN codes and scales in every row past a length, in spare pages and in the rest of the last page, and table
    entries of any value behind it, change no bit; the output's neighbours stay."""
    torch = _t()
    lens, hq, hkv, d, ps = [33, 1, 0, 64, 95], 4, 2, 128, 48
    c = Cache(kind, hkv, d, ps, lens, 81, max_pages=4).fill(82)
    q = torch.from_numpy(np.random.RandomState(83).standard_normal((5, hq, d)).astype(np.float32)).cuda()
    want = attend(c, q, lens, hq, 0.1)
    keep = np.zeros((c.n_pages, ps), bool)
    for s, n in enumerate(lens):
        for p in range(n):
            keep[c.place(s, p)] = True
    cb = {F16: 2 * d, Q8: d, Q4: d // 2}[kind]
    for i in range(2):
        raw = c.pools[i].cpu().numpy().reshape(c.n_pages, hkv, -1)
        codes = raw[:, :, :ps * cb].reshape(c.n_pages, hkv, ps, cb)
        codes.transpose(0, 2, 1, 3)[~keep] = 0xFF  # fp16: NaN
        if kind != F16:
            raw[:, :, ps * cb:].reshape(c.n_pages, hkv, ps, -1).transpose(0, 2, 1, 3)[~keep] = 0xFF
        c.pools[i].copy_(torch.from_numpy(raw.ravel()))
    t = c.table_h.copy()
    for s, n in enumerate(lens):
        t[s, -(-n // ps):] = [2 ** 31 - 1, -1, c.n_pages, -2 ** 31][s % 4]
    c.table.copy_(torch.from_numpy(t))
    guarded = torch.full((7, hq, d), 7.0, device="cuda")
    got = attend(c, q, lens, hq, 0.1, out=guarded[1:6])
    assert torch.equal(got, want)
    assert torch.all(guarded[0] == 7) and torch.all(guarded[6] == 7)
    assert ntx.ntx_device_status() == 0


@pytest.mark.parametrize("kind", TYPES)
def test_attention_carries_nans_and_infinities_of_its_rows_only(kind):
    """A NaN in a key or a value of a sequence makes that sequence's heads NaN and no others."""
    torch = _t()
    lens, hq, hkv, d = [70, 70, 70], 4, 2, 64
    w = sg.fill_f32(91, "w", 210 * hkv * d).reshape(210, hkv, d)
    for which in range(2):
        c = Cache(kind, hkv, d, 16, lens, 92)
        x = [w.copy(), w.copy()]
        x[which][70 + 40, 1, 3] = np.nan  # sequence 1, position 40, KV head 1
        seq = torch.arange(3, dtype=torch.int32, device="cuda").repeat_interleave(70)
        pos = torch.arange(70, dtype=torch.int32, device="cuda").repeat(3)
        ntx.ntx_kv_append(c.kv, *[torch.from_numpy(a).cuda() for a in x], hkv * d, hkv * d, seq, pos, 210)
        q = torch.from_numpy(sg.fill_f32(93, "q", 3 * hq * d)).cuda()
        bad = torch.isnan(attend(c, q, lens, hq, 0.1)).cpu().numpy()
        assert not bad[0].any() and not bad[2].any() and not bad[1, :2].any()
        assert bad[1, 2:].all() if which == 0 else bad[1, 2:, 3].all()


def test_attention_bad_pages_and_lengths():
    """A page outside the pool counts as zeros, a length outside the table is cut to it: status 5, no other effect."""
    torch = _t()
    lens, hq, hkv, d, ps = [100, 60], 4, 2, 64, 16
    for kind in TYPES:
        c = Cache(kind, hkv, d, ps, lens, 95).fill(96)
        q = np.random.RandomState(97).standard_normal((2, hq, d)).astype(np.float32)
        qd = torch.from_numpy(q).cuda()
        ref, bound = attention_ref(c, q, lens, hq, 0.1)
        for bad in (c.n_pages, -1, 2 ** 31 - 1):
            t = c.table_h.copy()
            t[0, 2] = bad
            c.table.copy_(torch.from_numpy(t))
            got = attend(c, qd, lens, hq, 0.1).cpu().numpy()
            assert ntx.ntx_device_status() == 5
            val, table = c.val, c.table_h
            c.val = [np.concatenate([v, np.zeros_like(v[:1])]) for v in val]
            c.table_h = np.where(t == bad, c.n_pages, t)
            ref0, bound0 = attention_ref(c, q, lens, hq, 0.1)
            c.val, c.table_h = val, table
            assert np.all(np.abs(got[0] - ref0[0]) <= bound0[0]) and np.all(np.abs(got[1] - ref[1]) <= bound[1])
        c.table.copy_(torch.from_numpy(c.table_h))
        full = c.max_pages * ps
        c2_lens = [full + 1, 60]
        got = attend(c, qd, c2_lens, hq, 0.1).cpu().numpy()
        assert ntx.ntx_device_status() == 5
        ref1, bound1 = attention_ref(c, q, [full, 60], hq, 0.1)
        assert np.all(np.abs(got - ref1) <= bound1)
        got = attend(c, qd, [-5, 60], hq, 0.1).cpu().numpy()
        assert ntx.ntx_device_status() == 5
        assert np.all(got[0] == 0) and np.all(np.abs(got[1] - ref[1]) <= bound[1])


def test_attention_pool_past_4_gib():
    """Pages whose byte offsets pass 32 bits, in both pools."""
    torch = _t()
    hkv, d, ps, hq = 8, 256, 1024, 16
    per = hkv * ps * 2 * d
    n_pages = (1 << 33) // per + 3
    pools = [torch.empty(n_pages * per, dtype=torch.uint8, device="cuda") for _ in range(2)]
    table = torch.tensor([[n_pages - 1], [n_pages - 2], [0]], dtype=torch.int32, device="cuda")
    kv = ntx.make_paged_kv(F16, hkv, d, ps, n_pages, *pools, table, 3, 1)
    lens, n = [200, 40, 130], 370
    w = [sg.fill_f32(98, nm, n * hkv * d).reshape(n, hkv, d) for nm in ("k", "v")]
    seq = torch.repeat_interleave(torch.arange(3, dtype=torch.int32, device="cuda"), torch.tensor(lens, device="cuda"))
    pos = torch.cat([torch.arange(m, dtype=torch.int32, device="cuda") for m in lens])
    ntx.ntx_kv_append(kv, *[torch.from_numpy(x).cuda() for x in w], hkv * d, hkv * d, seq, pos, n)
    small = Cache(F16, hkv, d, ps, lens, 99)
    ntx.ntx_kv_append(small.kv, *[torch.from_numpy(x).cuda() for x in w], hkv * d, hkv * d, seq, pos, n)
    back = torch.zeros(2, n, hkv, d, device="cuda")
    ntx.ntx_kv_read(kv, back[0], back[1], hkv * d, hkv * d, seq, pos, n)
    for i in range(2):
        assert torch.equal(back[i], torch.from_numpy(w[i]).cuda().half().float())
    q = torch.from_numpy(sg.fill_f32(98, "q", 3 * hq * d)).cuda()
    want = attend(small, q, lens, hq, 0.06)
    ws_n = ntx.ntx_attn_paged_workspace_bytes(kv, hq)
    ws, got = torch.empty(ws_n, dtype=torch.uint8, device="cuda"), torch.empty_like(want)
    ntx.ntx_attn_decode_paged(kv, q, hq * d, got, hq, torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.06, ws, ws_n)
    assert torch.equal(got, want)


def test_attention_query_rows_inside_wider_rows_and_shared_pages():
    """q as part of a fused projection row; two sequences that share a prefix page."""
    torch = _t()
    kind, hq, hkv, d, ps = Q8, 8, 2, 128, 32
    c = Cache(kind, hkv, d, ps, [64, 64], 101).fill(102)
    t = c.table_h.copy()
    t[1, 0] = t[0, 0]
    c.table_h = t
    c.table.copy_(torch.from_numpy(t))
    wide = (hq + 2 * hkv) * d
    x = np.random.RandomState(103).standard_normal((2, wide)).astype(np.float32)
    lens = [64, 50]
    got = attend(c, torch.from_numpy(x).cuda(), lens, hq, 0.09, q_stride=wide).cpu().numpy()
    ref, bound = attention_ref(c, x[:, :hq * d].reshape(2, hq, d), lens, hq, np.float32(0.09).item())
    assert np.all(np.abs(got - ref) <= bound)


def test_attention_runs_are_equal_bit_for_bit():
    torch = _t()
    lens = [700, 3, 0, 1500, 64]
    for kind in TYPES:
        c = Cache(kind, 4, 128, 16, lens, 111).fill(112)
        q = torch.from_numpy(sg.fill_f32(113, "q", 5 * 16 * 128)).cuda()
        first = attend(c, q, lens, 16, 0.09)
        for _ in range(3):
            assert torch.equal(attend(c, q, lens, 16, 0.09), first)


def test_one_page_per_sequence_is_the_contiguous_cache():
    """An F16 pool of one page of max_ctx rows is the cache of ntx_attn_decode: both calls agree."""
    torch = _t()
    hq, hkv, d, ctx, n = 32, 8, 128, 512, 401
    c = Cache(F16, hkv, d, ctx, [n], 121, spare=0).fill(122)
    q = torch.from_numpy(sg.fill_f32(123, "q", hq * d)).cuda()
    got = attend(c, q, [n], hq, d ** -0.5).view(-1)
    ws_n = ntx.ntx_attn_workspace_bytes(hq, hkv, d, ctx)
    ws, out = torch.empty(ws_n, dtype=torch.uint8, device="cuda"), torch.empty(hq * d, device="cuda")
    ntx.ntx_attn_decode(q, *c.pools, out, hq, hkv, d, n, ctx, ws, ws_n)
    _, bound = attention_ref(c, q.view(1, hq, d).cpu().numpy(), [n], hq, d ** -0.5)
    assert np.all(np.abs((got - out).cpu().numpy()) <= 2 * bound.ravel())


# ------------------------------------------------------------------ head norm + rotation
def norm_rope_ref(x, w, pos, rot, halves, theta, eps):
    """x fp32 [n, heads, D]; (out, size of each output's terms) in 64 bits."""
    x = x.astype(np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1 if w is None else w.astype(np.float64))
    i = np.arange(rot // 2)
    a = pos.astype(np.float64)[:, None] * np.power(np.float64(np.float32(theta)), -2.0 * i / max(rot, 1))
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    e0, e1 = (i, i + rot // 2) if halves else (2 * i, 2 * i + 1)
    out, size = y.copy(), np.abs(y)
    out[..., e0], out[..., e1] = y[..., e0] * c - y[..., e1] * s, y[..., e0] * s + y[..., e1] * c
    size[..., e0] = size[..., e1] = np.abs(y[..., e0]) + np.abs(y[..., e1])
    return out, size


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("n,hq,hk,d,rot", [(1, 32, 8, 128, 128), (7, 4, 2, 64, 48), (33, 5, 1, 256, 256), (3, 2, 2, 2, 2),
                                           (5, 3, 1, 80, 80), (4, 3, 3, 130, 66), (19, 1, 0, 128, 0), (6, 0, 4, 96, 2),
                                           (2, 70, 9, 254, 254), (600, 2, 1, 64, 64)])
def test_norm_rope_matches(n, hq, hk, d, rot, halves):
    torch = _t()
    rs = np.random.RandomState(n + d)
    pos = rs.randint(0, 131072, n).astype(np.int32)
    pos[0] = 0
    if n > 2:
        pos[1], pos[2] = 2 ** 31 - 1, -1
    theta, eps = 5e5, 1e-6
    x = [(rs.standard_normal((n, h, d)) * np.exp2(rs.randint(-20, 21, (n, h, 1)))).astype(np.float32) for h in (hq, hk)]
    if n > 3:
        x[0][3] = 0
    w = [(1 + 0.2 * rs.standard_normal(d)).astype(np.float32), None if d == 80 else rs.standard_normal(d).astype(np.float32)]
    dev = [torch.from_numpy(a).cuda() for a in x]
    out = [torch.full((n, h, d), CANARY, dtype=torch.int32, device="cuda") for h in (hq, hk)]
    wd = [None if a is None else torch.from_numpy(a).cuda() for a in w]
    ntx.ntx_qk_norm_rope(*[a if a.numel() else None for a in dev], *[a if a.numel() else None for a in out], hq * d, hk * d,
                         *wd, torch.from_numpy(pos).cuda(), n, hq, hk, d, rot, int(halves), theta, eps)
    for i in range(2):
        if not x[i].size:
            continue
        got = out[i].cpu().numpy()
        assert np.all(got[pos < 0].view(np.uint32) == CANARY)
        ref, size = norm_rope_ref(x[i], w[i], pos, rot, halves, theta, np.float64(np.float32(eps)))
        live = pos >= 0
        assert np.all(np.abs(got.view(np.float32) - ref)[live] <= 2e-6 * size[live])
        assert np.array_equal(dev[i].cpu().numpy(), x[i])  # the input stays


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_norm_rope_angles_past_32_bits(d, halves):
    """theta below 1: frequencies above 1, quarter turns past 2^31.  theta = 2^-8 and rot_dim 16 make the frequency of
    pair i 2^i, so that the reference's angles are exact.  The kernel's: three roundings of 2^-53 (the frequency, by
    1 / pi, by the position) and what exp2 is off by (2 at most), 2^-51 of the angle at most; at 2^38 that is 2^-13."""
    torch = _t()
    pos = np.array([2 ** 31 - 1, 2 ** 31 - 12345, 2 ** 30 + 7, 123456789, 1], np.int32)
    n, hq, hk, rot, theta = len(pos), 3, 2, 16, 2.0 ** -8
    x = np.random.RandomState(d).standard_normal((n, hq + hk, d)).astype(np.float32)
    b = torch.from_numpy(x).cuda()
    w = (hq + hk) * d
    ntx.ntx_qk_norm_rope(b, b.view(-1)[hq * d:], b, b.view(-1)[hq * d:], w, w, None, None, torch.from_numpy(pos).cuda(), n,
                         hq, hk, d, rot, int(halves), theta, 1e-6)
    ref, size = norm_rope_ref(x, None, pos, rot, halves, theta, np.float64(np.float32(1e-6)))
    i = np.arange(rot // 2)
    turn = np.zeros((n, 1, d))
    turn[:, 0, i if halves else 2 * i] = turn[:, 0, i + rot // 2 if halves else 2 * i + 1] = \
        pos.astype(np.float64)[:, None] * np.exp2(i)
    assert np.all(np.abs(b.cpu().numpy() - ref) <= (2e-6 + turn * 2.0 ** -51) * size)


def test_norm_rope_in_place_in_a_fused_row():
    """q and k inside the rows of one projection, in place, at an odd stride; v and the gaps stay."""
    torch = _t()
    n, hq, hk, d = 9, 6, 2, 64
    for wide in ((hq + 2 * hk) * d, (hq + 2 * hk) * d + 3):
        x = sg.fill_f32(131, f"x{wide}", n * wide).reshape(n, wide)
        pos = np.array([0, 5, -1, 100, 7, 1, 2, 3, 99999], np.int32)
        w = torch.ones(d, device="cuda")
        b = torch.from_numpy(x).cuda()
        ntx.ntx_qk_norm_rope(b, b.view(-1)[hq * d:], b, b.view(-1)[hq * d:], wide, wide, w, w, torch.from_numpy(pos).cuda(), n, hq, hk, d,
                             d, ntx.NTX_ROPE_HALVES, 1e4, 1e-5)
        got = b.cpu().numpy()
        ref, size = norm_rope_ref(x[:, :(hq + hk) * d].reshape(n, hq + hk, d), None, pos, d, True, 1e4, 1e-5)
        live = pos >= 0
        assert np.array_equal(got[~live], x[~live]) and np.array_equal(got[:, (hq + hk) * d:], x[:, (hq + hk) * d:])
        assert np.all(np.abs(got[:, :(hq + hk) * d].reshape(ref.shape) - ref)[live] <= 2e-6 * size[live])


def test_norm_rope_adjacent_turns_like_ntx_rope():
    torch = _t()
    hq, hk, d, pos = 4, 2, 128, 777
    x = sg.fill_f32(141, "x", (hq + hk) * d)
    y = x.reshape(-1, d) / np.sqrt((x.reshape(-1, d).astype(np.float64) ** 2).mean(-1, keepdims=True) + 1e-5)
    a = torch.from_numpy(y.astype(np.float32)).cuda().view(-1)
    ntx.ntx_rope(a, a[hq * d:], hq, hk, d, pos, 5e5)
    b = torch.from_numpy(x).cuda()
    ntx.ntx_qk_norm_rope(b, b[hq * d:], b, b[hq * d:], hq * d, hk * d, None, None,
                         torch.tensor([pos], dtype=torch.int32, device="cuda"), 1, hq, hk, d, d, ntx.NTX_ROPE_ADJACENT, 5e5,
                         1e-5)
    assert torch.all((a - b).abs() <= 4e-6 * np.abs(y).max())


def test_norm_rope_nan_stays_in_its_head():
    torch = _t()
    n, hq, hk, d = 2, 3, 1, 64
    x = sg.fill_f32(142, "x", n * (hq + hk) * d).reshape(n, hq + hk, d)
    x[1, 2, 9], x[0, 0, 1] = np.nan, np.inf
    b = torch.from_numpy(x).cuda()
    ntx.ntx_qk_norm_rope(b, b[:, hq:].contiguous(), b, torch.empty(n, hk, d, device="cuda"), (hq + hk) * d, hk * d, None, None,
                         torch.tensor([3, 4], dtype=torch.int32, device="cuda"), n, hq, hk, d, d, 0, 5e5, 1e-5)
    bad = torch.isnan(b).cpu().numpy()
    assert bad[1, 2].all() and bad[0, 0].any() and not bad[0, 1:].any() and not bad[1, :2].any()


# ------------------------------------------------------------------ together
class Decoder:
    """One attention layer of a decode step over a batch: head norm and rotation, the cache's write, attention."""

    def __init__(self, kind, n, hq, hkv, d, ps, max_ctx, seed):
        torch = _t()
        self.n, self.hq, self.hkv, self.d = n, hq, hkv, d
        self.c = Cache(kind, hkv, d, ps, [max_ctx] * n, seed)
        self.wide = (hq + 2 * hkv) * d
        self.x = torch.zeros(n, self.wide, device="cuda")
        self.w = [torch.from_numpy((1 + 0.1 * sg.fill_f32(seed, nm, d)).astype(np.float32)).cuda() for nm in ("wq", "wk")]
        self.pos = torch.full((n,), -1, dtype=torch.int32, device="cuda")
        self.len = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.out = torch.zeros(n, hq, d, device="cuda")
        self.ws_n = ntx.ntx_attn_paged_workspace_bytes(self.c.kv, hq)
        self.ws = torch.empty(self.ws_n, dtype=torch.uint8, device="cuda")

    def step(self, stream=None):
        x = self.x.view(-1)
        nq, nk = self.hq * self.d, self.hkv * self.d
        k, v = x[nq:], x[nq + nk:]
        ntx.ntx_qk_norm_rope(x, k, x, k, self.wide, self.wide, *self.w, self.pos, self.n, self.hq, self.hkv, self.d, self.d,
                             ntx.NTX_ROPE_HALVES, 5e5, 1e-6, stream)
        ntx.ntx_kv_append(self.c.kv, k, v, self.wide, self.wide, None, self.pos, self.n, stream)
        ntx.ntx_attn_decode_paged(self.c.kv, x, self.wide, self.out, self.hq, self.len, self.d ** -0.5, self.ws, self.ws_n,
                                  stream)


@pytest.mark.parametrize("kind", TYPES)
def test_decode_steps_of_a_batch_match_the_formulas(kind):
    """Sequences that start at different steps and one that never does, 70 steps through all three calls; each
    step's attention against the 64-bit formulas on what the reference's own quantiser keeps of its rotated keys.
    The keys a rotation leaves differ from the reference's by its rounding, so a code may land one step off where
    the 64-bit value is next to a border: the reference therefore takes the cache's codes, after checking that each
    is within a code step of its own value."""
    torch = _t()
    n, hq, hkv, d, ps, steps = 4, 8, 2, 64, 16, 70
    m = Decoder(kind, n, hq, hkv, d, ps, 96, 151)
    start = [0, 13, 40, 1000]
    for t in range(steps):
        x = sg.fill_f32(152, f"x{t}", n * m.wide).reshape(n, m.wide)
        pos = np.array([t - s if t >= s else -1 for s in start], np.int32)
        m.x.copy_(torch.from_numpy(x))
        m.pos.copy_(torch.from_numpy(pos))
        m.len.copy_(torch.from_numpy(pos + 1))
        m.step()
        if t % 23 and t != steps - 1:
            continue
        got = m.out.cpu().numpy()
        w = [a.cpu().numpy() for a in m.w]
        q, qsize = norm_rope_ref(x[:, :hq * d].reshape(n, hq, d), w[0], pos.clip(0), d, True, 5e5, 1e-6)
        k, _ = norm_rope_ref(x[:, hq * d:(hq + hkv) * d].reshape(n, hkv, d), w[1], pos.clip(0), d, True, 5e5, 1e-6)
        m.c.val = [values_of(kind, *m.c.host(i)) for i in range(2)]
        top = np.abs(k).reshape(n, hkv, -1, 32).max(-1).repeat(32, -1)
        unit = {F16: 2.0 ** -11 * np.abs(k) + 2.0 ** -24, Q8: top / 127 * 0.55, Q4: top / 8 * 1.01}[kind]
        for s in range(n):
            if pos[s] >= 0:
                page, row = m.c.place(s, pos[s])
                assert np.all(np.abs(m.c.val[0][page, :, row] - k[s]) <= unit[s] + 4e-6 * top[s])
        qd = m.x.cpu().numpy()[:, :hq * d].reshape(n, hq, d)
        live = pos >= 0
        assert np.all(np.abs(qd - q)[live] <= 2e-6 * qsize[live])
        ref, bound = attention_ref(m.c, qd, list(pos + 1), hq, d ** -0.5)
        assert np.all(np.abs(got - ref) <= bound), t


def test_two_captured_graphs_share_a_workspace_and_follow_the_lengths():
    """A step captured for two caches of different types on one stream, with one workspace, replayed with new
    inputs, positions and lengths: the same bits as calls made one by one."""
    torch = _t()
    a, b = Decoder(Q8, 3, 8, 2, 128, 16, 400, 161), Decoder(F16, 3, 8, 2, 64, 32, 400, 162)
    a2, b2 = Decoder(Q8, 3, 8, 2, 128, 16, 400, 161), Decoder(F16, 3, 8, 2, 64, 32, 400, 162)
    big = torch.empty(max(a.ws_n, b.ws_n), dtype=torch.uint8, device="cuda")
    a.ws = b.ws = big
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graphs = []
    for m in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            m.step(torch.cuda.current_stream())
        graphs.append(g)
    torch.cuda.synchronize()
    for t in range(0, 390, 30):
        for m, m2, g in ((a, a2, graphs[0]), (b, b2, graphs[1])):
            x = torch.from_numpy(sg.fill_f32(163, f"x{t}{m.d}", m.n * m.wide)).cuda().view(m.n, -1)
            pos = torch.tensor([t, t // 2, -1 if t < 100 else t - 100], dtype=torch.int32, device="cuda")
            for y in (m, m2):
                y.x.copy_(x)
                y.pos.copy_(pos)
                y.len.copy_(pos + 1)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            graphs[0].replay()
            graphs[1].replay()
        a2.step()
        b2.step()
        torch.cuda.synchronize()
        for m, m2 in ((a, a2), (b, b2)):
            assert torch.equal(m.out, m2.out)
            for i in range(2):
                assert torch.equal(m.c.pools[i], m2.c.pools[i])


def test_calls_on_two_streams_at_once():
    """Two decoders with workspaces of their own on two streams: neither disturbs the other."""
    torch = _t()
    pairs = []
    for seed, kind in ((171, Q4), (172, F16)):
        pairs.append([Decoder(kind, 8, 16, 4, 128, 16, 640, seed) for _ in range(2)])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for (m, m2), seed in zip(pairs, (173, 174)):
        for y in (m, m2):
            y.c.fill(seed)
            y.x.copy_(torch.from_numpy(sg.fill_f32(seed, "x", y.n * y.wide)).cuda().view(y.n, -1))
            y.pos.copy_(torch.arange(8, dtype=torch.int32) * 80 + 3)
            y.len.copy_(y.pos + 1)
    torch.cuda.synchronize()
    x0 = [m.x.clone() for m, _ in pairs]
    for _ in range(10):
        for (m, _), st, x in zip(pairs, streams, x0):
            with torch.cuda.stream(st):
                m.x.copy_(x)
            m.step(st)
    torch.cuda.synchronize()
    for _, m2 in pairs:
        m2.step()
    torch.cuda.synchronize()
    for m, m2 in pairs:
        assert torch.equal(m.out, m2.out)


# ------------------------------------------------------------------ large caches, first calls
@pytest.mark.parametrize("kind,d,ps", [(F16, 256, 2 ** 23 + 16), (Q8, 256, 2 ** 24 + 16), (Q4, 256, 2 ** 25 + 16)])
def test_one_page_longer_than_4_gib(kind, d, ps):
    """A contiguous cache whose rows and scales lie past 32-bit byte offsets.  Keys are zero, so all weights are
    1 / n; values are zero but for rows at the far end, in the middle and at the front.  The sum of n equal weights
    and of the values is exact to 1e-5 relative (every partial sum of the weights is a multiple of 2^-24 of it)."""
    torch = _t()
    size = ntx.ntx_paged_kv_bytes(kind, 1, d, ps, 1)
    assert size > 2 ** 32
    pools = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    kv = ntx.make_paged_kv(kind, 1, d, ps, 1, *pools, torch.zeros(1, dtype=torch.int32, device="cuda"), 1, 1)
    n = ps - 3
    pos = torch.tensor([n - 1, ps // 2 + 5, 0, n - 40], dtype=torch.int32, device="cuda")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    v = torch.from_numpy(sg.fill_f32(181, "v", 4 * d).reshape(4, d)).cuda()
    ntx.ntx_kv_append(kv, torch.zeros_like(v), v, d, d, ids, pos, 4)
    back = torch.zeros(2, 4, d, device="cuda")
    ntx.ntx_kv_read(kv, back[0], back[1], d, d, ids, pos, 4)
    h = v.cpu().numpy()
    codes, scales = blocks_of(kind, h)
    want = values_of(kind, codes, scales)
    assert torch.all(back[0] == 0) and np.array_equal(back[1].cpu().numpy(), want.astype(np.float32))
    # rows of a zeroed Q4_0 pool hold code 0, -8 times the scale 0
    ws_n = ntx.ntx_attn_paged_workspace_bytes(kv, 2)
    ws, out = torch.empty(ws_n, dtype=torch.uint8, device="cuda"), torch.empty(2, d, device="cuda")
    q = torch.from_numpy(sg.fill_f32(181, "q", 2 * d)).cuda()
    ntx.ntx_attn_decode_paged(kv, q, 2 * d, out, 2, torch.tensor([n], dtype=torch.int32, device="cuda"), 0.0625, ws, ws_n)
    got = out.cpu().numpy().astype(np.float64)
    mean = want.sum(0) / n
    assert np.all(np.abs(got - mean) <= 1e-5 * np.abs(want).sum(0) / n)
    del pools, kv
    torch.cuda.empty_cache()


FIRST_CALL_IN_A_CAPTURE = """
import sys
sys.path.insert(0, {root!r})
import torch
import quantized_weight_gemv_dequant_b200 as ntx
hkv, hq, d, ps = 2, 8, 128, 16
pools = [torch.zeros(ntx.ntx_paged_kv_bytes(ntx.NTX_Q8_0, hkv, d, ps, 4), dtype=torch.uint8, device="cuda") for _ in range(2)]
kv = ntx.make_paged_kv(ntx.NTX_Q8_0, hkv, d, ps, 4, *pools, torch.arange(4, dtype=torch.int32, device="cuda"), 1, 4)
x = torch.randn((hq + 2 * hkv) * d, device="cuda")
pos = torch.zeros(1, dtype=torch.int32, device="cuda")
n = torch.ones(1, dtype=torch.int32, device="cuda")
ws_n = ntx.ntx_attn_paged_workspace_bytes(kv, hq)
ws, out = torch.zeros(ws_n, dtype=torch.uint8, device="cuda"), torch.zeros(hq, d, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    s = torch.cuda.current_stream()
    k, v = x[hq * d:], x[(hq + hkv) * d:]
    ntx.ntx_qk_norm_rope(x, k, x, k, hq * d, hkv * d, None, None, pos, 1, hq, hkv, d, d, 1, 1e4, 1e-6, s)
    ntx.ntx_kv_append(kv, k, v, hkv * d, hkv * d, None, pos, 1, s)
    ntx.ntx_attn_decode_paged(kv, x, hq * d, out, hq, n, 0.1, ws, ws_n, s)
g.replay()
torch.cuda.synchronize()
want = torch.zeros(hkv, d, device="cuda")
ntx.ntx_kv_read(kv, None, want, 0, hkv * d, None, pos, 1)
assert torch.allclose(out, want.repeat_interleave(hq // hkv, 0), rtol=1e-6, atol=0)
assert ntx.ntx_device_status() == 0
print("same")
"""


def test_first_calls_of_a_process_inside_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_A_CAPTURE.format(root=root)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]


def test_attention_workspace_is_enough_and_no_more_is_touched():
    """Guard bytes behind the workspace of every kernel variant stay, at lengths that split every item."""
    torch = _t()
    for kind in TYPES:
        for d in (64, 128, 256):
            for hq, hkv in ((2, 2), (12, 2), (16, 1), (40, 1)):
                c = Cache(kind, hkv, d, 16, [3000, 700], 191)
                for p in c.pools:
                    p.zero_()
                n = ntx.ntx_attn_paged_workspace_bytes(c.kv, hq)
                ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
                q = torch.ones(2, hq, d, device="cuda")
                out = attend(c, q, [3000, 700], hq, 0.1, ws=ws[:n])
                assert torch.all(ws[n:] == 0x5A) and torch.all(out == 0)
