"""The paged attention's two-kernel path: parts of all items' chunks and their join.

A table of more than 8192 positions takes it whatever the lengths, so every cache
here has one of 16384 (the tables in test_gpu_paged.py are narrower: nearly all of
its attention cases run in one launch of clusters).  Every call gets a workspace
full of NaN bytes with guard bytes behind it, and must have written to the one and
not to the other: a call that did not use its workspace was not on this path.

Bounds are those of test_gpu_paged.py, the reference the formula in fp64 on what the
cache holds."""
import os
import subprocess
import sys

import numpy as np
import pytest

import quantized_weight_gemv_dequant_b200 as ntx
import synthgen as sg
from test_gpu_paged import F16, Q4, Q8, STEP, TYPES, Cache, Decoder, _gpu, _t  # noqa: F401

pytestmark = pytest.mark.gpu

WIDE = 1 << 14
GUARD = 4096


class WideCache(Cache):
    """Valid random contents in every row, and in 64 bits what they stand for."""

    def __init__(self, kind, hkv, d, ps, lens, seed, spare=2):
        super().__init__(kind, hkv, d, ps, lens, seed, spare=spare, max_pages=WIDE // ps)
        torch = _t()
        gen = torch.Generator(device="cuda").manual_seed(seed)
        shape = (self.n_pages, hkv, ps, d)
        for p in self.pools:
            if kind == F16:
                p.copy_(torch.randn(shape, generator=gen, device="cuda").half().view(torch.uint8).ravel())
                continue
            raw = p.view(self.n_pages, hkv, -1)
            cb = ps * d // (1 if kind == Q8 else 2)
            raw[..., :cb] = torch.randint(0, 256, raw[..., :cb].shape, generator=gen, device="cuda", dtype=torch.uint8)
            scale = (0.5 + torch.rand((*shape[:-1], d // 32), generator=gen, device="cuda")) / (75 if kind == Q8 else 5)
            raw[..., cb:] = scale.half().view(torch.uint8).view(self.n_pages, hkv, -1)

    def values(self, which):
        """fp64 [pages, heads, ps, D] on the device."""
        torch = _t()
        raw = self.pools[which].view(self.n_pages, self.hkv, -1)
        shape = (self.n_pages, self.hkv, self.ps, self.d)
        if self.kind == F16:
            return raw.contiguous().view(torch.float16).view(shape).double()
        cb = self.ps * self.d // (1 if self.kind == Q8 else 2)
        scale = raw[..., cb:].contiguous().view(torch.float16).view(*shape[:-1], -1, 1).double()
        codes = raw[..., :cb].contiguous()
        if self.kind == Q8:
            q = codes.view(torch.int8).view(*shape[:-1], -1, 32).double()
        else:
            c = codes.view(*shape[:-1], -1, 16)
            q = torch.cat([c & 15, c >> 4], -1).double() - 8
        return (q * scale).view(shape)


def reference(c, q, lens, hq, scale):
    """(out, bound) in fp64 on the device; q fp32 [seqs, hq, D]."""
    torch = _t()
    g, vals = hq // c.hkv, [c.values(i) for i in range(2)]
    out, bound = (torch.zeros(len(lens), hq, c.d, dtype=torch.float64, device="cuda") for _ in range(2))
    for s, n in enumerate(lens):
        if n == 0:
            continue
        pages = torch.from_numpy(c.table_h[s, :-(-n // c.ps)]).cuda().long()
        k, v = (x[pages].permute(1, 0, 2, 3).reshape(c.hkv, -1, c.d)[:, :n] for x in vals)
        a = q[s].double().view(c.hkv, g, c.d)
        x = scale * (a @ k.transpose(1, 2))
        p = torch.softmax(x, -1)
        out[s] = (p @ v).view(hq, c.d)
        ds = (c.d + 8) * STEP * abs(scale) * (a.abs() @ k.abs().transpose(1, 2)).amax(-1) + 4 * STEP * x.abs().amax(-1)
        bound[s] = ((2 * ds + (n / 16 + 64) * STEP)[..., None] * (p @ v.abs())
                    + (n * 2.0 ** -35 + 2.0 ** -29) * v.abs().amax()).view(hq, c.d)
    return out, bound


class Workspace:
    def __init__(self, *needs):
        torch = _t()
        self.n = max(ntx.ntx_attn_paged_workspace_bytes(c.kv, hq) for c, hq in needs)
        self.all = torch.full((self.n + GUARD,), 0xFF, dtype=torch.uint8, device="cuda")

    def check(self):
        torch = _t()
        assert torch.any(self.all[:self.n] != 0xFF), "the workspace was not used: not the path that these tests are for"
        assert torch.all(self.all[self.n:] == 0xFF)


def attend(c, q, lens, hq, scale, ws=None, out=None, q_stride=None):
    torch = _t()
    ws = ws or Workspace((c, hq))
    if out is None:
        out = torch.full((len(lens), hq, c.d), float("nan"), device="cuda")
    ntx.ntx_attn_decode_paged(c.kv, q, q_stride or hq * c.d, out, hq, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                              scale, ws.all, ws.n)
    ws.check()
    return out


def queries(n, hq, d, seed, sigma=1.0):
    torch = _t()
    return torch.randn((n, hq, d), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * sigma


def check(kind, hq, hkv, d, ps, lens, seed, sigma=1.0, scale=None):
    torch = _t()
    c = WideCache(kind, hkv, d, ps, lens, seed)
    q = queries(len(lens), hq, d, seed + 1, sigma)
    scale = np.float32(d ** -0.5 if scale is None else scale).item()
    got = attend(c, q, lens, hq, scale).double()
    ref, bound = reference(c, q, lens, hq, scale)
    assert torch.all(torch.isfinite(got))
    over = (got - ref).abs() - bound
    assert torch.all(over <= 0), (float(over.max()), np.unravel_index(int(over.argmax()), over.shape))
    return c


# Query heads per KV head: alone, full and partial tiles of four, eight and sixteen, and several tiles to a group.
GROUPS = [(4, 4), (8, 2), (15, 3), (12, 1), (40, 1), (64, 1)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", GROUPS)
def test_types_and_heads(kind, d, hq, hkv):
    """Empty sequences, one position, and items of up to 25 parts; units fewer than the warps, so a chunk to a part."""
    check(kind, hq, hkv, d, 32, [1, 77, 0, 200, 33, 400, 0], 100 + d + hq)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 128), (6, 1, 64), (16, 1, 128), (12, 2, 256)])
@pytest.mark.parametrize("n", [16, 33, 256, 290, 511, 2048, 2100, 4100, 16383, 16384])
def test_parts_of_an_item(kind, hq, hkv, d, n):
    """One sequence in 1 part, up to 8, up to 64, and more (each has a join of its own), and a full table."""
    check(kind, hq, hkv, d, 16, [n], n + d)
    if n < 4100:
        check(kind, hq, hkv, d, 48, [n, 1, 700], n + d + 1)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (4, 4, 64), (30, 5, 64), (24, 2, 64), (12, 2, 128), (48, 3, 128),
                                      (40, 1, 128), (4, 2, 256), (24, 2, 256)])
def test_shares_cut_across_items(kind, hq, hkv, d):
    """More units than warps, lengths from 0 to thousands: a part ends one item, holds others whole and begins one."""
    torch = _t()
    rs = np.random.RandomState(d + hq)
    n = 4 + 320 // hkv  # units for every warp of the largest grid: 4 CTAs of 4 warps to an SM, chunks of 64 positions
    lens = [0, 1] + [int(2.0 ** x) for x in rs.uniform(0, 12.5, n - 4)] + [3000, 5]
    rs.shuffle(lens)
    c = WideCache(kind, hkv, d, 16, lens, d + hq)
    q, scale = queries(n, hq, d, 3), d ** -0.5
    ws = Workspace((c, hq))
    got = attend(c, q, lens, hq, scale, ws=ws).double()
    assert torch.any(ws.all[ws.n * 9 // 10:ws.n] != 0xFF)  # the last warps too
    ref, bound = reference(c, q, lens, hq, scale)
    over = (got - ref).abs() - bound
    assert torch.all(over <= 0), (float(over.max()), np.unravel_index(int(over.argmax()), over.shape))


@pytest.mark.parametrize("kind", TYPES)
def test_most_sequences(kind):
    """32 sequences to a lane of the search for a part's first item."""
    rs = np.random.RandomState(7)
    check(kind, 8, 2, 128, 16, [int(x) for x in rs.randint(0, 70, 1024)], 8)
    lens = [0] * 1024
    lens[0], lens[511], lens[1023] = 40, 3, 65
    check(kind, 4, 1, 128, 16, lens, 9)
    check(kind, 9, 1, 64, 16, [0] * 33 + [17], 10)


def test_all_empty():
    torch = _t()
    c = WideCache(Q8, 2, 128, 16, [0] * 5, 11)
    assert torch.all(attend(c, queries(5, 8, 128, 12), [0] * 5, 8, 0.1) == 0)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("sigma,scale", [(30.0, None), (1e-6, None), (1e5, 1e-6), (1e-30, 1e29), (1.0, -0.1), (1.0, 0.0)])
def test_peaked_and_flat_scores(kind, sigma, scale):
    check(kind, 8, 2, 128, 32, [300, 90, 2500], 21, sigma=sigma, scale=scale)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (64, 12, 1), (256, 16, 1)])
def test_what_lies_behind_a_sequence_is_ignored(kind, d, hq, hkv):
    """NaN codes and scales in every row past a length and in spare pages, any table entry behind it: not a bit changes."""
    torch = _t()
    lens, ps = [33, 1, 0, 1000, 95], 48
    c = WideCache(kind, hkv, d, ps, lens, 31)
    q = queries(len(lens), hq, d, 32)
    want = attend(c, q, lens, hq, 0.1)
    keep = torch.zeros(c.n_pages, ps, dtype=torch.bool)
    for s, n in enumerate(lens):
        for p in range(n):
            keep[c.place(s, p)] = True
    keep = keep.cuda()
    cb = {F16: 2 * d, Q8: d, Q4: d // 2}[kind]
    for p in c.pools:
        raw = p.view(c.n_pages, hkv, -1)
        raw[..., :ps * cb].view(c.n_pages, hkv, ps, cb).permute(0, 2, 1, 3)[~keep] = 0xFF
        if kind != F16:
            rest = raw[..., ps * cb:].reshape(c.n_pages, hkv, ps, -1)
            rest.permute(0, 2, 1, 3)[~keep] = 0xFF
            raw[..., ps * cb:] = rest.view(c.n_pages, hkv, -1)
    t = c.table_h.copy()
    for s, n in enumerate(lens):
        t[s, -(-n // ps):] = [2 ** 31 - 1, -1, c.n_pages, -2 ** 31][s % 4]
    c.table.copy_(torch.from_numpy(t))
    guarded = torch.full((len(lens) + 2, hq, d), 7.0, device="cuda")
    got = attend(c, q, lens, hq, 0.1, out=guarded[1:-1])
    assert torch.equal(got, want) and torch.all(guarded[0] == 7) and torch.all(guarded[-1] == 7)
    assert ntx.ntx_device_status() == 0


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("which", [0, 1])
def test_nans_stay_with_their_sequence_and_head(kind, which):
    torch = _t()
    lens, hq, hkv, d, ps = [70, 900, 70], 8, 2, 128, 16
    c = WideCache(kind, hkv, d, ps, lens, 41)
    page, row = c.place(1, 840)
    raw = c.pools[which].view(c.n_pages, hkv, -1)[page, 1]
    at = row * 2 * d + 6 if kind == F16 else (ps * d // (1 if kind == Q8 else 2)) + row * d // 16  # element 3, block 0's scale
    raw[at:at + 2] = torch.tensor([0x00, 0x7E], dtype=torch.uint8, device="cuda")
    bad = torch.isnan(attend(c, queries(3, hq, d, 42), lens, hq, 0.1))
    assert not bad[0].any() and not bad[2].any() and not bad[1, :4].any()
    if which == 0:
        assert bad[1, 4:].all()
    else:
        hit = slice(3, 4) if kind == F16 else slice(0, 32)
        assert bad[1, 4:, hit].all() and int(bad.sum()) == 4 * (1 if kind == F16 else 32)


@pytest.mark.parametrize("kind", TYPES)
def test_bad_pages_and_lengths(kind):
    """A page outside the pool counts as zeros, a length outside the table is cut to it: status 5, no other effect."""
    torch = _t()
    lens, hq, hkv, d, ps = [1000, 60], 8, 2, 128, 16
    c = WideCache(kind, hkv, d, ps, lens, 51)
    q = queries(2, hq, d, 52)
    for bad in (c.n_pages, -1, 2 ** 31 - 1, -2 ** 31):
        t = c.table_h.copy()
        t[0, 20], t[0, 21] = bad, bad
        c.table.copy_(torch.from_numpy(t))
        got = attend(c, q, lens, hq, 0.1).double()
        assert ntx.ntx_device_status() == 5
        zero = WideCache(kind, hkv, d, ps, [16 * c.n_pages], 53, spare=1)  # the pool with a page of zeros behind it
        for a, b in zip(zero.pools, c.pools):
            a.zero_()
            a[:b.numel()] = b
        zero.table_h = np.where(t == bad, c.n_pages, t)
        ref, bound = reference(zero, q, lens, hq, 0.1)
        assert torch.all((got - ref).abs() <= bound)
    c.table.copy_(torch.from_numpy(c.table_h))
    ref, bound = reference(c, q, lens, hq, 0.1)
    got = attend(c, q, [-5, 60], hq, 0.1).double()
    assert ntx.ntx_device_status() == 5
    assert torch.all(got[0] == 0) and torch.all((got[1] - ref[1]).abs() <= bound[1])
    full = WideCache(kind, hkv, d, ps, [WIDE, 60], 54)
    ref, bound = reference(full, q, [WIDE, 60], hq, 0.1)
    got = attend(full, q, [2 ** 31 - 1, 60], hq, 0.1).double()
    assert ntx.ntx_device_status() == 5
    assert torch.all((got - ref).abs() <= bound)


def test_query_rows_inside_wider_rows_and_shared_pages():
    torch = _t()
    for kind, (hq, hkv, d, ps) in zip(TYPES, ((8, 2, 128, 32), (12, 1, 64, 32), (16, 1, 256, 32))):
        c = WideCache(kind, hkv, d, ps, [640, 640], 61)
        c.table_h[1, :10] = c.table_h[0, :10]
        c.table.copy_(torch.from_numpy(c.table_h))
        wide = (hq + 2 * hkv) * d
        x = queries(2, 1, wide, 62).view(2, wide)
        got = attend(c, x, [640, 500], hq, 0.09, q_stride=wide).double()
        ref, bound = reference(c, x[:, :hq * d].reshape(2, hq, d), [640, 500], hq, np.float32(0.09).item())
        assert torch.all((got - ref).abs() <= bound)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hq,hkv,d", [(16, 4, 128), (12, 1, 64), (24, 2, 256)])
def test_runs_are_equal_bit_for_bit(kind, hq, hkv, d):
    """Repeats, and calls with what other lengths left in the workspace."""
    torch = _t()
    lens = [700, 3, 0, 1500, 64, 9000]
    c = WideCache(kind, hkv, d, 16, lens, 71)
    q = queries(len(lens), hq, d, 72)
    first, ws = attend(c, q, lens, hq, 0.09), Workspace((c, hq))
    for i in range(6):
        if i % 2:
            attend(c, q, [5, 0, 0, 1500, 0, 8000 - 900 * i], hq, 0.09, ws=ws)
        assert torch.equal(attend(c, q, lens, hq, 0.09, ws=ws), first)


@pytest.mark.parametrize("kind", TYPES)
def test_one_launch_agrees(kind):
    """The same contents through a table of 2048 positions, which one launch of clusters takes."""
    torch = _t()
    lens, hq, hkv, d, ps = [2048, 700, 0, 31], 16, 2, 128, 16
    c = WideCache(kind, hkv, d, ps, lens, 81)
    q = queries(4, hq, d, 82)
    got = attend(c, q, lens, hq, 0.09)
    _, bound = reference(c, q, lens, hq, np.float32(0.09).item())
    table = c.table[:, :2048 // ps].contiguous()
    kv = ntx.make_paged_kv(kind, hkv, d, ps, c.n_pages, *c.pools, table, 4, 2048 // ps)
    n = ntx.ntx_attn_paged_workspace_bytes(kv, hq)
    out, ws = torch.empty_like(got), torch.empty(n, dtype=torch.uint8, device="cuda")
    ntx.ntx_attn_decode_paged(kv, q, hq * d, out, hq, torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.09, ws, n)
    assert torch.all((got - out).abs() <= 2 * bound)


# ------------------------------------------------------------------ graphs, streams, first calls
class WideDecoder(Decoder):
    """A decode step whose attention is on this path."""

    def __init__(self, kind, n, hq, hkv, d, ps, ctx, seed, ws=None):
        super().__init__(kind, n, hq, hkv, d, ps, ctx, seed)
        torch = _t()
        used = self.c.table
        table = torch.full((n, WIDE // ps), -1, dtype=torch.int32, device="cuda")
        table[:, :used.shape[1]] = used
        self.c.table = table
        self.c.kv = ntx.make_paged_kv(kind, hkv, d, ps, self.c.n_pages, *self.c.pools, table, n, WIDE // ps)
        self.own = ws or Workspace((self.c, hq))
        self.ws, self.ws_n = self.own.all, self.own.n


def test_two_captured_graphs_share_a_workspace():
    torch = _t()
    shape = [(Q8, 3, 8, 2, 128, 16, 1200, 91), (F16, 3, 24, 2, 64, 32, 1200, 92), (Q4, 3, 16, 1, 256, 16, 1200, 93)]
    alone = [WideDecoder(*s) for s in shape]
    shared = Workspace(*[(m.c, m.hq) for m in alone])
    captured = [WideDecoder(*s, ws=shared) for s in shape]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graphs = []
    for m in captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            m.step(torch.cuda.current_stream())
        graphs.append(g)
    torch.cuda.synchronize()
    assert torch.all(shared.all == 0xFF)  # a capture runs nothing
    for t in range(0, 1190, 110):
        for m, m2 in zip(captured, alone):
            x = torch.from_numpy(sg.fill_f32(94, f"x{t}{m.d}", m.n * m.wide)).cuda().view(m.n, -1)
            pos = torch.tensor([t, t // 2, -1 if t < 300 else t - 300], dtype=torch.int32, device="cuda")
            for y in (m, m2):
                y.x.copy_(x)
                y.pos.copy_(pos)
                y.len.copy_(pos + 1)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for g in graphs:
                g.replay()
        for m2 in alone:
            m2.step()
        torch.cuda.synchronize()
        for m, m2 in zip(captured, alone):
            assert torch.equal(m.out, m2.out) and torch.all(torch.isfinite(m.out))
            for i in range(2):
                assert torch.equal(m.c.pools[i], m2.c.pools[i])
    shared.check()
    for m2 in alone:
        m2.own.check()


def test_calls_on_two_streams_at_once():
    """Workspaces of their own, many calls in flight on either stream: neither disturbs the other."""
    torch = _t()
    cs = [WideCache(kind, hkv, d, 16, lens, 101) for kind, hkv, d, lens in
          ((Q4, 4, 128, [900] * 8), (F16, 1, 64, [2000, 3, 0, 700]))]
    hqs, lens = (16, 12), [[900 - 30 * i for i in range(8)], [2000, 3, 0, 700]]
    qs = [queries(len(n), hq, c.d, 102) for n, hq, c in zip(lens, hqs, cs)]
    want = [attend(c, q, n, hq, 0.1) for c, q, n, hq in zip(cs, qs, lens, hqs)]
    ws = [Workspace((c, hq)) for c, hq in zip(cs, hqs)]
    dev = [torch.tensor(n, dtype=torch.int32, device="cuda") for n in lens]
    outs = [[torch.full_like(w, float("nan")) for _ in range(20)] for w in want]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for j in range(2):
            ntx.ntx_attn_decode_paged(cs[j].kv, qs[j], hqs[j] * cs[j].d, outs[j][i], hqs[j], dev[j], 0.1, ws[j].all, ws[j].n,
                                      streams[j])
    torch.cuda.synchronize()
    for j in range(2):
        ws[j].check()
        for o in outs[j]:
            assert torch.equal(o, want[j])


FIRST_CALL_IN_A_CAPTURE = """
import sys
sys.path.insert(0, {root!r})
import torch
import quantized_weight_gemv_dequant_b200 as ntx
hkv, hq, d, ps, n = 2, 8, 128, 16, 600
pages = 640 // ps
pools = [torch.zeros(ntx.ntx_paged_kv_bytes(ntx.NTX_Q4_0, hkv, d, ps, pages), dtype=torch.uint8, device="cuda") for _ in range(2)]
table = torch.full((1, 1024), -1, dtype=torch.int32, device="cuda")
table[0, :pages] = torch.arange(pages, dtype=torch.int32, device="cuda")
kv = ntx.make_paged_kv(ntx.NTX_Q4_0, hkv, d, ps, pages, *pools, table, 1, 1024)
x = torch.randn(hq * d, device="cuda")
lens = torch.tensor([n], dtype=torch.int32, device="cuda")
ws_n = ntx.ntx_attn_paged_workspace_bytes(kv, hq)
ws, out = torch.full((ws_n,), 255, dtype=torch.uint8, device="cuda"), torch.full((hq, d), 5.0, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    ntx.ntx_attn_decode_paged(kv, x, hq * d, out, hq, lens, 0.1, ws, ws_n, torch.cuda.current_stream())
g.replay()
torch.cuda.synchronize()
assert torch.all(out == 0) and torch.any(ws != 255) and ntx.ntx_device_status() == 0
print("same")
"""


def test_first_call_of_a_process_inside_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_A_CAPTURE.format(root=root)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
