"""Host-side checks of the paged cache calls: sizes and refusals, each before
any device work (CPU only: no call here reaches a launch)."""
import ctypes
import itertools

import pytest

import quantized_weight_gemv_dequant_b200 as ntx

FAKE = 0x7F0000000000  # never dereferenced: every call below fails its argument check, or does nothing
TYPES = (ntx.NTX_F16, ntx.NTX_Q8_0, ntx.NTX_Q4_0)
INV, SHAPE, QTYPE, ALIGN, NOMEM = (ntx.NTX_ERR_INVALID_ARG, ntx.NTX_ERR_SHAPE, ntx.NTX_ERR_QTYPE, ntx.NTX_ERR_ALIGN,
                                   ntx.NTX_ERR_NOMEM)


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_weight_gemv_dequant_b200 import build
    build.build()


def _rc(fn, *args):
    try:
        fn(*args)
    except ntx.NtxError as e:
        return e.code
    return 0


def _kv(**change):
    a = dict(type=ntx.NTX_Q8_0, n_kv_heads=8, head_dim=128, page_size=64, n_pages=100, k_pages=FAKE,
             v_pages=FAKE + 0x1000000, page_table=FAKE + 0x2000000, n_seqs=4, max_pages=20)
    a.update(change)
    return ntx.make_paged_kv(**a)


def test_pool_bytes_closed_forms():
    for (t, per32), h, d, ps, n in itertools.product(((ntx.NTX_F16, 64), (ntx.NTX_Q8_0, 34), (ntx.NTX_Q4_0, 18)),
                                                     (1, 8), (64, 128, 256), (16, 48, 4096), (1, 77)):
        assert ntx.ntx_paged_kv_bytes(t, h, d, ps, n) == n * ps * h * d // 32 * per32
    assert ntx.ntx_paged_kv_bytes(ntx.NTX_F16, 8, 128, 16, 2 ** 31 - 1) == (2 ** 31 - 1) * 16 * 8 * 256


@pytest.mark.parametrize("change,code", [
    (dict(type=ntx.NTX_F32), QTYPE), (dict(type=ntx.NTX_Q6_K), QTYPE), (dict(type=-1), QTYPE),
    (dict(head_dim=96), SHAPE), (dict(head_dim=0), SHAPE), (dict(head_dim=512), SHAPE),
    (dict(n_kv_heads=0), SHAPE), (dict(n_kv_heads=1025), SHAPE),
    (dict(page_size=8), SHAPE), (dict(page_size=40), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=-16), SHAPE),
    (dict(n_pages=0), SHAPE), (dict(n_seqs=0), SHAPE), (dict(n_seqs=1025), SHAPE), (dict(max_pages=0), SHAPE),
    (dict(max_pages=2 ** 25), SHAPE),
    (dict(k_pages=None), INV), (dict(v_pages=None), INV), (dict(page_table=None), INV),
    (dict(k_pages=FAKE + 8), ALIGN), (dict(v_pages=FAKE + 2), ALIGN), (dict(page_table=FAKE + 2), ALIGN),
])
def test_every_call_refuses_a_bad_cache(change, code):
    kv = _kv(**change)
    f = [FAKE + 0x3000000, FAKE + 0x4000000]
    assert _rc(ntx.ntx_kv_append, kv, *f, 8192, 8192, None, FAKE, 2) == code
    assert _rc(ntx.ntx_kv_read, kv, *f, 8192, 8192, None, FAKE, 2) == code or change.get("n_seqs") == 1
    hq = 4 * max(1, change.get("n_kv_heads", 8))
    assert _rc(ntx.ntx_attn_decode_paged, kv, f[0], hq * 512, f[1] + 2 ** 40, hq, FAKE, 0.1, FAKE, 1 << 40) == code
    if code == SHAPE and set(change) & {"head_dim", "n_kv_heads", "page_size", "n_pages"}:
        a = dict(n_kv_heads=8, head_dim=128, page_size=64, n_pages=100)
        a.update(change)
        assert _rc(ntx.ntx_paged_kv_bytes, ntx.NTX_Q8_0, *a.values()) == INV


def test_append_and_read_argument_errors():
    kv = _kv()
    k, v, ids, pos = (FAKE + i * 0x1000000 for i in range(3, 7))
    for fn in (ntx.ntx_kv_append, ntx.ntx_kv_read):
        assert _rc(fn, None, k, v, 1024, 1024, ids, pos, 2) == INV
        assert _rc(fn, kv, k, v, 1023, 1024, ids, pos, 2) == SHAPE
        assert _rc(fn, kv, k, v, 1024, 1000, ids, pos, 2) == SHAPE
        assert _rc(fn, kv, k, v, 1024, -1024, ids, pos, 2) == SHAPE
        assert _rc(fn, kv, k, v, 1024, 1024, ids, pos, -1) == SHAPE
        assert _rc(fn, kv, k, v, 1024, 1024, None, pos, 5) == SHAPE  # 5 tokens, 4 sequences
        assert _rc(fn, kv, k, v, 1024, 1024, ids, None, 2) == INV
        assert _rc(fn, kv, k + 2, v, 1024, 1024, ids, pos, 2) == ALIGN
        assert _rc(fn, kv, k, v, 1024, 1024, ids + 1, pos, 2) == ALIGN
        assert _rc(fn, kv, k, v, 1024, 1024, ids, pos + 2, 2) == ALIGN
        assert _rc(fn, kv, k, v, 1024, 1024, ids, None, 0) == 0  # nothing to do
    assert _rc(ntx.ntx_kv_append, kv, None, v, 1024, 1024, ids, pos, 2) == INV
    assert _rc(ntx.ntx_kv_append, kv, k, None, 1024, 1024, ids, pos, 2) == INV
    assert _rc(ntx.ntx_kv_read, kv, None, None, 0, 0, ids, pos, 2) == 0  # nothing asked for


def test_attention_argument_errors():
    kv = _kv()
    q, out, lens, ws = FAKE + 0x3000000, FAKE + 0x4000000, FAKE, FAKE + 0x5000000
    n = ntx.ntx_attn_paged_workspace_bytes(kv, 32)
    assert n > 0
    ok = [kv, q, 4096, out, 32, lens, 0.1, ws, n]

    def rc(**change):
        names = ["kv", "q", "stride", "out", "hq", "lens", "scale", "ws", "bytes"]
        a = dict(zip(names, ok))
        a.update(change)
        return _rc(ntx.ntx_attn_decode_paged, *a.values())

    assert rc(kv=None) == INV and rc(q=None) == INV and rc(out=None) == INV and rc(lens=None) == INV
    assert rc(ws=None) == INV and rc(scale=float("nan")) == INV and rc(scale=float("inf")) == INV
    assert rc(hq=31) == SHAPE and rc(hq=0) == SHAPE and rc(hq=-8) == SHAPE and rc(hq=8 * 65, stride=1 << 20) == SHAPE
    assert rc(stride=4092) == SHAPE
    assert rc(stride=4098) == ALIGN and rc(q=q + 4) == ALIGN and rc(out=out + 8) == ALIGN and rc(ws=ws + 4) == ALIGN
    assert rc(lens=lens + 2) == ALIGN
    assert rc(out=q) == INV and rc(out=q + 3 * 4096 * 4) == INV and rc(out=q - 4 * 4096 * 4 + 16) == INV
    assert rc(bytes=n - 1) == NOMEM
    assert "workspace" in ntx.ntx_last_error()
    assert ntx.ntx_attn_paged_workspace_bytes(kv, 31) == 0
    assert ntx.ntx_attn_paged_workspace_bytes(_kv(head_dim=96), 32) == 0
    assert ntx.lib().ntx_attn_paged_workspace_bytes(None, 32) == 0


def test_norm_rope_argument_errors():
    q, k, qo, ko, wq, wk, pos = (FAKE + i * 0x1000000 for i in range(7))
    ok = dict(q=q, k=k, qo=qo, ko=ko, qs=4096, ks=1024, wq=wq, wk=wk, pos=pos, n=3, hq=32, hk=8, d=128, r=128, pair=0,
              theta=5e5, eps=1e-6)

    def rc(**change):
        return _rc(ntx.ntx_qk_norm_rope, *{**ok, **change}.values())

    assert rc(d=127) == SHAPE and rc(d=0) == SHAPE and rc(d=258) == SHAPE
    assert rc(r=129) == SHAPE and rc(r=63) == SHAPE and rc(r=-2) == SHAPE and rc(r=130) == SHAPE
    assert rc(n=-1) == SHAPE and rc(hq=-1) == SHAPE and rc(hk=-1) == SHAPE
    assert rc(qs=4095) == SHAPE and rc(ks=1023) == SHAPE
    assert rc(pair=2) == INV and rc(pair=-1) == INV
    assert rc(theta=0.0) == INV and rc(theta=float("nan")) == INV and rc(theta=float("inf")) == INV
    assert rc(eps=-1e-6) == INV and rc(eps=float("nan")) == INV
    assert rc(pos=None) == INV and rc(q=None) == INV and rc(ko=None) == INV
    assert rc(q=q + 2) == ALIGN and rc(wk=wk + 1) == ALIGN and rc(pos=pos + 2) == ALIGN
    assert rc(qo=q + 16) == INV and rc(ko=k - 16) == INV  # neither in place nor apart
    assert rc(n=0) == 0 and rc(n=0, pos=None) == 0
    assert rc(hq=0, hk=0) == 0  # nothing to do


def test_struct_matches_the_header():
    # seven int32, padding to 8, three pointers
    assert ctypes.sizeof(ntx.ntx_paged_kv) == 56 and ntx.ntx_paged_kv.k_pages.offset == 32
