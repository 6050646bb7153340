"""Infinities in the paged cache: an output that an infinite value reaches is infinite or NaN; a sequence's outputs over a
KV head with an infinite key are NaN, or those without that key's position (a score of minus infinity: F16, or a block's
infinite scale times its sum of q and codes, which counts as one product); every other output is what it is without.
On both paths of the attention (one launch, parts and their join)."""
import numpy as np
import pytest

import quantized_weight_gemv_dequant_b200 as ntx
import synthgen as sg
from test_gpu_paged import F16, STEP, TYPES, Cache, _gpu, _t, attend, values_of  # noqa: F401

pytestmark = pytest.mark.gpu

LENS, HQ, HKV, D, PS = [70, 90, 40], 8, 2, 64, 16
AT = (1, 50, 1, 37)  # sequence, position, KV head, element


def _append(kind, w, wide):
    torch = _t()
    c = Cache(kind, HKV, D, PS, LENS, 5, max_pages=(1 << 14) // PS if wide else None)
    seq = torch.from_numpy(np.repeat(np.arange(3), LENS).astype(np.int32)).cuda()
    pos = torch.from_numpy(np.concatenate([np.arange(m) for m in LENS]).astype(np.int32)).cuda()
    ntx.ntx_kv_append(c.kv, *[torch.from_numpy(x).cuda() for x in w], HKV * D, HKV * D, seq, pos, sum(LENS))
    c.val = [values_of(kind, *c.host(i)) for i in range(2)]
    return c


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("big", [1e20, -1e20])  # beyond any type's largest: an infinity, or a scale that is one
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("kind", TYPES)
def test_an_infinity_reaches_what_the_formula_gives_it(kind, which, big, wide):
    torch = _t()
    s, p, h, e = AT
    n = sum(LENS)
    w = [sg.fill_f32(6, nm, n * HKV * D).reshape(n, HKV, D) for nm in ("k", "v")]
    q = sg.fill_f32(7, "q", 3 * HQ * D).reshape(3, HQ, D)
    qd = torch.from_numpy(q).cuda()
    plain = _append(kind, w, wide)
    want = attend(plain, qd, LENS, HQ, 0.1).cpu().numpy()
    w[which][LENS[0] + p, h, e] = big
    c = _append(kind, w, wide)
    page, row = c.place(s, p)
    assert np.isinf(c.val[which][page, h, row, e])
    got = attend(c, qd, LENS, HQ, 0.1).cpu().numpy()
    mine = np.zeros(got.shape, bool)  # the outputs of the sequence's query heads over that KV head
    mine[s, h * (HQ // HKV):(h + 1) * (HQ // HKV)] = True
    assert np.array_equal(got[~mine], want[~mine])
    if which == 0:
        scale = np.float32(0.1).item()
        k, v = (np.delete(c.seq_values(i, s, LENS[s])[h], p, 0) for i in range(2))
        for head in range(h * (HQ // HKV), (h + 1) * (HQ // HKV)):
            a = q[s, head].astype(np.float64)
            x = scale * (k @ a)
            weight = np.exp(x - x.max())
            weight /= weight.sum()
            ds = (D + 8) * STEP * scale * (np.abs(k) @ np.abs(a)).max() + 4 * STEP * np.abs(x).max()
            bound = (2 * ds + (len(k) / 16 + 64) * STEP) * (weight @ np.abs(v)) + (len(k) * 2.0 ** -35 + 2.0 ** -29) * np.abs(v).max()
            assert np.isnan(got[s, head]).all() or np.all(np.abs(got[s, head] - weight @ v) <= bound)
    else:
        cols = np.zeros(got.shape, bool)
        if kind == F16:
            cols[..., e] = True
        else:
            cols[..., e // 32 * 32:e // 32 * 32 + 32] = True
        assert not np.isfinite(got[mine & cols]).any()
        assert np.isfinite(got[mine & ~cols]).all()
        if kind == F16:  # (a block's infinite scale is also its chunk's largest)
            assert np.array_equal(got[mine & ~cols], want[mine & ~cols])
