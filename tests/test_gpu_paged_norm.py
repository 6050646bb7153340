"""Head norm with rotation where a warp takes several rows of a token and several tokens: from about 38000 rows on
(592 CTAs of 8 warps, eight rounds), which the small shapes of test_gpu_paged.py do not reach.  The same reference in
fp64, here on the device, and the same bound, 2e-6 of |a| + |b| of an output's pair."""
import numpy as np
import pytest

import quantized_weight_gemv_dequant_b200 as ntx
from test_gpu_paged import _gpu, _t  # noqa: F401

pytestmark = pytest.mark.gpu

THETA, EPS = 5e5, 1e-6


def reference(x, w, pos, rot, halves):
    """x fp32 [n, heads, D]; (out, size of each output's terms) in fp64."""
    torch = _t()
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + float(np.float32(EPS)))
    if w is not None:
        y = y * w.double()
    i = np.arange(rot // 2)
    f = torch.from_numpy(np.power(np.float64(np.float32(THETA)), -2.0 * i / max(rot, 1))).cuda()
    a = pos.double()[:, None, None] * f
    c, s = torch.cos(a), torch.sin(a)
    e0, e1 = (slice(0, rot // 2), slice(rot // 2, rot)) if halves else (slice(0, rot, 2), slice(1, rot, 2))
    out, size = y.clone(), y.abs()
    out[..., e0], out[..., e1] = y[..., e0] * c - y[..., e1] * s, y[..., e0] * s + y[..., e1] * c
    size[..., e0] = size[..., e1] = y[..., e0].abs() + y[..., e1].abs()
    return out, size


# heads and tokens: rows to a warp, and what is left for a token's last share
SHAPES = [
    (8192, 64, 8, 128, 128),  # 16 rows, in fours
    (2100, 20, 5, 64, 64),    # 2 rows, the last share 1
    (700, 100, 31, 64, 64),   # 3 rows, the last share 2; shares across queries and keys
    (2000, 33, 7, 256, 256),  # 3 rows of 256
    (4000, 33, 7, 256, 256),  # more than 4
    (3000, 64, 8, 128, 64),   # part of the head rotated: in halves without 16-byte accesses
    (9000, 7, 3, 80, 80),     # a head that is no power of two
    (9001, 5, 0, 64, 32),     # queries alone
    (9001, 0, 7, 128, 128),   # keys alone
    (50001, 1, 0, 64, 64),    # one row to a token, several tokens to a warp
    (30011, 1, 1, 256, 256),  # a query's row and a key's to a warp
    (300, 300, 11, 128, 128),
    (1, 65536, 1024, 64, 64),  # all of one token
]


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,hq,hk,d,rot", SHAPES)
def test_norm_rope_of_many_rows(n, hq, hk, d, rot, halves, in_place):
    torch = _t()
    gen = torch.Generator(device="cuda").manual_seed(n + d)
    pos = torch.randint(0, 131072, (n,), generator=gen, device="cuda", dtype=torch.int32)
    if n > 1:
        pos[torch.rand(n, generator=gen, device="cuda") < 0.05] = -1
        pos[n // 2] = 1 << 20
    size = [h * d for h in (hq, hk)]
    wide = sum(size) + (8 if in_place else 0)  # in place: q and k in the rows of one buffer
    x = torch.randn((n, wide), generator=gen, device="cuda") * torch.exp2(
        torch.randint(-6, 7, (n, 1), generator=gen, device="cuda").float())
    w = [1 + 0.2 * torch.randn(d, generator=gen, device="cuda") for _ in range(2)]
    parts = [x[:, :size[0]], x[:, size[0]:sum(size)]]
    if in_place:
        src = x.clone()
        dst, stride = [src.view(-1), src.view(-1)[size[0]:]], [wide, wide]
        inp = dst
    else:
        inp = [p.contiguous() for p in parts]
        dst, stride = [torch.full_like(p, 7.0) for p in inp], size
    ptr = [[t if s else None for t, s in zip(ts, size)] for ts in (inp, dst)]
    ntx.ntx_qk_norm_rope(*ptr[0], *ptr[1], *stride, *w, pos, n, hq, hk, d, rot, int(halves), THETA, EPS)
    if in_place:
        assert torch.equal(src[:, sum(size):], x[:, sum(size):])
        got = [src[:, :size[0]], src[:, size[0]:sum(size)]]
    else:
        got = dst
        for a, b in zip(inp, parts):
            assert torch.equal(a, b)
    for g, p, h, weight in zip(got, parts, (hq, hk), w):
        if h == 0:
            continue
        g, live = g.reshape(n, h, d), pos >= 0
        unused = g[~live]
        assert torch.equal(unused, p.reshape(n, h, d)[~live]) if in_place else torch.all(unused == 7)
        for t in range(0, n, 2048):  # a piece at a time: fp64
            on = live[t:t + 2048]
            ref, terms = reference(p.reshape(n, h, d)[t:t + 2048][on], weight, pos[t:t + 2048][on], rot, halves)
            assert torch.all((g[t:t + 2048][on] - ref).abs() <= 2e-6 * terms)
