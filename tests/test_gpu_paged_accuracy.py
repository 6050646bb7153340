"""Paged attention over block types where a score's terms are small beside the
block's scale: keys with a channel far larger than the rest of its block, and
queries whose mean is not zero.

Two bounds.  The first is the worst case, as in test_gpu_paged.py.  The second
is a plain fp32 evaluation (products and sums one after the other) of the same
cache: every rounding of it is half a step of a partial sum at most, the matrix
instruction's truncations a whole one of the same partial sums, and q in two
fp16 numbers is off by half a step; so the kernel's error, as the root of the
mean square over all outputs, is at most twice the plain form's."""
import numpy as np
import pytest

import quantized_weight_gemv_dequant_b200 as ntx
from test_gpu_paged import F16, Q4, Q8, TYPES, Cache, _gpu, _t, attend, attention_ref, values_of  # noqa: F401

pytestmark = pytest.mark.gpu


def fp32_attention(cache, q, lens, hq, scale):
    """out [seqs, hq, D], every product and sum rounded to fp32."""
    g, f = hq // cache.hkv, np.float32
    out = np.zeros(q.shape, f)
    for s, n in enumerate(lens):
        k, v = (cache.seq_values(i, s, n).astype(f).repeat(g, 0) for i in range(2))
        x, o, l = np.zeros((hq, n), f), np.zeros((hq, cache.d), f), np.zeros((hq, 1), f)
        for j in range(cache.d):
            x += k[:, :, j] * q[s, :, j, None]
        x *= f(scale)
        p = np.exp(x - x.max(-1, keepdims=True))
        for j in range(n):
            o += p[:, j, None] * v[:, j]
            l += p[:, j, None]
        out[s] = o / l
    return out


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (16, 2, 128), (8, 1, 256)])
@pytest.mark.parametrize("outlier", [1.0, 30.0])
@pytest.mark.parametrize("there", [1.0, 0.0])  # what of the query is left in the large channels
@pytest.mark.parametrize("wide", [False, True])
def test_attention_of_queries_with_a_mean_over_uneven_keys(kind, hq, hkv, d, outlier, there, wide):
    """`wide`: a table of more positions than one launch takes, so the parts and their join."""
    torch = _t()
    lens, ps = [40, 2, 17, 33, 5, 64], 16
    c = Cache(kind, hkv, d, ps, lens, 11, max_pages=(1 << 14) // ps if wide else None)
    rs = np.random.RandomState(d + hq)
    n = sum(lens)
    w = [rs.standard_normal((n, hkv, d)).astype(np.float32) for _ in range(2)]
    large = np.arange(0, d, 32) + rs.randint(0, 32, d // 32)
    if kind == Q4:
        outlier = min(outlier, 8.0)  # beyond, the other codes are all zero
    w[0][..., large] *= np.float32(outlier)
    q = (1 + 0.3 * rs.standard_normal((len(lens), hq, d))).astype(np.float32)
    q[..., large] *= np.float32(there)
    seq = torch.from_numpy(np.repeat(np.arange(len(lens)), lens).astype(np.int32)).cuda()
    pos = torch.from_numpy(np.concatenate([np.arange(m) for m in lens]).astype(np.int32)).cuda()
    ntx.ntx_kv_append(c.kv, *[torch.from_numpy(x).cuda() for x in w], hkv * d, hkv * d, seq, pos, n)
    c.val = [values_of(kind, *c.host(i)) for i in range(2)]
    scale = np.float32(d ** -0.5).item()
    got = attend(c, torch.from_numpy(q).cuda(), lens, hq, scale).cpu().numpy().astype(np.float64)
    ref, bound = attention_ref(c, q, lens, hq, scale)
    assert np.all(np.abs(got - ref) <= bound)

    def off(x):
        return float(np.sqrt(np.mean((x - ref) ** 2)))

    assert off(got) <= 2 * off(fp32_attention(c, q, lens, hq, scale)), (off(got), off(fp32_attention(c, q, lens, hq, scale)))
