"""Which rows of one buffer the paged cache's calls accept as outputs, against a byte-by-byte comparison."""
import numpy as np
import pytest

import quantized_weight_gemv_dequant_b200 as ntx
import synthgen as sg
from test_gpu_paged import F16, Cache, _gpu, _t, attend  # noqa: F401

pytestmark = pytest.mark.gpu


def test_norm_rope_takes_any_rows_that_do_not_meet():
    """400 random layouts of q, k and their outputs in one buffer, strides equal or not: a call is refused exactly where an
    output meets other rows, and otherwise leaves the outputs of a call with buffers of its own and nothing else."""
    torch = _t()
    rs = np.random.RandomState(3)
    size, d, hk = 2000, 8, 1
    data = torch.from_numpy(sg.fill_f32(4, "x", size)).cuda()
    took = {False: 0, True: 0}
    for _ in range(400):
        n, hq = int(rs.randint(1, 6)), int(rs.randint(1, 3))
        width = [hq * d, hk * d]
        stride = [w + int(rs.choice([0, 3, 8, 40, 120, 200])) for w in width]
        if rs.rand() < 0.6:
            stride = [max(stride)] * 2
        at = [int(rs.randint(0, min(size - (n - 1) * s - w, 260))) for s, w in zip(stride, width)] * 2
        for i in range(2):
            if rs.rand() < 0.6:  # not in place
                at[2 + i] = int(rs.randint(0, min(size - (n - 1) * stride[i] - width[i], 400)))
        cells = [{a + t * stride[i % 2] + e for t in range(n) for e in range(width[i % 2])} for i, a in enumerate(at)]
        q, k, qo, ko = cells
        meet = bool((q & qo and at[0] != at[2]) or (k & ko and at[1] != at[3]) or q & ko or k & qo or qo & ko)
        took[meet] += 1
        b = data.clone()
        pos = torch.arange(n, dtype=torch.int32, device="cuda") * 37
        args = (*stride, None, None, pos, n, hq, hk, d, d, int(rs.randint(0, 2)), 1e4, 1e-6)
        try:
            ntx.ntx_qk_norm_rope(*[b[a:] for a in at], *args)
            refused = False
        except ntx.NtxError as e:
            assert e.code == ntx.NTX_ERR_INVALID_ARG
            refused = True
        assert refused == meet, (at, stride, width, n)
        want = data.clone()
        if not refused:
            src, out = data.clone(), [torch.zeros(size, device="cuda") for _ in range(2)]
            ntx.ntx_qk_norm_rope(src[at[0]:], src[at[1]:], out[0][at[2]:], out[1][at[3]:], *args)
            for i in range(2):
                idx = torch.tensor(sorted(cells[2 + i]), device="cuda")
                want[idx] = out[i][idx]
        assert torch.equal(b, want)
    assert min(took.values()) > 50  # both kinds are among them


def test_attention_output_between_query_rows():
    torch = _t()
    lens, hq, hkv, d = [20, 33], 4, 2, 64
    c = Cache(F16, hkv, d, 16, lens, 5).fill(6)
    w = hq * d
    x = torch.from_numpy(sg.fill_f32(7, "q", 5 * w)).cuda()
    want = attend(c, x, lens, hq, 0.1, q_stride=4 * w)
    got = attend(c, x, lens, hq, 0.1, q_stride=4 * w, out=x[w + 8:w + 8 + 2 * w].view(2, hq, d))
    assert torch.equal(got, want)
    back = torch.from_numpy(sg.fill_f32(7, "q", 5 * w)).cuda()
    assert torch.equal(x[:w + 8], back[:w + 8]) and torch.equal(x[3 * w + 8:], back[3 * w + 8:])
