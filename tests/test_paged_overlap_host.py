"""Refusals of overlapping rows by the paged cache's calls (CPU: every call here is refused before a launch)."""
import pytest

import quantized_weight_gemv_dequant_b200 as ntx

FAKE = 0x7F0000000000  # never dereferenced


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


@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("case", ["q_out over k", "k_out over q", "q_out over k_out", "swapped", "q_out over the next q row",
                                  "k_out inside q's row", "one float"])
def test_norm_rope_refuses_outputs_over_other_rows(case, n):
    """One buffer of rows of 40 heads of 64: queries in heads 0 to 31, keys in 32 to 39, or apart."""
    d, hq, hk = 64, 32, 8
    wide = (hq + hk) * d
    q, k, far = FAKE, FAKE + hq * d * 4, FAKE + (1 << 30)
    qo, ko = {
        "q_out over k": (k, far), "k_out over q": (far, q), "q_out over k_out": (far, far + 64), "swapped": (k, q),
        "q_out over the next q row": (q + wide * 4 - 4, far) if n > 1 else (q + 4, far),
        "k_out inside q's row": (q, q + 5 * d * 4), "one float": (far, q + (hq * d - 1) * 4)}[case]
    assert _rc(ntx.ntx_qk_norm_rope, q, k, qo, ko, wide, wide, None, None, FAKE + (1 << 31), n, hq, hk, d, d, 0, 1e4,
               1e-6) == ntx.NTX_ERR_INVALID_ARG
    assert "overlaps" in ntx.ntx_last_error()


def test_norm_rope_refuses_rows_of_different_strides_that_meet():
    """Keys at 0, 200, 400 and 600 floats of a buffer, outputs of 64 floats from 600 on in steps of 100."""
    d = 64
    q, k, far = FAKE, FAKE + (1 << 30), FAKE + (1 << 31)
    assert _rc(ntx.ntx_qk_norm_rope, q, k, k + 4 * 500 + 400, far, 100, 200, None, None, far + (1 << 30), 4, 1, 1, d, d, 0, 1e4,
               1e-6) == ntx.NTX_ERR_INVALID_ARG


def test_attention_refuses_an_output_over_a_query_row():
    kv = ntx.make_paged_kv(ntx.NTX_F16, 2, 64, 16, 4, FAKE, FAKE + (1 << 20), FAKE + (2 << 20), 2, 2)
    n = ntx.ntx_attn_paged_workspace_bytes(kv, 4)
    q, stride = FAKE + (3 << 20), 1024
    for out in (q, q + (1024 - 512 + 4) * 4, q + 1024 * 4 + 240 * 4, q - 512 * 4 + 16, q + 768 * 4):
        assert _rc(ntx.ntx_attn_decode_paged, kv, q, stride, out, 4, FAKE, 0.1, FAKE + (4 << 20), n) == \
            ntx.NTX_ERR_INVALID_ARG
