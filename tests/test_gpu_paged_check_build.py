"""The paged cache's calls in the bounds-checked debug build: every index check passes, places outside the cache are
still the kernels' own to refuse, and every output and pool byte is the release build's (check_paged_run.py)."""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def _run(lib, out):
    r = subprocess.run([sys.executable, os.path.join(HERE, "check_paged_run.py"), out], env=dict(os.environ, NTX_LIB=lib),
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    with np.load(out) as z:
        return {k: z[k] for k in z.files}


def test_paged_calls_pass_the_checks_and_match_release(tmp_path):
    from quantized_weight_gemv_dequant_b200 import build
    rel = _run(build.build(), str(tmp_path / "release.npz"))
    chk = _run(build.build_check(), str(tmp_path / "check.npz"))
    assert int(rel["check_enabled"][0]) == 0 and int(chk["check_enabled"][0]) == 1
    assert int(chk["check_site"][0]) == 0, (int(chk["check_site"][0]), int(chk["check_index"][0]))
    assert set(rel["statuses"]) == {0, 5} and rel.keys() == chk.keys()
    for k in rel:
        if not k.startswith("check_"):
            assert rel[k].shape == chk[k].shape and rel[k].tobytes() == chk[k].tobytes(), k
