"""The FA_DEBUG_BOUNDS build on the paged-cache operators: small ragged cases of every entry point run with no check
failing and outputs identical, bit for bit, to the ordinary build's."""
import os
import subprocess
import sys

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "quantized_attention_amax_b200", "csrc")


def test_paged_kernels_check_their_indices():
    """Every kernel file has checks, and points them at the status word before its launches."""
    for f in ("rope.cu", "paged_decode.cu", "paged_chunk.cu", "paged_weights.cu", "paged_evict.cu"):
        src = open(os.path.join(CSRC, f)).read()
        assert src.count("bounds_attach()") >= 1 and src.count("in_bounds(") + src.count(".holds(") >= 1, f


@pytest.mark.gpu
def test_bounds_build_runs_the_paged_entry_points_clean(tmp_path):
    from quantized_attention_amax_b200 import build
    build.build()
    build.build(bounds=True)
    outs = {}
    for lib in ("bounds", "release"):
        env = dict(os.environ)
        env.pop("FAQ_LIB", None)
        if lib == "bounds":
            env["FAQ_LIB"] = "bounds"
        path = str(tmp_path / f"{lib}.npz")
        r = subprocess.run([sys.executable, os.path.join(HERE, "_bounds_paged_cases.py"), path], capture_output=True, text=True,
                           timeout=600, env=env, cwd=ROOT)
        assert r.returncode == 0, r.stdout + r.stderr  # FA_ERR_BOUNDS would raise here
        outs[lib] = dict(np.load(path))
    assert outs["bounds"].keys() == outs["release"].keys() and len(outs["release"]) > 200
    for name in outs["release"]:
        a, b = outs["bounds"][name], outs["release"][name]
        assert a.dtype == b.dtype and a.tobytes() == b.tobytes(), name
