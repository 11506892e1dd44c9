"""abi_layers.cpp (chunked delta rule, its one-token form, layer norm) under
AddressSanitizer and UndefinedBehaviorSanitizer on the host pass, with
tests/sanitize/layer_checks.cpp: the validation paths and the workspace plans at
the largest sizes that are accepted.  No call reaches a launch."""
import os
import subprocess

import pytest

from test_host_sanitizers import CSRC, HIPCC, ROOT, SAN_ENV, _clean, _run

SOURCES = ["abi.cpp", "abi_layers.cpp", "delta_step.hip", "delta_chunk.hip", "delta_chunk_bwd.hip", "layer_norm.hip",
           "scan_seq.hip", "ssd_chunk.hip", "ssd_chunk16.hip", "ssd_blocked.hip", "ssd_fwd.hip", "delta_rule.hip",
           "noalloc.hip", "finite.hip", "ssd_pad.hip"]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is not installed")
def test_layer_host_code_under_sanitizers(tmp_path):
    flags = ["-O1", "-g", "-std=c++17", "-fPIC", "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=undefined", "-I", os.path.join(ROOT, "include")]
    sources = [os.path.join(CSRC, s) for s in SOURCES] + [os.path.join(ROOT, "tests", "sanitize", "layer_checks.cpp")]
    objs, procs = [], []
    for src in sources:
        objs.append(str(tmp_path / (os.path.basename(src).split(".")[0] + ".o")))
        procs.append(subprocess.Popen([HIPCC, "-x", "hip", "-c", src, "-o", objs[-1]] + flags,
                                      stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True))
    for p in procs:
        _, err = p.communicate()
        assert p.returncode == 0, err[-4000:]
    exe = str(tmp_path / "layer_checks")
    _run([HIPCC, "-fsanitize=address,undefined", "--offload-arch=gfx950", "-o", exe] + objs)
    env = dict(SAN_ENV)
    env.pop("SSMVJP_CHECK_FINITE", None)
    res = _run([exe], env=env, timeout=300)
    _clean(res)
    assert "0 failure(s)" in res.stdout
