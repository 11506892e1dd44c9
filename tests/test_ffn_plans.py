"""Which tiles the sizes of test_gpu_gated_ffn_values.py get from the rules of gated_ffn.hip: a change of a rule that leaves
a kind of tile without a test fails here."""
import os
import subprocess

import pytest

from block_ref import BF, F32
from test_gpu_gated_ffn_values import SIZES
from test_host_sanitizers import HIPCC, ROOT

LARGE, MID, NARROW, FEW = range(4)  # 256 x 256, 128 x 128, 128 x 64, 32 x 64


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """Host code only: the kernels' device code, which no call here reaches, is not built."""
    at = tmp_path_factory.mktemp("plans")
    obj, exe = str(at / "ffn_plans.o"), str(at / "ffn_plans")
    subprocess.run([HIPCC, "-x", "hip", "--cuda-host-only", "-fPIC", "-O0", "-std=c++17", "--offload-arch=gfx950", "-I", f"{ROOT}/include",
                    "-c", f"{ROOT}/tests/sanitize/ffn_plans.cpp", "-o", obj], check=True, capture_output=True, timeout=300)
    names = subprocess.run(["nm", "-u", obj], check=True, capture_output=True, text=True).stdout.split()
    lib = os.path.join(os.path.dirname(os.path.dirname(HIPCC)), "lib")
    subprocess.run(["g++", obj, "-o", exe, f"-L{lib}", "-lamdhip64", f"-Wl,-rpath,{lib}"]
                   + [f"-Wl,--defsym={n}=0" for n in names if n.startswith("__hip_fatbin")], check=True, capture_output=True, timeout=300)
    lines = "".join(f"{M} {D} {F} {int(dtype is BF)}\n" for M, D, F, dtype in SIZES)
    out = subprocess.run([exe], input=lines, check=True, capture_output=True, text=True, timeout=60).stdout.splitlines()
    assert len(out) == len(SIZES)
    return [(size, [int(v) for v in line.split()]) for size, line in zip(SIZES, out)]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is not installed")
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_the_sizes_meet_every_kind_of_tile(plans, dtype):
    rows = [v for size, v in plans if size[3] is dtype]
    both = lambda kinds: {(k, cut) for k in kinds for cut in (False, True)}  # noqa: E731
    smaller, alone = (MID, NARROW, FEW), (LARGE, MID, NARROW, FEW)
    assert {(v[0], v[1] > 1) for v in rows} == both(alone)
    assert {(v[2], v[3] > 1) for v in rows} == both(alone)
    assert {(v[4], v[5] > 1) for v in rows} == both((LARGE, MID, NARROW))
    one = [v for v in rows if v[6]]
    assert {(v[7], v[9]) for v in one} == {(x, w) for x in smaller for w in (MID, NARROW)}
    assert {(v[7], v[8] > 1) for v in one} == both(smaller)
    assert {(v[9], v[10] > 1) for v in one} == both((MID, NARROW))
