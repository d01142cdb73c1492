"""The shapes that the GPU tests check against fp64 come to every form of the 8-bit float product
kernels that any call can come to (no GPU): the entry points run against stand-ins of their launchers
(sanitize/fp8_forms.cpp), once for the lists of shapes and once over all sizes, so that a cost or a
limit changed in fp8_launch.h cannot leave a form unchecked."""
import os
import re
import shutil
import subprocess

import pytest

import test_fp8_forms_gpu as more
import test_fp8_gpu as first
from test_resource_usage import _report

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = os.path.join(ROOT, "tests", "sanitize")
CSRC = os.path.join(ROOT, "packed_int4_convrot_amd", "csrc")

pytestmark = pytest.mark.skipif(not shutil.which("g++"), reason="host compiler g++ not found")


@pytest.fixture(scope="module")
def forms(tmp_path_factory):
    """What the driver prints for its commands, line by line."""
    exe = str(tmp_path_factory.mktemp("forms") / "fp8_forms")
    sources = [os.path.join(SAN, f) for f in ("fp8_forms.cpp", "stub_launch.cpp")]
    sources += [os.path.join(CSRC, f) for f in ("ck_api.cpp", "ck_fp8_api.cpp")]
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", *sources, "-o", exe],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr

    def run(commands):
        r = subprocess.run([exe], input="\n".join(commands), capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stdout + r.stderr
        assert "refused" not in r.stdout + r.stderr, r.stdout + r.stderr
        return r.stdout.splitlines()
    return run


@pytest.fixture(scope="module")
def reachable(forms):
    """Every form, with a call that comes to it."""
    return dict(line.split(": ") for line in forms(["sweep"]))


def test_the_gpu_tests_check_every_form(forms, reachable):
    calls = ["linear %d %d %d" % s for s in first.LINEARS + more.LINEARS]
    calls += ["%s %d %d %d" % (op, *s) for op in ("ffn", "backward") for s in first.BLOCKS + more.BLOCKS]
    lines = forms(calls)
    assert len(lines) == len(calls)
    checked = {f for line in lines for f in line.split("; ") if f}
    missing = {f: call for f, call in reachable.items() if f not in checked}
    assert not missing, missing
    assert len(reachable) > 60


def test_no_kernel_is_compiled_that_no_call_reaches(reachable):
    """The kernels in the build's report, by their template arguments."""
    kinds, compiled = ("bf16", "gated", "grad", "sums"), set()
    for k in _report()["kernels"]:
        few = re.search(r"fp8_few_kernelILNS0_6SourceE(\d)ELNS_9Fp8ResultE(\d)ELi(\d)ELi(\d+)E", k["kernel"])
        tiled = re.search(r"fp8_tiled_kernelINS0_4TileI(?:Li(\d)E)(?:Li(\d)E)(?:Li(\d)E)(?:Li(\d)E)Li\dEEELNS_9Fp8ResultE(\d)E",
                          k["kernel"])
        if few:
            source, kind, rows16, tiles = map(int, few.groups())
            compiled.add("few %s %s %d %d" % (("codes", "raw", "fp32")[source], kinds[kind], rows16,
                                              tiles // (2 if kinds[kind] == "gated" else 1)))
        elif tiled:
            wn, wm, tn, tm, kind = map(int, tiled.groups())
            compiled.add("tiled %dx%d %s" % (32 * wn * tn, 32 * wm * tm, kinds[kind]))
        else:
            assert "fp8_few" not in k["kernel"] and "fp8_tiled" not in k["kernel"], k["kernel"]
    assert compiled == {f.replace(" passes", "").replace(" runs", "") for f in reachable}
