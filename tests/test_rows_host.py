"""Checks without a GPU of the operators that choose weights row by row: the
router, the mixture-of-experts layer and the low-rank adapters refuse bad
arguments before anything is enqueued, their workspace sizes follow from the
sizes alone, and their host code runs clean under AddressSanitizer and
UndefinedBehaviorSanitizer (a driver with stand-ins for the launchers).

The fake device pointers are never dereferenced: every call here fails
validation, or has no rows.
"""
import json
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = os.path.join(ROOT, "tests", "sanitize")
CSRC = os.path.join(ROOT, "packed_int4_convrot_amd", "csrc")

ck = pytest.importorskip("packed_int4_convrot_amd")
lib = ck.lib

INVALID, UNSUPPORTED, WORKSPACE = ck.CK_ERR_INVALID_ARG, ck.CK_ERR_UNSUPPORTED, 3


def at(i):
    """The i-th of a row of 256-byte aligned fake addresses, 256 MiB apart."""
    return 0x100000000 + i * 0x10000000


def route(logits=at(0), kind=0, T=4, E=100, ldl=100, k=4, renorm=1, ids=at(1), weights=at(2)):
    return lib.ck_moe_route(logits, kind, T, E, ldl, k, renorm, ids, weights, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID),
    (dict(T=2 ** 22), UNSUPPORTED),
    (dict(E=0), INVALID),
    (dict(E=1025, ldl=1025), UNSUPPORTED),
    (dict(k=0), INVALID),
    (dict(k=33), UNSUPPORTED),
    (dict(kind=2), INVALID),
    (dict(ldl=99), INVALID),
    (dict(logits=None), INVALID),
    (dict(logits=at(0) + 2), INVALID),
    (dict(logits=at(0) + 1, kind=1), INVALID),
    (dict(ids=None), INVALID),
    (dict(ids=at(1) + 2), INVALID),
    (dict(weights=None), INVALID),
    (dict(weights=at(2) + 1), INVALID),
    (dict(ids=at(0) + 3 * 400), INVALID),           # the last row of the logits
    (dict(weights=at(0)), INVALID),
    (dict(weights=at(1) + 4 * 4 * 4 - 4), INVALID),  # the last slot of ids
])
def test_route_refuses(kw, status):
    assert route(**kw) == status
    assert b"ck_moe_route" in lib.ck_last_error_msg()


def test_route_without_tokens():
    assert route(T=0, logits=None, ids=None, weights=None) == ck.CK_OK


SPACE = lib.ck_moe_workspace_bytes(3, 128, 8, 2)
MOE = dict(x=at(0), T=3, H=256, ldx=256, logits=at(1), kind=0, ldl=8, k=2, renorm=1, E=8, I=128, Gw=64, w1=at(2),
           s1=at(3), z1=at(4), w2=at(5), s2=at(6), z2=at(7), out=at(8), ldo=256, ids=at(9), weights=at(10),
           ws=at(11), ws_bytes=SPACE)


def moe(**kw):
    a = dict(MOE, **kw)
    return lib.ck_moe_w4a16(a["x"], a["T"], a["H"], a["ldx"], a["logits"], a["kind"], a["ldl"], a["k"], a["renorm"],
                            a["E"], a["I"], a["Gw"], a["w1"], a["s1"], a["z1"], a["w2"], a["s2"], a["z2"], a["out"],
                            a["ldo"], a["ids"], a["weights"], a["ws"], a["ws_bytes"], None)


def moe_experts(**kw):
    a = dict(MOE, **kw)
    return lib.ck_moe_experts_w4a16(a["x"], a["T"], a["H"], a["ldx"], a["ids"], a["weights"], a["k"], a["E"], a["I"],
                                    a["Gw"], a["w1"], a["s1"], a["z1"], a["w2"], a["s2"], a["z2"], a["out"],
                                    a["ldo"], a["ws"], a["ws_bytes"], None)


MOE_BAD = [
    (dict(T=-1), INVALID),
    (dict(T=2 ** 22), UNSUPPORTED),
    (dict(H=0), INVALID),
    (dict(H=96, ldx=96, ldo=96), INVALID),
    (dict(H=32832, ldx=32832, ldo=32832), UNSUPPORTED),
    (dict(I=0), INVALID),
    (dict(I=100), INVALID),
    (dict(I=32832), UNSUPPORTED),
    (dict(E=0), INVALID),
    (dict(E=1025, ldl=1025), UNSUPPORTED),
    (dict(k=0), INVALID),
    (dict(k=33), UNSUPPORTED),
    (dict(Gw=128), UNSUPPORTED),
    (dict(x=None), INVALID),
    (dict(x=at(0) + 8), INVALID),
    (dict(ldx=248), INVALID),
    (dict(ldx=260), INVALID),
    (dict(out=None), INVALID),
    (dict(out=at(8) + 2), INVALID),
    (dict(ldo=128), INVALID),
    (dict(ldo=260), INVALID),
    (dict(ids=None), INVALID),
    (dict(weights=at(10) + 2), INVALID),
    (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=SPACE - 1), WORKSPACE),
    (dict(ws=at(11) + 16), WORKSPACE),
    (dict(out=at(0)), INVALID),                       # over x
    (dict(out=at(2) + 8 * 256 * 128 - 256), INVALID),  # over the last bytes of w1
    (dict(out=at(7)), INVALID),                       # over z2
    (dict(ws=at(5)), INVALID),                        # over w2
    (dict(ws=at(8)), INVALID),                        # over out
    (dict(ids=at(8) + 16), INVALID),                  # within out
    (dict(weights=at(11) + 4), INVALID),              # within the workspace
    (dict(weights=at(9) + 20), INVALID),              # within ids
] + [(dict([(n, at(2) + 4)]), INVALID) for n in ("w1", "s1", "z1", "w2", "s2", "z2")] \
  + [(dict([(n, None)]), INVALID) for n in ("w1", "s1", "w2", "s2")]


@pytest.mark.parametrize("kw,status", MOE_BAD + [
    (dict(kind=7), INVALID),
    (dict(logits=None), INVALID),
    (dict(ldl=7), INVALID),
    (dict(ids=at(1)), INVALID),      # over the logits
    (dict(weights=at(0)), INVALID),  # over x
])
def test_moe_refuses(kw, status):
    assert moe(**kw) == status
    assert b"ck_moe_w4a16" in lib.ck_last_error_msg()


@pytest.mark.parametrize("kw,status", MOE_BAD)
def test_moe_experts_refuses(kw, status):
    assert moe_experts(**kw) == status
    assert b"ck_moe_experts_w4a16" in lib.ck_last_error_msg()


def test_moe_without_tokens():
    assert moe(T=0, x=None, logits=None, out=None, ids=None, weights=None, ws=None, ws_bytes=0) == ck.CK_OK
    assert moe_experts(T=0, x=None, out=None, ids=None, weights=None, ws=None, ws_bytes=0) == ck.CK_OK


def test_moe_workspace_sizes():
    size = lib.ck_moe_workspace_bytes
    for bad in ((0, 64, 8, 2), (-3, 64, 8, 2), (4, 0, 8, 2), (4, 64, 0, 2), (4, 64, 1025, 2), (4, 64, 8, 0),
                (4, 64, 8, 33), (4, 32832, 8, 2), (2 ** 22, 64, 8, 2)):
        assert size(*bad) == 0
    for T, I, E, k in ((1, 64, 8, 1), (7, 1280, 128, 8), (128, 1280, 128, 8), (3, 32768, 1024, 32)):
        assert size(T, I, E, k) >= T * k * (I * 4 + 8192 * 4) and size(T, I, E, k) % 256 == 0
    # No more room from the tokens of one full pass on.
    assert size(128, 1280, 128, 8) == size(129, 1280, 128, 8) == size(2 ** 22 - 1, 1280, 128, 8)


LSPACE = lib.ck_lora_workspace_bytes(5, 256, 16, 3)


def lora(x=at(0), M=5, K=256, ldx=256, index=at(1), L=3, R=16, a=at(2), b=at(3), scaling=at(4), ranks=at(5), N=96,
         base=at(6), ldb=96, out=at(7), ldo=96, ws=at(8), ws_bytes=LSPACE):
    return lib.ck_lora_add(x, M, K, ldx, index, L, R, a, b, scaling, ranks, N, base, ldb, out, ldo, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID),
    (dict(M=2 ** 22), UNSUPPORTED),
    (dict(K=0), INVALID),
    (dict(K=96, ldx=96), INVALID),
    (dict(K=32832, ldx=32832), UNSUPPORTED),
    (dict(L=0), INVALID),
    (dict(L=2 ** 22), UNSUPPORTED),
    (dict(R=0), INVALID),
    (dict(R=12), INVALID),
    (dict(R=264), UNSUPPORTED),
    (dict(N=0), INVALID),
    (dict(N=40, ldb=40, ldo=40), UNSUPPORTED),
    (dict(N=2 ** 22, ldb=2 ** 22, ldo=2 ** 22), UNSUPPORTED),
    (dict(M=2 ** 21, N=2 ** 20, ldb=2 ** 20, ldo=2 ** 20), UNSUPPORTED),  # one launch
    (dict(a=None), INVALID),
    (dict(a=at(2) + 8), INVALID),
    (dict(b=None), INVALID),
    (dict(b=at(3) + 2), INVALID),
    (dict(scaling=at(4) + 2), INVALID),
    (dict(ranks=at(5) + 1), INVALID),
    (dict(x=None), INVALID),
    (dict(x=at(0) + 2), INVALID),
    (dict(ldx=248), INVALID),
    (dict(ldx=260), INVALID),
    (dict(index=None), INVALID),
    (dict(index=at(1) + 2), INVALID),
    (dict(out=None), INVALID),
    (dict(ldo=100), INVALID),
    (dict(ldo=88), INVALID),
    (dict(base=at(6) + 8), INVALID),
    (dict(ldb=88), INVALID),
    (dict(ldb=100), INVALID),
    (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=LSPACE - 1), WORKSPACE),
    (dict(ws=at(8) + 128), WORKSPACE),
    (dict(out=at(0)), INVALID),                      # over x
    (dict(out=at(1)), INVALID),                      # over the indices
    (dict(out=at(2)), INVALID),                      # over a
    (dict(out=at(3) + 3 * 96 * 16 * 2 - 16), INVALID),  # over the last bytes of b
    (dict(out=at(4)), INVALID),                      # over the scalings
    (dict(out=at(6) + 96 * 2), INVALID),             # base, a row on
    (dict(base=at(7), ldb=104), INVALID),            # base is out, with another stride
    (dict(ws=at(7)), INVALID),
    (dict(ws=at(6)), INVALID),
    (dict(ws=at(2)), INVALID),
])
def test_lora_refuses(kw, status):
    assert lora(**kw) == status
    assert b"ck_lora_add" in lib.ck_last_error_msg()


def test_lora_without_rows():
    assert lora(M=0, x=None, index=None, base=None, out=None, ws=None, ws_bytes=0) == ck.CK_OK


def test_lora_workspace_sizes():
    size = lib.ck_lora_workspace_bytes
    for bad in ((0, 64, 8, 1), (2 ** 22, 64, 8, 1), (4, 0, 8, 1), (4, 32832, 8, 1), (4, 64, 0, 1), (4, 64, 264, 1),
                (4, 64, 8, 0)):
        assert size(*bad) == 0
    for M, K, R, L in ((1, 64, 8, 1), (1, 3840, 16, 300), (301, 10240, 40, 7), (1024, 3840, 256, 2),
                       (1025, 3840, 256, 2), (8192, 3840, 64, 8)):
        parts, rest = divmod(size(M, K, R, L), M * R * 4)
        assert 1 <= parts <= 8 and rest < 256 and size(M, K, R, L) % 256 == 0


def test_new_kernels_are_in_the_resource_report():
    """(That no kernel of the report spills is checked with the other kernels'.)"""
    report = os.path.join(ROOT, "packed_int4_convrot_amd", "_build", "resource_usage.json")
    if not os.path.exists(report):
        pytest.skip("library not built")
    with open(report) as f:
        names = " ".join(k["kernel"] for k in json.load(f)["kernels"])
    for kernel in ("moe_route_kernel", "moe_up_few_kernel", "moe_up_kernel", "moe_down_few_kernel", "moe_down_kernel",
                   "moe_combine_kernel", "lora_shrink_few_kernel", "lora_shrink_many_kernel", "lora_expand_kernel"):
        assert kernel in names, kernel


@pytest.mark.skipif(not shutil.which("g++"), reason="host compiler g++ not found")
def test_rows_abi_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "rows_driver")
    flags = ["-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined,float-cast-overflow",
             "-fno-sanitize-recover=all", "-Wall", "-Wextra", "-Werror"]
    sources = [os.path.join(SAN, "rows_driver.cpp"), os.path.join(SAN, "stub_launch.cpp"),
               os.path.join(CSRC, "ck_api.cpp"), os.path.join(CSRC, "ck_rows_api.cpp")]
    r = subprocess.run(["g++", "-std=c++17", *flags, *sources, "-o", exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and "0 failures" in r.stdout, r.stdout + r.stderr
    assert "runtime error" not in r.stderr
