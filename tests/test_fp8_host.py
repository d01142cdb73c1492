"""Checks without a GPU of the 8-bit float operators: bad arguments are refused before anything
is enqueued, workspace sizes follow from the sizes alone, the host code runs clean under
AddressSanitizer and UndefinedBehaviorSanitizer, and what the binding hands to the C ABI.

The fake device pointers are never dereferenced: every call here fails validation, has no
rows, or is recorded instead of made.
"""
import gc
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = os.path.join(ROOT, "tests", "sanitize")
CSRC = os.path.join(ROOT, "packed_int4_convrot_amd", "csrc")

ck = pytest.importorskip("packed_int4_convrot_amd")
lib = ck.lib

OK, INVALID, UNSUPPORTED, WORKSPACE = ck.CK_OK, ck.CK_ERR_INVALID_ARG, ck.CK_ERR_UNSUPPORTED, ck.CK_ERR_WORKSPACE
MANY = 2 ** 22


def at(i):
    """The i-th of a row of 256-byte aligned fake addresses, 256 MiB apart."""
    return 0x100000000 + i * 0x10000000


def quant(x=at(0), M=4, K=400, ldx=400, codes=at(1), ldq=400, scales=at(2), lds=4):
    return lib.ck_fp8_quant(x, M, K, ldx, codes, ldq, scales, lds, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(M=MANY), UNSUPPORTED),
    (dict(K=0), INVALID), (dict(K=-16), INVALID), (dict(K=392), INVALID), (dict(K=32784, ldx=32784), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(x=at(0) + 8), INVALID), (dict(ldx=392), INVALID), (dict(ldx=404), INVALID),
    (dict(codes=None), INVALID), (dict(codes=at(1) + 8), INVALID), (dict(ldq=384), INVALID), (dict(ldq=408), INVALID),
    (dict(ldq=2 ** 23 + 16), UNSUPPORTED),
    (dict(scales=None), INVALID), (dict(scales=at(2) + 2), INVALID), (dict(lds=0), INVALID), (dict(lds=6), INVALID),
    (dict(lds=2 ** 23 + 4), UNSUPPORTED),
    (dict(codes=at(0) + 3 * 800), INVALID),    # the last row of x
    (dict(scales=at(0) + 796), INVALID),
    (dict(scales=at(1) + 3 * 400 + 396), INVALID),
])
def test_quant_refuses(kw, status):
    assert quant(**kw) == status
    assert b"ck_fp8_quant" in lib.ck_last_error_msg()


def weights(w=at(0), N=48, K=272, ldi=272, codes=at(1), ldw=272, scales=at(2)):
    return lib.ck_fp8_quantize_weights(w, N, K, ldi, codes, ldw, scales, None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=0), INVALID), (dict(N=40), UNSUPPORTED), (dict(N=MANY), UNSUPPORTED),
    (dict(K=0), INVALID), (dict(K=264), INVALID), (dict(K=32784), UNSUPPORTED),
    (dict(w=None), INVALID), (dict(w=at(0) + 4), INVALID), (dict(ldi=264), INVALID), (dict(ldi=276), INVALID),
    (dict(codes=None), INVALID), (dict(codes=at(1) + 4), INVALID), (dict(ldw=256), INVALID), (dict(ldw=280), INVALID),
    (dict(scales=None), INVALID),
    (dict(codes=at(0)), INVALID), (dict(scales=at(0) + 47 * 544 + 543), INVALID), (dict(scales=at(1) + 1), INVALID),
])
def test_quantize_weights_refuses(kw, status):
    assert weights(**kw) == status
    assert b"ck_fp8_quantize_weights" in lib.ck_last_error_msg()


def transpose(codes=at(0), ldw=272, scales=at(1), N=48, K=272, codes_t=at(2), ldt=48, scales_t=at(3)):
    return lib.ck_fp8_transpose_weights(codes, ldw, scales, N, K, codes_t, ldt, scales_t, None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=0), INVALID), (dict(N=40), UNSUPPORTED), (dict(K=-16), INVALID), (dict(K=264), UNSUPPORTED),
    (dict(N=MANY), UNSUPPORTED), (dict(K=MANY), UNSUPPORTED),
    (dict(codes=None), INVALID), (dict(ldw=256), INVALID), (dict(scales=None), INVALID),
    (dict(codes_t=None), INVALID), (dict(codes_t=at(2) + 4), INVALID), (dict(ldt=32), INVALID), (dict(ldt=56), INVALID),
    (dict(scales_t=None), INVALID), (dict(codes_t=at(0)), INVALID), (dict(scales_t=at(1) + 2), INVALID),
    (dict(scales_t=at(2) + 5), INVALID),
])
def test_transpose_refuses(kw, status):
    assert transpose(**kw) == status
    assert b"ck_fp8_transpose_weights" in lib.ck_last_error_msg()


def gemm(codes=at(0), ldq=400, scales=at(1), lds=4, M=4, K=400, w=at(2), ldw=400, sw=at(3), N=144, bias=at(4),
         out=at(5), ldo=144):
    return lib.ck_fp8_gemm(codes, ldq, scales, lds, M, K, w, ldw, sw, N, bias, out, ldo, None)


LINEAR = lib.ck_fp8_linear_workspace_bytes(4, 400, 144)


def linear(x=at(0), ldx=400, M=4, K=400, w=at(2), ldw=400, sw=at(3), N=144, bias=at(4), out=at(5), ldo=144, ws=at(6),
           ws_bytes=LINEAR):
    return lib.ck_fp8_linear(x, M, K, ldx, w, ldw, sw, N, bias, out, ldo, ws, ws_bytes, None)


BOTH = [
    (dict(M=-1), INVALID), (dict(M=MANY), UNSUPPORTED), (dict(K=0), INVALID), (dict(K=408), INVALID),
    (dict(K=32784, ldw=32784), UNSUPPORTED), (dict(N=0), INVALID), (dict(N=136), UNSUPPORTED), (dict(N=MANY), UNSUPPORTED),
    (dict(M=MANY - 1, N=MANY - 16, ldo=MANY - 16), UNSUPPORTED),
    (dict(w=None), INVALID), (dict(w=at(2) + 8), INVALID), (dict(ldw=384), INVALID), (dict(ldw=408), INVALID),
    (dict(ldw=2 ** 23 + 16), UNSUPPORTED), (dict(sw=None), INVALID), (dict(bias=at(4) + 1), INVALID),
    (dict(out=None), INVALID), (dict(out=at(5) + 8), INVALID), (dict(ldo=136), INVALID), (dict(ldo=148), INVALID),
    (dict(out=at(0)), INVALID), (dict(out=at(2) + 143 * 400 + 384), INVALID), (dict(out=at(4) + 272), INVALID),
    (dict(sw=at(5) + 3 * 288 + 287), INVALID),
]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(codes=None), INVALID), (dict(codes=at(0) + 4), INVALID), (dict(ldq=384), INVALID), (dict(ldq=404), INVALID),
    (dict(scales=None), INVALID), (dict(scales=at(1) + 1), INVALID), (dict(lds=3), INVALID), (dict(lds=0), INVALID),
    (dict(out=at(1)), INVALID),
])
def test_gemm_refuses(kw, status):
    assert gemm(**kw) == status
    assert b"ck_fp8_gemm" in lib.ck_last_error_msg()


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(x=None), INVALID), (dict(x=at(0) + 8), INVALID), (dict(ldx=392), INVALID), (dict(ldx=404), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=LINEAR - 1), WORKSPACE), (dict(ws=at(6) + 128), WORKSPACE),
    (dict(ws=at(0)), INVALID), (dict(ws=at(2)), INVALID), (dict(ws=at(5)), INVALID),
])
def test_linear_refuses(kw, status):
    assert linear(**kw) == status
    assert b"ck_fp8_linear" in lib.ck_last_error_msg()


FFN, BACK = (f(3, 144, 256) for f in (lib.ck_fp8_ffn_workspace_bytes, lib.ck_fp8_ffn_backward_workspace_bytes))


def ffn(x=at(0), M=3, H=144, ldx=144, I=256, w1=at(1), s1=at(2), w2=at(3), s2=at(4), out=at(5), ldo=144, gu=at(6),
        ldg=512, ws=at(7), ws_bytes=FFN):
    return lib.ck_fp8_ffn(x, M, H, ldx, I, w1, s1, w2, s2, out, ldo, gu, ldg, ws, ws_bytes, None)


def backward(x=at(0), M=3, H=144, ldx=144, I=256, w1=at(1), s1=at(2), w2=at(3), s2=at(4), out=at(5), ldo=144, gu=at(6),
             ldg=512, ws=at(7), ws_bytes=BACK):
    return lib.ck_fp8_ffn_backward(x, M, H, ldx, gu, ldg, I, w1, s1, w2, s2, out, ldo, ws, ws_bytes, None)


BLOCK = [
    (dict(M=-1), INVALID), (dict(M=MANY), UNSUPPORTED), (dict(H=0), INVALID), (dict(H=136, ldx=136), INVALID),
    (dict(H=32784, ldx=32784, ldo=32784), UNSUPPORTED), (dict(I=0), INVALID), (dict(I=192), INVALID),
    (dict(I=32896, ldg=65792), UNSUPPORTED), (dict(M=MANY - 1, I=32768, ldg=65536, H=32768, ldx=32768, ldo=32768), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(x=at(0) + 2), INVALID), (dict(ldx=136), INVALID), (dict(ldx=148), INVALID),
    (dict(w1=None), INVALID), (dict(w1=at(1) + 8), INVALID), (dict(s1=None), INVALID), (dict(w2=None), INVALID),
    (dict(w2=at(3) + 8), INVALID), (dict(s2=None), INVALID),
    (dict(out=None), INVALID), (dict(out=at(5) + 2), INVALID), (dict(ldo=136), INVALID), (dict(ldo=148), INVALID),
    (dict(gu=at(6) + 8), INVALID), (dict(ldg=504), INVALID), (dict(ldg=516), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=FFN - 1), WORKSPACE), (dict(ws=at(7) + 64), WORKSPACE),
    (dict(out=at(0)), INVALID), (dict(out=at(1) + 512 * 144 - 16), INVALID), (dict(out=at(3)), INVALID),
    (dict(out=at(4)), INVALID), (dict(out=at(6)), INVALID), (dict(ws=at(1)), INVALID), (dict(ws=at(5)), INVALID),
    (dict(ws=at(6)), INVALID),
]


@pytest.mark.parametrize("kw,status", BLOCK + [(dict(gu=at(0)), INVALID), (dict(gu=at(3)), INVALID)])
def test_ffn_refuses(kw, status):
    assert ffn(**kw) == status
    assert b"ck_fp8_ffn:" in lib.ck_last_error_msg()


@pytest.mark.parametrize("kw,status", BLOCK + [(dict(gu=None), INVALID)])
def test_backward_refuses(kw, status):
    assert backward(**kw) == status
    assert b"ck_fp8_ffn_backward" in lib.ck_last_error_msg()


def test_without_rows():
    assert quant(M=0, x=None, codes=None, scales=None) == OK
    assert gemm(M=0, codes=None, scales=None, out=None) == OK
    assert linear(M=0, x=None, out=None, ws=None, ws_bytes=0) == OK
    assert ffn(M=0, x=None, out=None, gu=None, ws=None, ws_bytes=0) == OK
    assert backward(M=0, x=None, out=None, gu=None, ws=None, ws_bytes=0) == OK


SIZES = (lib.ck_fp8_linear_workspace_bytes, lib.ck_fp8_ffn_workspace_bytes, lib.ck_fp8_ffn_backward_workspace_bytes)


@pytest.mark.parametrize("size", SIZES)
def test_workspaces_serve_every_smaller_call(size):
    rows, H, I = [*range(1, 300), 1000, 4095, 8192, MANY - 1], (16, 144, 3840, 32768), (128, 1280, 32768)
    for h in H:
        for i in I:
            sizes = [size(m, h, i) for m in rows]
            assert all(0 < a <= b for a, b in zip(sizes, sizes[1:]))
    for m in (1, 64, 65, 8192):
        assert all(size(m, a, i) <= size(m, b, i) for a, b in zip(H, H[1:]) for i in I)
        assert all(size(m, h, a) <= size(m, h, b) for a, b in zip(I, I[1:]) for h in H)


@pytest.mark.parametrize("bad", [(0, 64, 128), (-1, 64, 128), (MANY, 64, 128), (4, 0, 128), (4, 72, 128), (4, 32784, 128),
                                 (4, 64, 0), (4, 64, 72)])
def test_workspaces_are_zero_for_refused_sizes(bad):
    assert [size(*bad) for size in SIZES] == [0, 0, 0]
    assert SIZES[1](4, 64, 192) == SIZES[2](4, 64, 192) == SIZES[1](4, 64, 32896) == 0


@pytest.mark.skipif(not shutil.which("g++"), reason="host compiler g++ not found")
def test_abi_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "fp8_driver")
    flags = ["-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined,float-cast-overflow",
             "-fno-sanitize-recover=all", "-Wall", "-Wextra", "-Werror"]
    sources = [os.path.join(SAN, "fp8_driver.cpp"), os.path.join(SAN, "stub_launch.cpp"),
               os.path.join(CSRC, "ck_api.cpp"), os.path.join(CSRC, "ck_fp8_api.cpp")]
    r = subprocess.run(["g++", "-std=c++17", *flags, *sources, "-o", exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and " 0 failures" in r.stdout, r.stdout + r.stderr
    assert "runtime error" not in r.stderr


# ---------------------------------------------------------------- the binding

@pytest.fixture
def calls(monkeypatch):
    """Arguments of the entry points' calls, which enqueue nothing; CPU tensors are taken."""
    seen = []

    def dense(t, name, dtype, shape):
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(name)
        return t

    def matrix(t, name, dtypes):
        if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype not in dtypes:
            raise ValueError(name)
        return t

    def record(*args):
        seen.append(args)
        return ck.CK_OK
    monkeypatch.setattr(ck, "_dense", dense)
    monkeypatch.setattr(ck, "_matrix", matrix)
    monkeypatch.setattr(ck, "_stream", lambda t: 0)
    for name in ("ck_fp8_gemm", "ck_fp8_linear", "ck_fp8_ffn", "ck_fp8_ffn_backward"):
        monkeypatch.setattr(ck.lib, name, record)
    return seen


def tensor(shape, dtype):
    return torch.zeros(shape, dtype=torch.uint8).view(dtype) if dtype.itemsize == 1 else torch.zeros(shape, dtype=dtype)


def linear_tensors():
    return [tensor((48, 144), ck.E4M3), tensor((1, 2), ck.E8M0)]


def ffn_tensors():
    return [tensor((512, 144), ck.E4M3), tensor((4, 2), ck.E8M0), tensor((144, 256), ck.E4M3), tensor((2, 2), ck.E8M0)]


def back_tensors():
    return [tensor((144, 512), ck.E4M3), tensor((2, 4), ck.E8M0), tensor((256, 144), ck.E4M3), tensor((2, 2), ck.E8M0)]


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


HANDLES = [(ck.Fp8Weights, linear_tensors, lambda h: ck.fp8_linear(bf(3, 144), h), (4, 6)),
           (ck.Fp8Ffn, ffn_tensors, lambda h: ck.fp8_ffn(bf(3, 144), h), (5, 6, 7, 8)),
           (ck.Fp8FfnTransposed, back_tensors, lambda h: ck.fp8_ffn_backward(bf(3, 144), bf(3, 512), h), (7, 8, 9, 10))]


@pytest.mark.parametrize("kind,tensors,call,where", HANDLES)
def test_a_handle_holds_the_memory_whose_address_it_passes(calls, kind, tensors, call, where):
    mine = tensors()
    held = [t.untyped_storage()._weak_ref() for t in mine]
    handle = kind(*mine)
    addresses = [t.data_ptr() for t in mine]
    call(handle)
    assert [calls[-1][i] for i in where] == addresses
    for t in mine:
        t.data = torch.zeros((4,), dtype=t.dtype)
    del mine, t
    gc.collect()
    assert not any(torch.UntypedStorage._expired(w) for w in held)
    call(handle)
    assert [calls[-1][i] for i in where] == addresses
    for w in held:
        torch.UntypedStorage._free_weak_ref(w)


@pytest.mark.parametrize("kind,tensors,call,where", HANDLES)
def test_a_handle_whose_storage_was_given_up_is_refused(calls, kind, tensors, call, where):
    for i in range(len(tensors())):
        mine = tensors()
        handle = kind(*mine)
        mine[i].untyped_storage().resize_(0)
        with pytest.raises(ValueError):
            call(handle)
    assert not calls


@pytest.mark.parametrize("kind,tensors,call,where", HANDLES)
def test_handles_of_other_shapes_and_types_are_refused(calls, kind, tensors, call, where):
    for i, t in enumerate(tensors()):
        for wrong in (None, t.view(torch.uint8), t[:-1], t[:, :-1], t[0]):
            mine = tensors()
            mine[i] = wrong
            with pytest.raises((ValueError, AttributeError) if wrong is None else ValueError):
                kind(*mine)


def test_what_does_not_fit_a_handle_is_refused(calls):
    w, f, b = ck.Fp8Weights(*linear_tensors()), ck.Fp8Ffn(*ffn_tensors()), ck.Fp8FfnTransposed(*back_tensors())
    codes, scales = ck.fp8_empty(3, 144, "cpu")
    space = torch.zeros((1 << 16,), dtype=torch.uint8)
    good = [lambda: ck.fp8_gemm(codes, scales, w), lambda: ck.fp8_linear(bf(3, 144), w, bias=bf(48), workspace=space),
            lambda: ck.fp8_ffn(bf(3, 144), f, gate_up=bf(3, 512)), lambda: ck.fp8_ffn_backward(bf(3, 144), bf(3, 512), b)]
    for call in good:
        call()
    assert len(calls) == len(good)
    for bad in (None, 3.0, bf(3, 128), bf(144), bf(1, 3, 144), torch.zeros((3, 144)), bf(144, 3).t(), bf(1, 144).expand(3, 144)):
        for call in (lambda: ck.fp8_linear(bad, w), lambda: ck.fp8_ffn(bad, f), lambda: ck.fp8_ffn_backward(bad, bf(3, 512), b),
                     lambda: ck.fp8_ffn_backward(bf(3, 144), bad, b), lambda: ck.fp8_gemm(bad, scales, w),
                     lambda: ck.fp8_gemm(codes, bad, w)):
            with pytest.raises(ValueError):
                call()
        if bad is not None:
            for call in (lambda: ck.fp8_linear(bf(3, 144), w, bias=bad), lambda: ck.fp8_linear(bf(3, 144), w, out=bad),
                         lambda: ck.fp8_linear(bf(3, 144), w, workspace=bad), lambda: ck.fp8_ffn(bf(3, 144), f, gate_up=bad),
                         lambda: ck.fp8_ffn_backward(bf(3, 144), bf(3, 512), b, dx=bf(3, 143))):
                with pytest.raises(ValueError):
                    call()
    assert len(calls) == len(good)


def test_scale_rows_need_room_up_to_a_multiple_of_four(calls):
    w = ck.Fp8Weights(*linear_tensors())
    codes, scales = ck.fp8_empty(3, 144, "cpu")
    assert scales.shape == (3, 2) and scales.stride() == (4, 1)
    ck.fp8_gemm(codes, scales, w)
    assert calls[-1][3] == 4
    ck.fp8_gemm(codes[:1], scales[:1], w)
    assert calls[-1][3] == 4
    with pytest.raises(ValueError):
        ck.fp8_gemm(codes[:1], tensor((1, 2), ck.E8M0), w)   # ends within the dword that is read
    assert len(calls) == 2
