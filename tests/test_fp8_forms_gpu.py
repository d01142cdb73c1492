"""Every form of the 8-bit float product kernels that a call can come to, against fp64 (fp8_bounds):
shapes beside those of test_fp8_gpu, whose lists test_fp8_forms holds against the rules on sizes."""
import pytest
import torch

import fp8_bounds as ref
from fp8_bounds import random_rows, random_weight, refused
from test_fp8_gpu import DEV, NAN, block, ck, padded, same

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# M, K, N: bf16 rows with each number of weight tiles a pass; 256 x 256 tiles with one run of scales
LINEARS = [(1, 3840, 10240), (2, 1040, 6160), (4, 2064, 14352), (3, 1168, 17696), (5, 400, 22544), (195, 16, 33984),
           (450, 272, 33984),
           # K split in parts of more than a run of scales, on 128 x 128 and on 64 x 64 tiles
           (1604, 16656, 784), (783, 17168, 560)]


@pytest.mark.parametrize("M,K,N", LINEARS)
def test_linear(M, K, N):
    x, _ = padded(random_rows(M, K, M + K + N, DEV), 8, NAN)
    weights = ck.Fp8Weights(*random_weight(N, K, N, DEV))
    bias = torch.randn((N,), device=DEV, generator=torch.Generator(DEV).manual_seed(1)).bfloat16()
    out, room = padded(torch.zeros((M, N), dtype=torch.bfloat16, device=DEV), 16, 3.0)
    print("linear", M, K, N, flush=True)
    ck.fp8_linear(x, weights, bias=bias, out=out)
    want = ref.linear(x.double(), ref.weight(*weights.tensors), bias.double())
    assert refused(out, *want) is None
    assert (room[:, N:] == 3.0).all()
    assert refused(ck.fp8_gemm(*ck.fp8_quant(x), weights, bias=bias), *want) is None
    assert same(out, ck.fp8_linear(x, weights, bias=bias))


# M, H, I: bf16 rows with each number of weight tiles a pass
BLOCKS = [(1, 1040, 6144), (1, 3840, 10240), (2, 1040, 14336), (3, 272, 8320),
          # few rows of codes, in 16-row tiles
          (13, 912, 4224), (13, 1072, 1280), (11, 1952, 4352),
          # fp32 rows between the products, each number of weight tiles of the second
          (5, 4144, 1280), (2, 8208, 1152), (1, 12368, 1280), (3, 24624, 640),
          # large tiles with more than a run of scales
          (4772, 8528, 1664), (4977, 8816, 2432)]


@pytest.mark.parametrize("M,H,I", BLOCKS)
def test_ffn_and_backward(M, H, I):
    x, w1, w2 = block(M, H, I)
    ffn = ck.Fp8Ffn(*w1, *w2)
    kept, room = padded(torch.zeros((M, 2 * I), dtype=torch.bfloat16, device=DEV), 8, 5.0)
    print("ffn", M, H, I, flush=True)
    out = ck.fp8_ffn(x, ffn, gate_up=kept)
    a, b = ref.weight(*w1), ref.weight(*w2)
    want, gate_up = ref.ffn(x.double(), a, b)
    assert refused(kept, *gate_up) is None and (room[:, 2 * I:] == 5.0).all()
    assert refused(out, *want) is None
    assert same(out, ck.fp8_ffn(x, ffn))
    del want, gate_up
    dy = random_rows(M, H, M, DEV)
    dy *= 2.0 ** -10
    back = ffn.transposed()
    dx, room = padded(torch.zeros((M, H), dtype=torch.bfloat16, device=DEV), 16, 7.0)
    print("backward", M, H, I, flush=True)
    ck.fp8_ffn_backward(dy, kept, back, dx=dx)
    assert refused(dx, *ref.backward(dy.double(), kept.double(), a, b)) is None
    assert (room[:, H:] == 7.0).all()
    assert same(dx, ck.fp8_ffn_backward(dy, kept, back))
