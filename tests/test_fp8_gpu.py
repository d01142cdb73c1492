"""The 8-bit float operators on the GPU against their definitions in fp64 (fp8_bounds)."""
import pytest
import torch

import fp8_bounds as ref
from fp8_bounds import random_rows, random_weight, refused

pytestmark = pytest.mark.gpu

ck = pytest.importorskip("packed_int4_convrot_amd")

DEV = torch.device("cuda:0")
NAN = float("nan")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(a, b):
    return torch.equal(bits(a), bits(b))


def padded(t, pad, fill):
    """The same values inside rows that are `pad` elements longer."""
    room = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    room[:, :t.shape[1]] = t
    return room[:, :t.shape[1]], room


# ------------------------------------------------------------------ quantisers

@pytest.mark.parametrize("M,K", [(1, 16), (3, 128), (5, 144), (2, 3840), (7, 2112), (33, 1024), (2, 32768), (300, 1040)])
def test_quant(M, K):
    x, _ = padded(random_rows(M, K, M + K, DEV), 8, NAN)
    print("quant", M, K, flush=True)
    codes, scales = ck.fp8_quant(x)
    want, s = ref.quant(x.double())
    assert torch.equal(scales.double(), s)
    assert torch.equal(codes.double(), want)


def test_quant_of_every_bf16():
    """Each finite bf16 beside a largest value of each exponent: every rounding and every scale."""
    every = torch.arange(-32768, 32768, dtype=torch.int32, device=DEV).to(torch.int16).view(torch.bfloat16)
    every = every[every.isfinite()]
    x = every[:every.numel() // 128 * 128].view(-1, 128)
    tops = torch.arange(0, 255, device=DEV, dtype=torch.int32)
    for low in (0, 0x5f, 0x60, 0x61, 0x7f):   # mantissas around 1.75
        top = ((tops << 7) | low).to(torch.int16).view(torch.bfloat16)
        for part in top.split(16):
            y = torch.where(x.abs() <= part[:, None, None].abs(), x, torch.zeros_like(x)).contiguous()
            y[:, :, 5] = part[:, None]
            y = y.view(-1, 128)
            codes, scales = ck.fp8_quant(y)
            want, s = ref.quant(y.double())
            assert torch.equal(scales.double(), s)
            assert torch.equal(codes.double(), want)


def test_quant_leaves_what_is_not_its_own():
    M, K = 5, 272
    x = random_rows(M, K, 1, DEV)
    codes, room = padded(torch.zeros((M, K), dtype=torch.uint8, device=DEV), 32, 77)
    scales, sroom = padded(torch.zeros((M, 3), dtype=torch.uint8, device=DEV), 5, 99)
    ck.fp8_quant(x, codes.view(ck.E4M3), scales.view(ck.E8M0))
    assert (room[:, K:] == 77).all() and (sroom[:, 3:] == 99).all()
    want, s = ref.quant(x.double())
    assert torch.equal(codes.view(ck.E4M3).double(), want) and torch.equal(scales.view(ck.E8M0).double(), s)


@pytest.mark.parametrize("bad", [NAN, float("inf"), -float("inf")])
def test_not_finite_reaches_only_its_own_row(bad):
    M, K, N = 37, 400, 160
    x = random_rows(M, K, 2, DEV)
    x[3, 200] = bad
    weights = ck.Fp8Weights(*random_weight(N, K, 3, DEV))
    out = ck.fp8_linear(x, weights)
    assert out[3].isnan().all()
    x[3] = 0
    clean = ck.fp8_linear(x, weights)
    keep = torch.arange(M, device=DEV) != 3
    assert clean.isfinite().all() and same(out[keep], clean[keep])


@pytest.mark.parametrize("N,K", [(16, 16), (128, 128), (144, 272), (400, 1040), (1040, 2112)])
def test_weights(N, K):
    w, _ = padded(random_rows(N, K, N, DEV), 24, NAN)
    codes, scales = ck.fp8_quantize_weights(w)
    rows, cols = ref.blocks(N), ref.blocks(K)
    y = torch.nn.functional.pad(w.double(), (0, cols * 128 - K, 0, rows * 128 - N))
    s = ref.scale_of(y.view(rows, 128, cols, 128).abs().amax(dim=(1, 3)))
    assert torch.equal(scales.double(), s)
    spread = s.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    assert torch.equal(codes.double(), ref.e4m3(w.double() / spread))
    t = ck.Fp8Weights(codes, scales).transposed()
    assert same(t.tensors[0], codes.view(torch.uint8).t().contiguous()) and same(t.tensors[1], scales.view(torch.uint8).t().contiguous())


# --------------------------------------------------------------------- linear

# M, K, N: lengths from one row, K inside a block and around 64 blocks (a run of scales), N inside
# a tile, a block of weights or a 16-row tile of them.
LINEARS = [(1, 16, 16), (1, 3840, 512), (2, 144, 48), (5, 128, 1040), (8, 1024, 128), (13, 2112, 272), (16, 512, 400),
           (17, 272, 528), (32, 3840, 256), (33, 400, 144), (64, 1040, 112), (65, 640, 384), (100, 8192, 144),
           (129, 8320, 272), (130, 8208, 16), (200, 8448, 32), (257, 256, 1040), (300, 2112, 1040), (513, 1168, 784),
           (1000, 384, 272), (3, 32768, 64), (70, 32768, 80)]


@pytest.mark.parametrize("M,K,N", LINEARS)
def test_linear(M, K, N):
    x, _ = padded(random_rows(M, K, M + K + N, DEV), 16, NAN)
    wc, ws = random_weight(N, K, N, DEV)
    wc, _ = padded(wc.view(torch.uint8), 48, 0x7f)
    weights = ck.Fp8Weights(wc.view(ck.E4M3), ws)
    bias = torch.randn((N,), device=DEV, generator=torch.Generator(DEV).manual_seed(1)).bfloat16() if M % 2 else None
    out, room = padded(torch.zeros((M, N), dtype=torch.bfloat16, device=DEV), 8, 3.0)
    print("linear", M, K, N, flush=True)
    ck.fp8_linear(x, weights, bias=bias, out=out)
    want = ref.linear(x.double(), ref.weight(wc.view(ck.E4M3), ws), None if bias is None else bias.double())
    assert refused(out, *want) is None
    assert (room[:, N:] == 3.0).all()
    # the same from codes, twice
    codes, scales = ck.fp8_quant(x)
    again = ck.fp8_gemm(codes, scales, weights, bias=bias)
    assert refused(again, *want) is None
    assert same(again, ck.fp8_gemm(codes, scales, weights, bias=bias))


def test_rows_do_not_depend_on_their_neighbours():
    """A row's result is the same bits wherever it stands among as many rows."""
    M, K, N = 300, 1040, 400
    x = random_rows(M, K, 5, DEV)
    weights = ck.Fp8Weights(*random_weight(N, K, 6, DEV))
    order = torch.randperm(M, device=DEV)
    assert same(ck.fp8_linear(x, weights)[order], ck.fp8_linear(x[order].contiguous(), weights))


def test_without_rows():
    weights = ck.Fp8Weights(*random_weight(32, 64, 6, DEV))
    assert ck.fp8_linear(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV), weights).shape == (0, 32)


# --------------------------------------------------------- feed-forward block

# M, H, I
BLOCKS = [(1, 16, 128), (1, 3840, 384), (2, 144, 128), (5, 272, 256), (16, 512, 1280), (17, 1040, 384), (37, 2112, 1280),
          (64, 128, 256), (65, 400, 128), (77, 2112, 640), (130, 256, 384), (257, 1040, 256), (300, 144, 896),
          (40, 64, 8320), (90, 8320, 128), (600, 640, 512)]


def block(M, H, I):
    x = random_rows(M, H, M + H + I, DEV)
    x *= 0.25
    w1, w2 = random_weight(2 * I, H, H, DEV), random_weight(H, I, I, DEV)
    # gate and up of size one or so, as trained weights give
    w1 = w1[0], (w1[1].float() * 2.0 ** -round(0.5 * (torch.tensor(float(H)).log2().item()))).to(ck.E8M0)
    return x, w1, w2


@pytest.mark.parametrize("M,H,I", BLOCKS)
def test_ffn(M, H, I):
    x, w1, w2 = block(M, H, I)
    ffn = ck.Fp8Ffn(*w1, *w2)
    kept, room = padded(torch.zeros((M, 2 * I), dtype=torch.bfloat16, device=DEV), 16, 5.0)
    print("ffn", M, H, I, flush=True)
    out = ck.fp8_ffn(x, ffn, gate_up=kept)
    want, gate_up = ref.ffn(x.double(), ref.weight(*w1), ref.weight(*w2))
    assert refused(kept, *gate_up) is None
    assert (room[:, 2 * I:] == 5.0).all()
    assert refused(out, *want) is None
    assert same(out, ck.fp8_ffn(x, ffn))


@pytest.mark.parametrize("M,H,I", BLOCKS)
def test_backward(M, H, I):
    x, w1, w2 = block(M, H, I)
    ffn = ck.Fp8Ffn(*w1, *w2).transposed()
    dy = random_rows(M, H, M, DEV)
    dy *= 2.0 ** -10
    g = torch.Generator().manual_seed(M + I)
    gate_up, _ = padded((2 * torch.randn((M, 2 * I), generator=g)).bfloat16().to(DEV), 8, NAN)
    dx, room = padded(torch.zeros((M, H), dtype=torch.bfloat16, device=DEV), 24, 7.0)
    print("backward", M, H, I, flush=True)
    ck.fp8_ffn_backward(dy, gate_up, ffn, dx=dx)
    want = ref.backward(dy.double(), gate_up.double(), ref.weight(*w1), ref.weight(*w2))
    assert refused(dx, *want) is None
    assert (room[:, H:] == 7.0).all()
    assert same(dx, ck.fp8_ffn_backward(dy, gate_up, ffn))
