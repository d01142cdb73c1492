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
           (1000, 384, 272), (3, 32768, 64), (70, 32768, 80),
           # each tile of the tiled product, with one and with two runs of scales
           (500, 272, 3824), (1000, 400, 3824), (2000, 272, 3824), (3000, 144, 3856), (8191, 400, 2064), (4200, 144, 3856),
           (450, 8336, 3600), (900, 8336, 3600), (1800, 8336, 3600), (2800, 8336, 3600), (4100, 8336, 3600),
           # few rows: each number of 16-row tiles of either operand, and passes
           (1, 16400, 4304), (2, 16400, 8256), (16, 3840, 4304), (16, 3840, 11584), (30, 8208, 3600), (20, 4112, 4304), (40, 4112, 3600),
           (33, 4112, 4304), (50, 4112, 3600), (1, 16, 33040), (3, 144, 50064), (2, 48, 24688),
           # K split: 64 and 128 weight rows a tile, two to eight splits, the last ones short, more than a run of scales
           (100, 3856, 1040), (65, 2064, 144), (64, 10240, 272), (130, 5120, 528), (500, 10256, 512), (2000, 20496, 272),
           (9, 18880, 3664), (20, 10944, 11584), (200, 20480, 3600), (60, 32752, 272), (50, 32768, 10752)]


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
          (40, 64, 8320), (90, 8320, 128), (600, 640, 512),
          (700, 144, 2688), (2000, 144, 2688), (2000, 144, 3840), (4200, 144, 3840),   # larger tiles
          (700, 144, 3840), (3000, 144, 3840), (600, 8336, 3840), (1000, 8336, 5120), (2000, 8336, 3840),
          # few rows: each number of 16-row tiles of either operand, and passes
          (17, 1520, 128), (20, 3840, 4224), (49, 2512, 128), (40, 5008, 4224), (50, 6992, 4224), (16, 5008, 11648),
          (20, 8464, 12288), (1, 16400, 8320), (2, 64, 16640), (1, 16, 24704), (1, 32, 32768),
          (100, 272, 10240), (300, 512, 5120),   # the second product's K split
          (100, 48, 32768)]                      # the widest


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


def test_keeping_gate_and_up_in_each_tile():
    """gate_up of 256 x 256 tiles, whose rows and columns end inside one, in wider rows."""
    M, H, I = 2030, 144, 2688
    x, w1, w2 = block(M, H, I)
    kept, room = padded(torch.zeros((M, 2 * I), dtype=torch.bfloat16, device=DEV), 8, 5.0)
    ck.fp8_ffn(x, ck.Fp8Ffn(*w1, *w2), gate_up=kept)
    want, gate_up = ref.ffn(x.double(), ref.weight(*w1), ref.weight(*w2))
    assert refused(kept, *gate_up) is None and (room[:, 2 * I:] == 5.0).all()


@pytest.mark.parametrize("M", [3, 40, 90, 700])
@pytest.mark.parametrize("bad", [NAN, float("inf")])
def test_not_finite_in_a_block_stays_in_its_row(M, bad):
    H, I = 272, 384
    x, w1, w2 = block(M, H, I)
    ffn = ck.Fp8Ffn(*w1, *w2)
    keep = torch.arange(M, device=DEV) != 1
    gate_up = torch.randn((M, 2 * I), device=DEV).bfloat16()

    def both():
        return ck.fp8_ffn(x, ffn), ck.fp8_ffn_backward(x, gate_up, ffn.transposed())
    x[1] = 0
    clean = both()
    x[1, 200] = bad
    sick = both()
    for a, b in zip(clean, sick):
        assert a.isfinite().all() and b[1].isnan().all() and same(a[keep], b[keep])
    x[1, 200] = 0
    gate_up[1, 5] = bad                        # one element of the gate
    dx = ck.fp8_ffn_backward(x, gate_up, ffn.transposed())
    assert same(dx[keep], clean[1][keep])


@pytest.mark.parametrize("M,K,N", [(3, 272, 144), (16, 2112, 272), (100, 272, 144), (100, 4112, 144), (1000, 272, 3600)])
def test_powers_of_two_only_move_the_exponents(M, K, N):
    x, (wc, ws) = random_rows(M, K, 3, DEV), random_weight(N, K, 4, DEV)
    want = ck.fp8_linear(x, ck.Fp8Weights(wc, ws))
    for e in (100, -100):
        moved = ck.Fp8Weights(wc, (ws.view(torch.uint8).int() - e).to(torch.uint8).view(ck.E8M0))
        assert same(ck.fp8_linear((x.double() * 2.0 ** e).bfloat16(), moved), want)


def test_rows_of_zeros_and_largest_values():
    for M in (4, 100, 600):
        H, I = 256, 256
        x, w1, w2 = block(M, H, I)
        ffn = ck.Fp8Ffn(*w1, *w2)
        x[:] = 0
        assert not ck.fp8_ffn(x, ffn).any()
        gate_up = torch.zeros((M, 2 * I), device=DEV, dtype=torch.bfloat16)
        assert not ck.fp8_ffn_backward(x + 1, gate_up, ffn.transposed()).any()
        # the logistic function at its ends: silu(-3e4) = -0, silu(3e4) = 3e4
        gate_up[:, :I], gate_up[:, I:] = -3e4, 2
        assert not ck.fp8_ffn_backward(x + 1, gate_up, ffn.transposed()).any()
        gate_up[:, :I] = 3e4
        want = ref.backward(x.double() + 1, gate_up.double(), ref.weight(*w1), ref.weight(*w2))
        assert refused(ck.fp8_ffn_backward(x + 1, gate_up, ffn.transposed()), *want) is None


@pytest.mark.parametrize("M,H,I", [(24, 256, 256), (200, 144, 384)])
def test_the_gradient_against_differences(M, H, I):
    """Inputs that the quantiser keeps (e4m3 values of one exponent range), so that the block is
    differentiable but for Q(h), which the gradient passes through.  Along the gradient itself
    d = dx: its terms (W1 d)_i dgu_i have one rounding of dgu each, by 2^-4 at most, of either sign
    (8 times the root of their squares' sum), besides dx's rounding to bf16, gate and up's (2^-8
    each, times at most 2 in the factors) and what the matrix core drops, below those."""
    g = torch.Generator().manual_seed(M)
    e4m3 = lambda t: t.clamp(-3.9, 3.9).to(torch.float8_e4m3fn).float()  # noqa: E731
    x = e4m3(torch.randn((M, H), generator=g)).bfloat16().to(DEV)
    dy = e4m3(torch.randn((M, H), generator=g)).bfloat16().to(DEV)
    _, w1, w2 = block(M, H, I)
    codes, scales = ck.fp8_quant(x)
    assert torch.equal(codes.double() * scales.double().repeat_interleave(128, 1)[:, :H], x.double())
    ffn = ck.Fp8Ffn(*w1, *w2)
    kept = torch.empty((M, 2 * I), dtype=torch.bfloat16, device=DEV)
    ck.fp8_ffn(x, ffn, gate_up=kept)
    dx = ck.fp8_ffn_backward(dy, kept, ffn.transposed()).double()
    a, b = ref.weight(*w1), ref.weight(*w2)

    def loss(t):
        gu = t @ a.t()
        return ((gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:] @ b.t()) * dy.double()).sum()
    d = dx / dx.norm()
    h = 1e-5
    measured = float((loss(x.double() + h * d) - loss(x.double() - h * d)) / (2 * h))
    gu = (x.double() @ a.t()).requires_grad_()
    ((gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:] @ b.t()) * dy.double()).sum().backward()
    terms = (d @ a.t()) * gu.grad
    sure = 8 * 2.0 ** -4 * float(terms.square().sum().sqrt())
    small = 2.0 ** -8 * float(dx.norm()) + 8 * 4 * 2.0 ** -8 * float(terms.square().sum().sqrt())
    assert sure + small < 0.2 * measured          # the test would see a factor left out
    assert abs(float((dx * d).sum()) - measured) <= sure + small


def test_the_linears_backward_pass_is_the_transposed_linear():
    M, K, N = 77, 400, 272
    codes, scales = random_weight(N, K, 3, DEV)
    back = ck.Fp8Weights(codes, scales).transposed()
    dy = random_rows(M, N, 4, DEV)
    want = ref.linear(dy.double(), ref.weight(codes, scales).t().contiguous())
    assert refused(ck.fp8_linear(dy, back), *want) is None


# ------------------------------------------------- calls as programs make them

class Step:
    """A training step of what lies beside frozen weights: a projection with adapters, the block,
    and the gradient back to the projection's input.  Buffers are allocated once."""

    def __init__(self, M, H, I, seed):
        self.x = random_rows(M, H, seed, DEV)
        g = torch.Generator().manual_seed(seed)
        full = (torch.randn((H, H), generator=g) * H ** -0.5).bfloat16().to(DEV)
        self.proj = ck.Fp8Weights(*ck.fp8_quantize_weights(full))
        self.back = self.proj.transposed()
        _, w1, w2 = block(M, H, I)
        self.ffn = ck.Fp8Ffn(*w1, *w2)
        self.ffn_back = self.ffn.transposed()
        a = (torch.randn((2, 16, H), generator=g) * H ** -0.5).bfloat16().to(DEV)
        b = (torch.randn((2, H, 16), generator=g) * 0.2).bfloat16().to(DEV)
        self.lora = ck.LoraAdapters(a, b)
        self.index = torch.randint(-1, 2, (M,), generator=g, dtype=torch.int32).to(DEV)
        self.dy = random_rows(M, H, seed + 1, DEV)
        self.y, self.out, self.dx, self.dp = (torch.empty_like(self.x) for _ in range(4))
        self.kept = torch.empty((M, 2 * I), dtype=torch.bfloat16, device=DEV)
        # One workspace serves the calls of a stream one after the other.
        need = max(ck.fp8_linear_workspace_bytes(M, H, H), ck.fp8_ffn_workspace_bytes(M, H, I),
                   ck.fp8_ffn_backward_workspace_bytes(M, H, I), ck.lora_workspace_bytes(M, H, 16, 2))
        self.space = torch.empty((need,), dtype=torch.uint8, device=DEV)

    def run(self):
        ws = self.space
        ck.fp8_linear(self.x, self.proj, out=self.y, workspace=ws)
        ck.lora_add(self.x, self.lora, self.index, base=self.y, out=self.y, workspace=ws)
        ck.fp8_ffn(self.y, self.ffn, out=self.out, gate_up=self.kept, workspace=ws)
        ck.fp8_ffn_backward(self.dy, self.kept, self.ffn_back, dx=self.dx, workspace=ws)
        ck.fp8_linear(self.dx, self.back, out=self.dp, workspace=ws)
        return self.results()

    def results(self):
        return [t.clone() for t in (self.y, self.out, self.kept, self.dx, self.dp)]


@pytest.mark.parametrize("M,H,I", [(1, 448, 384), (20, 448, 384), (64, 448, 384), (130, 448, 384), (1030, 448, 384),
                                   (100, 2112, 4224)])
def test_a_run_together_captured_and_replayed(M, H, I):
    step = Step(M, H, I, M)
    eager = step.run()
    y, out, kept, dx, dp = (t.double() for t in eager)
    w1, s1, w2, s2 = step.ffn.tensors
    want, gate_up = ref.ffn(y, ref.weight(w1, s1), ref.weight(w2, s2))
    assert refused(eager[1], *want) is None and refused(eager[2], *gate_up) is None
    assert refused(eager[3], *ref.backward(step.dy.double(), kept, ref.weight(w1, s1), ref.weight(w2, s2))) is None
    assert refused(eager[4], *ref.linear(dx, ref.weight(*step.proj.tensors).t().contiguous())) is None
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step.run()
    other = step.x.flip(0).contiguous()
    mine = step.x.clone()
    step.x.copy_(other)
    swapped = step.run()
    for x, expected in ((mine, eager), (other, swapped), (mine, eager)):
        step.x.copy_(x)
        for t in (step.y, step.out, step.kept, step.dx, step.dp):
            t.fill_(NAN)
        step.space.fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(step.results(), expected):
            assert same(a, b)
        torch.randn((64, 64), device=DEV) @ torch.randn((64, 64), device=DEV)   # work of another kind in between


def test_two_graphs_and_two_streams():
    """Two steps with workspaces of their own, on two streams at once and as two graphs replayed in turn."""
    steps = [Step(M, 320, 256, M) for M in (30, 200)]
    want = [s.run() for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        for s, stream in zip(steps, streams):
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                s.run()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert all(same(a, b) for a, b in zip(s.results(), w))
    graphs = [torch.cuda.CUDAGraph() for _ in steps]
    for s, graph in zip(steps, graphs):
        with torch.cuda.graph(graph):
            s.run()
    for i in (0, 1, 1, 0):
        for t in (steps[i].out, steps[i].dp):
            t.fill_(NAN)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(steps[i].results(), want[i]))


@pytest.mark.parametrize("M,H,I", [(1, 272, 256), (8, 272, 256), (33, 272, 256), (65, 272, 256), (300, 272, 256),
                                   (20, 272, 8320), (100, 272, 4352), (130, 4112, 256)])
def test_a_workspace_full_of_nan_changes_nothing(M, H, I):
    """And what a call leaves in it is not read by the next."""
    x, w1, w2 = block(M, H, I)
    ffn, weights = ck.Fp8Ffn(*w1, *w2), ck.Fp8Weights(*random_weight(144, H, 5, DEV))
    need = max(ck.fp8_ffn_backward_workspace_bytes(M, H, I), ck.fp8_linear_workspace_bytes(M, H, 144))
    space = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    want = ck.fp8_ffn(x, ffn), ck.fp8_linear(x, weights)
    for _ in range(2):
        assert same(ck.fp8_ffn(x, ffn, workspace=space), want[0])
        assert same(ck.fp8_linear(x, weights, workspace=space), want[1])
        assert same(ck.fp8_linear(x, weights), want[1])
        space.fill_(0xff)


def test_rows_beyond_32_bit_offsets():
    """Codes of more than 4 GiB: the last rows are what they are by themselves."""
    M, K, N, last = 540_000, 8192, 48, 300
    weights = ck.Fp8Weights(*random_weight(N, K, 6, DEV))
    codes, scales = ck.fp8_empty(M, K, DEV)
    assert codes.numel() > 2 ** 32
    x = random_rows(last, K, 7, DEV)
    c, s = ck.fp8_quant(x)
    codes.view(torch.uint8).zero_()
    scales.view(torch.uint8).fill_(127)
    codes.view(torch.uint8)[M - last:] = c.view(torch.uint8)
    scales.view(torch.uint8)[M - last:] = s.view(torch.uint8)
    out = ck.fp8_gemm(codes, scales, weights)
    assert refused(out[M - last:], *ref.linear(x.double(), ref.weight(*weights.tensors))) is None
    assert not out[:M - last].any()
    del codes, scales, out
    wide = torch.zeros((140_000, 32768), dtype=torch.bfloat16, device=DEV)   # bf16 rows of 9 GB
    wide[-5:, :K] = x[-5:]
    c, s = ck.fp8_quant(wide[:, :K])
    want = ck.fp8_quant(x[-5:])
    assert torch.equal(c[-5:].double(), want[0].double()) and torch.equal(s[-5:].double(), want[1].double())
    assert not c.view(torch.uint8)[:-5].any()


def test_weights_beyond_32_bit_offsets():
    """The last rows of a weight of more than 4 GiB, for few rows and for many."""
    N, K = 264_192, 16384
    codes = torch.zeros((N, K), dtype=torch.uint8, device=DEV)
    scales = torch.full((ref.blocks(N), ref.blocks(K)), 127, dtype=torch.uint8, device=DEV)
    assert codes.numel() > 2 ** 32
    c, s = random_weight(256, K, 8, DEV)
    codes[N - 256:], scales[-2:] = c.view(torch.uint8), s.view(torch.uint8)
    big, small = ck.Fp8Weights(codes.view(ck.E4M3), scales.view(ck.E8M0)), ck.Fp8Weights(c, s)
    for M in (2, 20, 100):
        x = random_rows(M, K, M, DEV)
        out = ck.fp8_linear(x, big)
        assert refused(out[:, N - 256:], *ref.linear(x.double(), ref.weight(c, s))) is None
        assert not out[:, :N - 256].any()


def test_bindings_refuse_what_does_not_fit():
    weights = ck.Fp8Weights(*random_weight(48, 144, 9, DEV))
    x = random_rows(3, 144, 1, DEV)
    short = torch.empty((ck.fp8_linear_workspace_bytes(3, 144, 48) - 1,), dtype=torch.uint8, device=DEV)
    with pytest.raises(ck.CKError, match="workspace"):
        ck.fp8_linear(x, weights, workspace=short)
    for call in (lambda: ck.fp8_linear(x.cpu(), weights), lambda: ck.fp8_linear(x, weights, bias=torch.zeros(48, device=DEV)),
                 lambda: ck.fp8_linear(x, weights, out=x), lambda: ck.fp8_quant(x.float()), lambda: ck.fp8_quant(x.cpu()),
                 lambda: ck.fp8_quantize_weights(x.cpu()), lambda: ck.fp8_quant(x[:, :136]),
                 lambda: ck.fp8_linear(x[:, 1:], weights), lambda: ck.Fp8Weights(weights.tensors[0], weights.tensors[1].cpu()),
                 lambda: ck.Fp8Weights(weights.tensors[0].cpu(), weights.tensors[1])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ck.CKError):
        ck.fp8_quantize_weights(x)             # three rows are no multiple of 16
