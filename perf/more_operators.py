"""What is measured of the 8-bit float operators: the quantiser of activations (e4m3, a scale
for each row and 128 columns), the linear on weights with a scale for each 128 x 128 block, the
gated feed-forward block built of two such products, and the block's backward pass to its input
(the weights are frozen).  Scales are powers of two (e8m0), the smallest that keep a block's
values within e4m3's range, 1 for a block of zeros.

`run` computes a case either in plain torch operations in fp32 (`own` false) or through the
library's entry points (`own` true), on the same prepared inputs; the library's result buffers
and workspace are kept from step to step.  `exact` is the definition in fp64, the roundings to
8 bits included.
"""
import math

import torch

own = False

DEV = "cuda:0"
B = 128
TOP = 448.0          # the largest e4m3 value
LEAST = -127         # exponent of the smallest scale


def listed():
    return [
        # The input of a decode step's linears, quantised once for all of them.
        dict(name="quant_batch_5", op="quant", rows=5, K=3840, pad=0),
        # A prompt's hidden activations, rows inside a wider buffer.
        dict(name="quant_prompt", op="quant", rows=8192, K=10240, pad=512),
        # One token: the latency of a decode step's projection.
        dict(name="linear_one_token", op="linear", rows=1, K=3840, N=10240, bias=False, pad=0),
        # An ordinary decode batch, square projection with a bias.
        dict(name="linear_batch_32", op="linear", rows=32, K=3840, N=3840, bias=True, pad=0),
        # Odd everything: rows, a half block of columns, results that end inside a block, padded rows.
        dict(name="linear_odd_301", op="linear", rows=301, K=2112, N=1040, bias=True, pad=40),
        # The largest product: packed prompts.
        dict(name="linear_prompt", op="linear", rows=8192, K=10240, N=3840, bias=False, pad=0),
        # One token through the feed-forward block.
        dict(name="ffn_one_token", op="ffn", rows=1, H=3840, I=10240, keep=False),
        # A decode batch of odd sizes.
        dict(name="ffn_odd_37", op="ffn", rows=37, H=2112, I=1280, keep=False),
        # The forward pass of an adapter's training step: gate and up are kept.
        dict(name="ffn_train_2000", op="ffn", rows=2000, H=2048, I=5120, keep=True),
        # The largest: packed prompts.
        dict(name="ffn_prompt", op="ffn", rows=8192, H=3840, I=10240, keep=False),
        # The backward pass of a short odd sequence, and of a whole batch.
        dict(name="grad_odd_77", op="grad", rows=77, H=2112, I=1280),
        dict(name="grad_batch", op="grad", rows=4096, H=3840, I=10240),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return min(hi, max(lo, int(v) // step * step))


def draw(rng):
    op = rng.choice(("quant", "linear", "linear", "ffn", "ffn", "grad", "grad"))
    rows = _log(rng, 1, 8192)
    if op == "quant":
        return dict(op=op, rows=rows, K=_log(rng, 256, 10240, 16), pad=rng.choice((0, 8, 512)))
    if op == "linear":
        return dict(op=op, rows=rows, K=_log(rng, 256, 10240, 16), N=_log(rng, 256, 10240, 16),
                    bias=rng.random() < 0.5, pad=rng.choice((0, 0, 64)))
    H, I = _log(rng, 256, 3840, 16), _log(rng, 256, 10240, 128)
    if op == "ffn":
        return dict(op=op, rows=rows, H=H, I=I, keep=rng.random() < 0.4)
    return dict(op=op, rows=rows, H=H, I=I)


# ------------------------------------------------------------------ inputs

def _blocks(n):
    return -(-n // B)


def _activations(g, M, K, pad=0):
    """bf16 [M, K] in rows of K + pad: N(0, 1) with a few columns twenty times as large."""
    x = torch.randn((M, K + pad), device=DEV, generator=g)
    x[:, torch.randperm(K, device=DEV, generator=g)[:max(1, K // 256)]] *= 20.0
    return x.to(torch.bfloat16)[:, :K]


def _weight(g, N, K):
    """e4m3 codes [N, K] and e8m0 scales of 128 x 128 blocks of an N(0, 1 / K) weight."""
    w = torch.randn((N, K), device=DEV, generator=g) * K ** -0.5
    padded = torch.nn.functional.pad(w, (0, _blocks(K) * B - K, 0, _blocks(N) * B - N))
    s = torch.exp2(torch.ceil(torch.log2(padded.view(_blocks(N), B, _blocks(K), B).abs().amax(dim=(1, 3)) / TOP)))
    codes = (w / s.repeat_interleave(B, 0)[:N].repeat_interleave(B, 1)[:, :K]).to(torch.float8_e4m3fn)
    return codes, s.to(torch.float8_e8m0fnu)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = dict(case=case)
    M, op = case["rows"], case["op"]
    if op == "quant":
        st["x"] = _activations(g, M, case["K"], case["pad"])
    elif op == "linear":
        st["x"] = _activations(g, M, case["K"], case["pad"])
        st["w"] = _weight(g, case["N"], case["K"])
        st["bias"] = torch.randn((case["N"],), device=DEV, generator=g).to(torch.bfloat16) if case["bias"] else None
    else:
        H, I = case["H"], case["I"]
        st["w1"], st["w2"] = _weight(g, 2 * I, H), _weight(g, H, I)
        if op == "ffn":
            st["x"] = _activations(g, M, H)
        else:
            st["dy"] = (torch.randn((M, H), device=DEV, generator=g) * 1e-3).to(torch.bfloat16)
            st["gate_up"] = torch.randn((M, 2 * I), device=DEV, generator=g).to(torch.bfloat16)
    if own:
        import packed_int4_convrot_amd as ck
        st["ck"] = ck
        space = 1
        if op == "quant":
            st["codes"], st["scales"] = ck.fp8_empty(M, case["K"], DEV)
        elif op == "linear":
            st["weights"] = ck.Fp8Weights(*st["w"])
            st["out"] = torch.empty((M, case["N"]), dtype=torch.bfloat16, device=DEV)
            space = ck.fp8_linear_workspace_bytes(M, case["K"], case["N"])
        else:
            st["ffn"] = ck.Fp8Ffn(*st["w1"], *st["w2"])
            st["out"] = torch.empty((M, H), dtype=torch.bfloat16, device=DEV)
            if op == "ffn":
                st["kept"] = torch.empty((M, 2 * I), dtype=torch.bfloat16, device=DEV) if case["keep"] else None
                space = ck.fp8_ffn_workspace_bytes(M, H, I)
            else:
                st["back"] = st["ffn"].transposed()
                space = ck.fp8_ffn_backward_workspace_bytes(M, H, I)
        st["space"] = torch.empty((max(space, 1),), dtype=torch.uint8, device=DEV)
    return st


# -------------------------------------------------------------- plain forms

def _two_to(e):
    """2^e in fp32 for whole -126 <= e <= 127, exactly (a power function rounds)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _plain_quant(x):
    """Codes [M, K] and scales [M, blocks] of an fp32 matrix."""
    M, K = x.shape
    y = torch.nn.functional.pad(x, (0, _blocks(K) * B - K)).view(M, _blocks(K), B)
    a = y.abs().amax(dim=2)
    m, e = torch.frexp(a)  # a = m 2^e, 1 / 2 <= m < 1; 448 = 7 / 8 * 2^9
    e = torch.where(a > 0, torch.clamp(e - 9 + (m > 0.875), min=LEAST), 0)
    codes = (y * _two_to(-e).unsqueeze(2)).to(torch.float8_e4m3fn).view(M, -1)[:, :K]
    return codes, 0.5 * _two_to(e + 1)


def _plain_values(codes, s):
    """The fp32 values that quantised activations stand for."""
    return codes.float() * s.repeat_interleave(B, dim=1)[:, :codes.shape[1]]


def _plain_weight(codes, s):
    N, K = codes.shape
    return codes.float() * s.float().repeat_interleave(B, 0)[:N].repeat_interleave(B, 1)[:, :K]


def run(state):
    case, op = state["case"], state["case"]["op"]
    if own:
        ck = state["ck"]
        if op == "quant":
            return ck.fp8_quant(state["x"], codes=state["codes"], scales=state["scales"])
        if op == "linear":
            return ck.fp8_linear(state["x"], state["weights"], bias=state["bias"], out=state["out"],
                                 workspace=state["space"])
        if op == "ffn":
            out = ck.fp8_ffn(state["x"], state["ffn"], out=state["out"], gate_up=state["kept"],
                             workspace=state["space"])
            return (out, state["kept"]) if case["keep"] else out
        return ck.fp8_ffn_backward(state["dy"], state["gate_up"], state["back"], dx=state["out"],
                                   workspace=state["space"])
    if op == "quant":
        codes, s = _plain_quant(state["x"].float())
        return codes.contiguous(), s.to(torch.float8_e8m0fnu)
    if op == "linear":
        y = torch.matmul(_plain_values(*_plain_quant(state["x"].float())), _plain_weight(*state["w"]).t())
        return (y if state["bias"] is None else y + state["bias"].float()).to(torch.bfloat16)
    w1, w2, I = _plain_weight(*state["w1"]), _plain_weight(*state["w2"]), case["I"]
    if op == "ffn":
        gu = torch.matmul(_plain_values(*_plain_quant(state["x"].float())), w1.t())
        g, u = gu[:, :I], gu[:, I:]
        h = g / (1.0 + torch.exp(-g)) * u
        out = torch.matmul(_plain_values(*_plain_quant(h)), w2.t()).to(torch.bfloat16)
        return (out, gu.to(torch.bfloat16)) if case["keep"] else out
    g, u = state["gate_up"][:, :I].float(), state["gate_up"][:, I:].float()
    dh = torch.matmul(_plain_values(*_plain_quant(state["dy"].float())), w2)
    sig = 1.0 / (1.0 + torch.exp(-g))
    dgu = torch.cat((dh * u * sig * (1.0 + g * (1.0 - sig)), dh * g * sig), dim=1)
    return torch.matmul(_plain_values(*_plain_quant(dgu)), w1).to(torch.bfloat16)


# ------------------------------------------------------------- what it costs

def work(case):
    M = case["rows"]
    if case["op"] == "quant":
        return dict(bytes=3 * M * case["K"] + M * _blocks(case["K"]), flops=2 * M * case["K"])
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        return dict(bytes=2 * M * K + N * K + _blocks(N) * _blocks(K) + 2 * M * N + (2 * N if case["bias"] else 0),
                    flops=2 * M * N * K)
    H, I = case["H"], case["I"]
    weights = 3 * H * I + 3 * _blocks(H) * _blocks(I)
    kept = 4 * M * I if case["op"] == "grad" or case["keep"] else 0
    return dict(bytes=4 * M * H + weights + kept, flops=6 * M * H * I)


# ------------------------------------------------------- the definition, fp64

def _e4m3(v):
    """Nearest e4m3 value, ties to even: three bits after the first, or steps of 2^-9 below 2^-6."""
    _, e = torch.frexp(v)
    step = ((torch.clamp(e - 1, min=-6) - 3 + 1023).long() << 52).view(torch.float64)
    return torch.clamp(torch.round(v / step) * step, -TOP, TOP)


def _exact_quant(x):
    """Values the codes stand for (without their scales) and scales [M, blocks], block by block."""
    codes, scales = torch.empty_like(x), []
    for b in range(_blocks(x.shape[1])):
        part = x[:, b * B:(b + 1) * B]
        a = part.abs().max(dim=1).values
        s = torch.full_like(a, 2.0 ** LEAST)
        for _ in range(2 ** 8):  # doubled until the largest value fits
            short = a > TOP * s
            if not short.any():
                break
            s = torch.where(short, 2.0 * s, s)
        s = torch.where(a == 0, 1.0, s)
        codes[:, b * B:(b + 1) * B] = _e4m3(part / s[:, None])
        scales.append(s)
    return codes, torch.stack(scales, dim=1)


def _exact_values(x):
    codes, s = _exact_quant(x)
    for b in range(s.shape[1]):
        codes[:, b * B:(b + 1) * B] *= s[:, b:b + 1]
    return codes


def _exact_weight(codes, s):
    w, scales = codes.double(), s.double()
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            w[i * B:(i + 1) * B, j * B:(j + 1) * B] *= scales[i, j]
    return w


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quant":
        return _exact_quant(st["x"].double())
    if case["op"] == "linear":
        y = _exact_values(st["x"].double()) @ _exact_weight(*st["w"]).t()
        return y if st["bias"] is None else y + st["bias"].double()
    w1, w2, I = _exact_weight(*st["w1"]), _exact_weight(*st["w2"]), case["I"]
    if case["op"] == "ffn":
        x = _exact_values(st["x"].double())
        g, u = x @ w1[:I].t(), x @ w1[I:].t()
        out = _exact_values(g * torch.sigmoid(g) * u) @ w2.t()
        return (out, torch.cat((g, u), dim=1)) if case["keep"] else out
    g, u = st["gate_up"].double().split(I, dim=1)
    dh = _exact_values(st["dy"].double()) @ w2
    sig = torch.sigmoid(g)
    dg, du = dh * u * (sig + g * sig * torch.sigmoid(-g)), dh * g * sig
    return _exact_values(dg) @ w1[:I] + _exact_values(du) @ w1[I:]
