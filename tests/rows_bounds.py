"""The mixture-of-experts layer in fp64 with an error bound close to the error that fp32
arithmetic makes, shared by the GPU tests and by the test that the bound refuses wrong results.

Per 64 columns g of a row a and a weight row n the kernels form s P + (z - 136 s) X, with
P = sum a (128 + q) and X = sum a in fp32, and add the groups up in fp32.  With u = 2^-24:
  * within a group every rounding is at most u times the sum of |a| (128 + q) s, or of
    |a| (136 s + |z|): at most u (280 s + |z|) A_g together, A_g the group's sum of |a|;
    72 of them;
  * over groups (two additions each) and parts of the columns (64 at most) a rounding is at
    most u times the sum of |a| |W|;
  * roundings are of either sign, so n of them add up to no more than 8 sqrt(n) times the
    largest but for a probability of e^-32 (a sum of bounded differences);
  * h keeps 16 significant bits, 2^-16 of it, and carries the errors of gate and up,
    |d silu / dg| <= 1.1; their sum over the second weight is again one of either sign;
  * bf16 output: half a step, at most 2^-8 of it.
A bound element by element lets pass what is smaller than the output's rounding.  Against
that the root mean square of the whole error may exceed the correctly rounded result's by a
tenth: what the kernels add is below a fifth of the rounding (1.02 together), one bf16 for h
would add as much as the rounding itself (1.41).
"""
import torch

U = 2.0 ** -24
SURE = 8.0
RMS = 1.1


def expert_weights(E, H, I, zeros, seed, device="cpu"):
    """Random (w1, s1, z1, w2, s2, z2), the same on every device."""
    g = torch.Generator().manual_seed(seed)

    def one(N, K):
        p = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, generator=g)
        s = torch.empty((E, K // 64, N)).uniform_(0.002, 0.02, generator=g).bfloat16()
        z = torch.empty((E, K // 64, N)).normal_(0, 0.01, generator=g).bfloat16() if zeros else None
        return p, s, z
    return [None if t is None else t.to(device) for t in one(2 * I, H) + one(H, I)]


def dense(p, s, z):
    """fp64 weight [N, K] of one expert."""
    q = torch.stack((p & 15, p >> 4), dim=-1).flatten(-2).double() - 8
    w = q * s.double().t().repeat_interleave(64, dim=1)
    return w if z is None else w + z.double().t().repeat_interleave(64, dim=1)


def product(a, w, s, z, parts):
    """a W^T and its error's bound; `parts` rows of A make up one row of a."""
    groups = a.shape[1] // 64
    reach = 280 * s.double().abs() + (0 if z is None else z.double().abs())       # [G, N]
    within = a.abs().view(-1, groups, 64).sum(dim=2).square() @ reach.square()
    return a @ w.t(), SURE * U * ((72 * parts * within).sqrt() + (2 * groups * parts + 64) ** 0.5 * (a.abs() @ w.abs().t()))


def layer(x, ids, w, tensors, hidden=lambda h: h, pick=lambda e: e):
    """out fp64 [T, H] and its error's bound before the last rounding.  `hidden` changes h and
    `pick` the expert whose weights are taken: mistakes to be refused."""
    w1, s1, z1, w2, s2, z2 = tensors
    I = w2.shape[2] * 2
    out = torch.zeros((x.shape[0], w2.shape[1]), dtype=torch.float64, device=x.device)
    err = torch.zeros_like(out)
    for e in range(w1.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        p = pick(e)
        y, dy = product(x[t].double(), dense(w1[p], s1[p], None if z1 is None else z1[p]), s1[p],
                        None if z1 is None else z1[p], 1)
        g, u, dg, du = y[:, :I], y[:, I:], dy[:, :I], dy[:, I:]
        silu = g * torch.sigmoid(g)
        h = hidden(silu * u)
        dh = 1.1 * dg * u.abs() + (silu.abs() + 1.1 * dg) * du + (2.0 ** -16 + 8 * U) * h.abs()
        b = dense(w2[p], s2[p], None if z2 is None else z2[p])
        y, dy = product(h, b, s2[p], None if z2 is None else z2[p], 2)
        c = w[t, j].double().unsqueeze(1)
        out.index_add_(0, t, c * y)
        err.index_add_(0, t, c.abs() * (dy + SURE * (dh.square() @ b.square().t()).sqrt() + 2 * ids.shape[1] * U * y.abs()))
    return out, err


def refused(got, ref, err):
    """None for a result within the bounds, else what it fails."""
    d = (got.double() - ref).abs()
    worst = (d / (err + 2.0 ** -8 * (ref.abs() + err)).clamp(min=1e-300)).max()
    if not worst <= 1:
        return "an element is off by %.3g of its bound" % worst
    rounding = (ref.to(torch.bfloat16).double() - ref).square().mean().sqrt()
    rms = d.square().mean().sqrt()
    if not rms <= RMS * rounding:
        return "the error is %.3f of the rounding's" % (rms / rounding)
    return None


# T, H, I, E, k, crowded: expert 0 takes every token, so that sets of eight pairs stand beside
# sets of few.
LAYERS = [
    (1, 512, 320, 40, 8, False), (8, 512, 192, 16, 4, False), (40, 1088, 704, 6, 6, False), (33, 256, 128, 8, 2, True),
    (129, 64, 64, 70, 8, False), (8, 3840, 1280, 4, 2, False), (12, 3840, 1280, 4, 2, False),
    (37, 2112, 832, 6, 5, True),
    # x in chunks: sets of more than four pairs from 4096 columns on, all from 8192 on; passes cut by the results' room
    (20, 4160, 192, 16, 2, True), (20, 8256, 128, 16, 2, True), (40, 8256, 64, 16, 1, True), (40, 16384, 64, 16, 1, True),
    (3, 32768, 64, 3, 2, False),
    # one token and a few whose hidden columns do not fit the few-pair form; h in chunks from 2048 columns on
    (1, 192, 1600, 40, 8, False), (2, 64, 2112, 9, 2, False), (20, 128, 2112, 8, 2, True), (24, 64, 4160, 6, 2, True),
    # sixteen logits a lane in front of few pairs; more than eight slots
    (1, 128, 64, 300, 8, False), (2, 64, 128, 1024, 8, False), (1, 128, 64, 20, 12, False), (5, 128, 192, 40, 20, False),
    (3, 64, 128, 64, 32, False),
]


def layer_inputs(T, H, I, E, k, crowded, device="cpu"):
    """x, logits and weights of a case, the same on every device (zero points but for odd k)."""
    g = torch.Generator().manual_seed(T * 7 + H + I)
    x = torch.randn((T, H), generator=g).bfloat16().to(device)
    logits = torch.randn((T, E), generator=g)
    if crowded:
        logits[:, 0] += 4
    return x, logits.to(device), expert_weights(E, H, I, k % 2 == 0, T + H + I + E, device)


# M, K, N, R, L: each form of the second product (one wave and four a workgroup, many rows)
# at 16, 32, 64 ranks and beyond.
ADAPTERS = [(1, 3840, 512, 16, 3), (16, 192, 272, 24, 16), (32, 3840, 1024, 16, 32), (40, 256, 272, 24, 5),
            (301, 1024, 528, 40, 7), (100, 320, 144, 136, 3), (200, 192, 272, 16, 3), (300, 192, 1040, 16, 40),
            (300, 192, 1040, 24, 40), (300, 192, 1040, 64, 40), (300, 128, 1040, 200, 40), (1030, 3840, 80, 16, 4),
            (1025, 192, 528, 24, 3), (1300, 1024, 528, 64, 8), (1100, 640, 272, 136, 30)]


def adapter_inputs(M, K, N, R, L, device="cpu"):
    """x, index and (a, b, scaling, ranks), the same on every device."""
    g = torch.Generator().manual_seed(M + K + N + R + L)
    x = torch.randn((M, K), generator=g).bfloat16()
    a = (torch.randn((L, R, K), generator=g) / K ** 0.5).bfloat16()
    b = (torch.randn((L, N, R), generator=g) * 0.3).bfloat16()
    scaling = torch.empty((L,)).uniform_(0.5, 2, generator=g)
    ranks = torch.randint(R // 2, R + 1, (L,), dtype=torch.int32, generator=g)
    index = torch.randint(-1, L, (M,), dtype=torch.int32, generator=g)
    index[0] = 0
    return x.to(device), index.to(device), tuple(t.to(device) for t in (a, b, scaling, ranks))


def adapters(x, index, tensors, between=lambda v: v, pick=lambda l: l):
    """out fp64 [M, N] without base and its error's bound before the last rounding, as `layer`:
    sums of K and R terms, scaling A x held to 16 significant bits."""
    a, b, scaling, ranks = tensors
    K, R = a.shape[2], a.shape[1]
    out = torch.zeros((x.shape[0], b.shape[1]), dtype=torch.float64, device=x.device)
    err = torch.zeros_like(out)
    for l in range(a.shape[0]):
        rows = (index == l).nonzero().flatten()
        if not rows.numel():
            continue
        p = pick(l)
        r = int(ranks[p])
        xa, aa, ba = x[rows].double(), a[p, :r].double(), b[p, :, :r].double()
        v = between(float(scaling[p]) * (xa @ aa.t()))
        dv = abs(float(scaling[p])) * SURE * U * (K + 64) ** 0.5 * (xa.abs() @ aa.abs().t()) + (2.0 ** -16 + 4 * U) * v.abs()
        out[rows] = v @ ba.t()
        err[rows] = SURE * (dv.square() @ ba.square().t()).sqrt() + SURE * U * (2 * R + 64) ** 0.5 * (v.abs() @ ba.abs().t())
    return out, err
