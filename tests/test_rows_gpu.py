"""The mixture-of-experts router and layer and the low-rank adapters against plain
fp64 implementations.

Tolerances are bounds derived from the arithmetic, element by element:
  * bf16 output: half a step, at most 2^-8 |ref|;
  * a sum of n fp32 terms in any order: n 2^-24 times the sum of their absolute
    values.  The kernels sum x (128 + q) s and x (z - 136 s), so the absolute
    values are those of these terms, not of x W;
  * between two products the intermediate value keeps 16 significant bits: 2^-16
    of it;
  * the error of an intermediate value reaches the output through the absolute
    values of the second weight; |d silu / dg| <= 1.1.
Routing ids are exact.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ck = pytest.importorskip("packed_int4_convrot_amd")

DEV = torch.device("cuda:0")
EPS = 2.0 ** -24
INF = float("inf")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


# ----------------------------------------------------------------- router

def ref_route(logits, k, renormalize):
    """ids int64 [T, k], weights fp64 [T, k], row by row from the definition."""
    l = logits.double().cpu().numpy()
    T, E = l.shape
    ids = np.full((T, k), -1, dtype=np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        v = np.where(np.isnan(l[t]), -INF, l[t])
        order = sorted((e for e in range(E) if v[e] > -INF), key=lambda e: (-v[e], e))
        if not order:
            continue
        top = v[order[0]]
        ex = np.array([(1.0 if v[e] == INF else 0.0) if top == INF else np.exp(v[e] - top) if v[e] > -INF else 0.0
                       for e in range(E)])
        sel = order[:k]
        den = ex[sel].sum() if renormalize else ex.sum()
        ids[t, :len(sel)] = sel
        w[t, :len(sel)] = ex[sel] / den
    return ids, w


def check_route(logits, k, renormalize, ids, w):
    rid, rw = ref_route(logits, k, renormalize)
    assert np.array_equal(ids.cpu().numpy(), rid)
    # exp (2 ulp), its argument's rounding (|d| ulp, |d| = -log of the weight at most), sums of up to 16 + 6
    # terms, a division
    w = w.cpu().numpy().astype(np.float64)
    d = -np.log(np.maximum(rw, 1e-38))
    assert (np.abs(w - rw) <= (40 + d) * EPS * rw + 1e-37).all(), np.abs(w - rw).max()


ROUTE = [(1, 1, 1), (1, 8, 3), (5, 60, 4), (3, 63, 8), (7, 64, 1), (2, 65, 2), (9, 128, 8), (6, 129, 32), (4, 256, 8),
         (3, 257, 6), (2, 1000, 32), (5, 1024, 10), (1030, 40, 5), (3, 4, 9)]


@pytest.mark.parametrize("T,E,k", ROUTE)
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route(T, E, k, kind, renormalize):
    l = (torch.randn((T, E), device=DEV, generator=gen(T + E)) * 3).to(kind)
    check_route(l, k, renormalize, *ck.moe_route(l, k, renormalize))


@pytest.mark.parametrize("E", [5, 64, 100, 200, 700])
def test_route_ties_masks_and_non_finite(E):
    g = gen(E)
    l = torch.randint(-2, 3, (48, E), device=DEV, generator=g).float()  # many ties
    l[1] = 0.0
    l[1, ::2] = -0.0                     # -0 ties with +0
    l[2] = -INF                          # nothing left
    l[3] = float("nan")
    l[4, 1:] = -INF                      # one expert
    l[5, E // 2] = INF
    l[6] = INF
    l[7, 0], l[7, -1] = float("nan"), INF
    l[8] = torch.finfo(torch.float32).min    # the lowest value is not -inf
    l[9, :E - 1] = torch.finfo(torch.float32).min
    l[10] = torch.finfo(torch.float32).tiny / 4 * torch.arange(E, device=DEV)  # denormals, in order
    l[11] = 1e-45
    l[11, 2] = 0.0
    l[12, :] = -INF
    l[12, -1] = -100.0
    for kind in (torch.float32, torch.bfloat16):
        for renorm in (True, False):
            check_route(l.to(kind), 4, renorm, *ck.moe_route(l.to(kind), 4, renorm))


def test_route_strided_and_empty():
    wide = torch.full((9, 100), float("nan"), device=DEV)
    wide[:, :70] = torch.randn((9, 70), device=DEV, generator=gen(1))
    l = wide[:, :70]
    check_route(l, 6, True, *ck.moe_route(l, 6))
    ids, w = ck.moe_route(torch.empty((0, 16), device=DEV), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)


# ------------------------------------------------------------------ experts

def expert_weights(E, H, I, zeros, seed):
    g = gen(seed)

    def one(N, K):
        p = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device=DEV, generator=g)
        s = torch.empty((E, K // 64, N), device=DEV).uniform_(0.002, 0.02, generator=g).bfloat16()
        z = torch.empty((E, K // 64, N), device=DEV).normal_(0, 0.01, generator=g).bfloat16() if zeros else None
        return p, s, z
    return one(2 * I, H) + one(H, I)


def dense64(p, s, z, e):
    """fp64 weight [N, K] of expert e, and the bound's weight 288 |s| + |z| (codes up to 143 and the offset 136)."""
    q = torch.stack((p[e] & 15, p[e] >> 4), dim=-1).flatten(-2).double() - 8
    sc = s[e].double().t().repeat_interleave(64, dim=1)
    zc = torch.zeros_like(sc) if z is None else z[e].double().t().repeat_interleave(64, dim=1)
    return q * sc + zc, 288 * sc.abs() + zc.abs()


def ref_experts(x, ids, w, tensors):
    """out fp64 [T, H] and the bound of its error, slot by slot."""
    w1, s1, z1, w2, s2, z2 = tensors
    T, H = x.shape
    E, I = w1.shape[0], w1.shape[1] // 2
    x = x.double()
    out = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    err = torch.zeros_like(out)
    n1, n2 = (H + 64) * EPS, (I + 64) * EPS
    ids, w = ids.long(), w.double()
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        a, aa = dense64(w1, s1, z1, e)
        b, ba = dense64(w2, s2, z2, e)
        y, dy = x[t] @ a.t(), n1 * (x[t].abs() @ aa.t())
        g, u, dg, du = y[:, :I], y[:, I:], dy[:, :I], dy[:, I:]
        silu = g * torch.sigmoid(g)
        h = silu * u
        dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + 2.0 ** -16 * h.abs() + 8 * EPS * h.abs()
        c = w[t, j].unsqueeze(1)
        out.index_add_(0, t, c * (h @ b.t()))
        err.index_add_(0, t, c.abs() * (dh @ b.abs().t() + n2 * ((h.abs() + dh) @ ba.t())))
    return out, err + 2.0 ** -8 * out.abs() + 64 * EPS * err


def assert_within(got, ref, bound):
    d = (got.double() - ref).abs()
    bad = ~(d <= bound)
    assert not bad.any(), "%d of %d outside, worst %.3g of the bound" % (
        int(bad.sum()), bad.numel(), float((d / bound.clamp(min=1e-300)).max()))


MOE = [(1, 64, 64, 1, 1), (1, 128, 64, 4, 2), (1, 512, 320, 40, 8), (2, 192, 128, 7, 3), (3, 192, 320, 5, 3),
       (8, 512, 192, 16, 4), (17, 448, 64, 3, 1), (33, 256, 128, 8, 2), (70, 128, 64, 4, 4), (129, 64, 64, 70, 8),
       (40, 1088, 704, 6, 6), (16, 64, 2112, 9, 2)]


@pytest.mark.parametrize("T,H,I,E,k", MOE)
@pytest.mark.parametrize("kind,renormalize,zeros", [(torch.float32, True, True), (torch.bfloat16, False, False)])
def test_moe(T, H, I, E, k, kind, renormalize, zeros):
    tensors = expert_weights(E, H, I, zeros, seed=H + I + T)
    g = gen(T * 7 + E)
    x = torch.randn((T, H), device=DEV, generator=g).bfloat16()
    l = torch.randn((T, E), device=DEV, generator=g).to(kind)
    print("moe T=%d H=%d I=%d E=%d k=%d" % (T, H, I, E, k), flush=True)
    out, ids, w = ck.moe(x, l, ck.MoeExperts(*tensors), k, renormalize)
    check_route(l, k, renormalize, ids, w)
    assert_within(out, *ref_experts(x, ids, w, tensors))
    again = ck.moe_experts(x, ids, w, ck.MoeExperts(*tensors))
    assert torch.equal(bits(out), bits(again))


def test_moe_many_tokens_run_in_passes():
    """More (token, slot) pairs than one pass holds, more slots than experts, strided rows."""
    T, H, I, E, k = 300, 128, 64, 3, 5
    tensors = expert_weights(E, H, I, True, seed=3)
    wide = torch.full((T, H + 24), float("nan"), device=DEV, dtype=torch.bfloat16)
    wide[:, :H] = torch.randn((T, H), device=DEV, generator=gen(5)).bfloat16()
    l = torch.randn((T, E), device=DEV, generator=gen(6))
    space = torch.full((T, H + 8), 7.0, device=DEV, dtype=torch.bfloat16)
    out, ids, w = ck.moe(wide[:, :H], l, ck.MoeExperts(*tensors), k, out=space[:, :H])
    check_route(l, k, True, ids, w)
    assert (ids[:, 3:] == -1).all()
    assert_within(out, *ref_experts(wide[:, :H], ids, w, tensors))
    assert (space[:, H:] == 7.0).all()


def test_moe_one_expert_takes_everything():
    T, H, I, E, k = 100, 192, 128, 64, 2
    tensors = expert_weights(E, H, I, True, seed=8)
    x = torch.randn((T, H), device=DEV, generator=gen(9)).bfloat16()
    l = torch.full((T, E), -INF, device=DEV)
    l[:, 61] = 1.0
    out, ids, w = ck.moe(x, l, ck.MoeExperts(*tensors), k)
    assert (ids == torch.tensor([61, -1], device=DEV)).all() and (w == torch.tensor([1.0, 0.0], device=DEV)).all()
    assert_within(out, *ref_experts(x, ids, w, tensors))


def test_moe_rows_without_experts_are_zero():
    T, H, I, E, k = 6, 128, 64, 8, 2
    tensors = expert_weights(E, H, I, True, seed=11)
    x = torch.randn((T, H), device=DEV, generator=gen(12)).bfloat16()
    l = torch.randn((T, E), device=DEV, generator=gen(13))
    l[2], l[5] = -INF, float("nan")
    experts = ck.MoeExperts(*tensors)
    out, ids, w = ck.moe(x, l, experts, k)
    assert not out[2].any() and not out[5].any() and (ids[2] == -1).all()
    assert_within(out, *ref_experts(x, ids, w, tensors))
    l[:] = -INF
    out, ids, w = ck.moe(x, l, experts, k)
    assert not out.any() and (ids == -1).all() and not w.any()
    out, _, _ = ck.moe(x[:0], l[:0], experts, k)
    assert out.shape == (0, H)


def test_moe_given_ids_with_empty_and_repeated_slots():
    T, H, I, E, k = 21, 256, 192, 6, 4
    tensors = expert_weights(E, H, I, False, seed=21)
    x = torch.randn((T, H), device=DEV, generator=gen(22)).bfloat16()
    ids = torch.randint(-3, E + 3, (T, k), device=DEV, generator=gen(23), dtype=torch.int32)
    ids[0] = 2                                   # one expert in every slot
    ids[1] = torch.tensor([-2 ** 31, 2 ** 31 - 1, E, -1], device=DEV)
    w = torch.randn((T, k), device=DEV, generator=gen(24))
    w[1] = float("nan")                          # the weight of an empty slot is not used
    experts = ck.MoeExperts(*tensors)
    out = ck.moe_experts(x, ids, w, experts)
    ref, bound = ref_experts(x, torch.where((ids < 0) | (ids >= E), -1, ids), torch.nan_to_num(w), tensors)
    assert_within(out, ref, bound)
    assert not out[1].any()


def test_moe_non_finite_token_stays_in_its_row():
    T, H, I, E, k = 40, 128, 64, 2, 2            # every token shares its tiles with others
    tensors = expert_weights(E, H, I, True, seed=31)
    experts = ck.MoeExperts(*tensors)
    x = torch.randn((T, H), device=DEV, generator=gen(32)).bfloat16()
    l = torch.randn((T, E), device=DEV, generator=gen(33))
    clean, _, _ = ck.moe(x, l, experts, k)
    x[3, 5], x[20, 100], x[21] = float("nan"), INF, -INF
    out, _, _ = ck.moe(x, l, experts, k)
    rest = [t for t in range(T) if t not in (3, 20, 21)]
    assert torch.equal(bits(out[rest]), bits(clean[rest]))
    assert not torch.isfinite(out[[3, 20, 21]].float()).any()


def test_moe_large_activations():
    """Gates far from zero: silu(g) is g or 0, without NaN."""
    T, H, I, E, k = 4, 128, 64, 2, 1
    tensors = expert_weights(E, H, I, True, seed=41)
    x = (torch.randn((T, H), device=DEV, generator=gen(42)) * 3e4).bfloat16()
    l = torch.randn((T, E), device=DEV, generator=gen(43))
    out, ids, w = ck.moe(x, l, ck.MoeExperts(*tensors), k)
    assert_within(out, *ref_experts(x, ids, w, tensors))


def test_moe_same_bits_again_in_graphs_and_on_other_streams():
    T, H, I, E, k = 24, 320, 192, 12, 3
    tensors = expert_weights(E, H, I, True, seed=51)
    experts = ck.MoeExperts(*tensors)
    xs = [torch.randn((T, H), device=DEV, generator=gen(52 + i)).bfloat16() for i in range(3)]
    ls = [torch.randn((T, E), device=DEV, generator=gen(62 + i)) for i in range(3)]
    want = [ck.moe(x, l, experts, k) for x, l in zip(xs, ls)]
    for (x, l), wo in zip(zip(xs, ls), want):
        for a, b in zip(ck.moe(x, l, experts, k), wo):
            assert torch.equal(bits(a), bits(b))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ck.moe(xs[1], ls[1], experts, k)
    side.synchronize()
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want[1]))
    x, l = xs[0].clone(), ls[0].clone()
    ck.moe(x, l, experts, k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ck.moe(x, l, experts, k)
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        l.copy_(ls[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want[i]))


def test_moe_weights_beyond_32_bit_offsets():
    """Expert slabs of more than 4 GiB: the last experts, and only they, are filled."""
    T, H, I, E, k = 2, 4096, 1280, 1024, 2
    small = expert_weights(2, H, I, True, seed=71)
    big = []
    for t in small:
        b = torch.empty((E,) + tuple(t.shape[1:]), dtype=t.dtype, device=DEV)
        b[E - 2:] = t
        big.append(b)
    assert big[0].numel() > 2 ** 32
    x = torch.randn((T, H), device=DEV, generator=gen(72)).bfloat16()
    ids = torch.tensor([[E - 1, E - 2], [E - 2, E - 1]], dtype=torch.int32, device=DEV)
    w = torch.rand((T, k), device=DEV, generator=gen(73))
    out = ck.moe_experts(x, ids, w, ck.MoeExperts(*big))
    assert_within(out, *ref_experts(x, ids - (E - 2), w, small))


# ----------------------------------------------------------------- adapters

def ref_lora(x, a, b, scaling, ranks, index, base):
    M, (L, R, K), N = x.shape[0], a.shape, b.shape[1]
    out = torch.zeros((M, N), dtype=torch.float64, device=DEV) if base is None else base.double()
    err = 2.0 ** -24 * out.abs()
    for l in range(L):
        rows = (index == l).nonzero().flatten()
        r = R if ranks is None else min(max(int(ranks[l]), 0), R)
        s = 1.0 if scaling is None else float(scaling[l])
        if not rows.numel() or not r:
            continue
        xa, aa, ba = x[rows].double(), a[l, :r].double(), b[l, :, :r].double()
        v = xa @ aa.t()
        dv = (K + 64) * EPS * (xa.abs() @ aa.abs().t()) + 2.0 ** -16 * v.abs()
        out[rows] = out[rows] + s * (v @ ba.t())
        err[rows] += abs(s) * ((dv + (R + 64) * EPS * v.abs()) @ ba.abs().t())
    return out, err + 2.0 ** -8 * out.abs() + 4 * EPS * err


def lora_case(M, K, N, R, L, seed, ranks=True, base=True):
    g = gen(seed)
    x = torch.randn((M, K), device=DEV, generator=g).bfloat16()
    a = (torch.randn((L, R, K), device=DEV, generator=g) / K ** 0.5).bfloat16()
    b = (torch.randn((L, N, R), device=DEV, generator=g) * 0.3).bfloat16()
    scaling = torch.empty((L,), device=DEV).uniform_(-2, 2, generator=g)
    rk = torch.randint(0, R + 1, (L,), device=DEV, generator=g, dtype=torch.int32) if ranks else None
    index = torch.randint(-1, L, (M,), device=DEV, generator=g, dtype=torch.int32)
    y = torch.randn((M, N), device=DEV, generator=g).bfloat16() if base else None
    return x, a, b, scaling, rk, index, y


LORA = [(1, 64, 16, 8, 1), (1, 3840, 512, 16, 3), (2, 128, 48, 8, 3), (17, 192, 272, 24, 2), (33, 320, 144, 40, 33),
        (64, 128, 128, 64, 5), (65, 448, 160, 72, 9), (200, 64, 32, 128, 3), (256, 192, 80, 16, 300),
        (257, 192, 80, 16, 4), (300, 576, 528, 40, 2), (700, 128, 272, 256, 5), (1000, 1088, 304, 64, 40),
        (1025, 192, 528, 24, 3), (1300, 640, 176, 136, 30), (2111, 320, 1040, 64, 2)]


@pytest.mark.parametrize("M,K,N,R,L", LORA)
@pytest.mark.parametrize("ranks,base", [(True, True), (False, False)])
def test_lora(M, K, N, R, L, ranks, base):
    x, a, b, sc, rk, index, y = lora_case(M, K, N, R, L, seed=M + K + N, ranks=ranks, base=base)
    print("lora M=%d K=%d N=%d R=%d L=%d" % (M, K, N, R, L), flush=True)
    out = ck.lora_add(x, ck.LoraAdapters(a, b, sc, rk), index, base=y)
    assert_within(out, *ref_lora(x, a, b, sc, rk, index, y))


@pytest.mark.parametrize("M", [50, 600, 1500])
def test_lora_runs_of_rows_and_no_scaling(M):
    """Prompts packed one after the other, an adapter for each, some without."""
    x, a, b, _, _, _, y = lora_case(M, 256, 192, 32, 6, seed=M)
    index = (torch.arange(M, device=DEV, dtype=torch.int32) * 9 // M) % 8 - 1
    out = ck.lora_add(x, ck.LoraAdapters(a, b), index, base=y)
    assert_within(out, *ref_lora(x, a, b, None, None, index, y))


@pytest.mark.parametrize("M", [40, 300, 1200])
def test_lora_rows_without_an_adapter_keep_base(M):
    x, a, b, sc, rk, _, y = lora_case(M, 128, 80, 16, 3, seed=M)
    index = torch.full((M,), -1, dtype=torch.int32, device=DEV)
    index[::3], index[1::3], index[2::3] = 3, -2 ** 31, 2 ** 31 - 1
    adapters = ck.LoraAdapters(a, b, sc)
    assert torch.equal(bits(ck.lora_add(x, adapters, index, base=y)), bits(y))
    assert not ck.lora_add(x, adapters, index).any()
    # ranks of zero and below
    rk = torch.tensor([0, -4, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    index = torch.randint(0, 2, (M,), device=DEV, generator=gen(1), dtype=torch.int32)
    assert torch.equal(bits(ck.lora_add(x, ck.LoraAdapters(a, b, sc, rk), index, base=y)), bits(y))
    index[:] = 2                                # a rank above R counts as R
    out = ck.lora_add(x, ck.LoraAdapters(a, b, sc, rk), index, base=y)
    assert_within(out, *ref_lora(x, a, b, sc, None, index, y))


@pytest.mark.parametrize("M", [9, 70, 1100])
def test_lora_rows_without_an_adapter_beside_rows_that_have_one(M):
    """They keep every bit of base (-0 and NaN too), whatever the neighbours' adapter holds."""
    x, a, b, _, _, _, y = lora_case(M, 128, 80, 16, 2, seed=M)
    index = torch.randint(-1, 2, (M,), device=DEV, generator=gen(M), dtype=torch.int32)
    index[0], index[-1] = -1, 1
    b[1, 5, 3], b[1, 7, 0] = float("inf"), float("nan")
    y[:, 3], y[:, 4], y[:, 6] = -0.0, float("nan"), float("inf")
    out = ck.lora_add(x, ck.LoraAdapters(a, b), index, base=y)
    assert torch.equal(bits(out)[index < 0], bits(y)[index < 0])
    assert out[index == 1][:, [5, 7]].float().isfinite().sum() == 0
    keep = [c for c in range(80) if c not in (3, 4, 5, 6, 7)]
    ref, tol = ref_lora(x, a, b, None, None, index, y)
    assert_within(out[:, keep], ref[:, keep], tol[:, keep])


@pytest.mark.parametrize("M,R", [(37, 40), (290, 40), (5, 200), (280, 200), (1100, 40)])
def test_lora_ignores_what_lies_beyond_a_rank(M, R):
    x, a, b, sc, _, index, y = lora_case(M, 192, 144, R, 4, seed=M)
    rk = torch.tensor([R - 3, 1, R // 2, R], dtype=torch.int32, device=DEV)
    ref = ref_lora(x, a, b, sc, rk, index, y)
    for l, r in enumerate(rk.tolist()):
        a[l, r:], b[l, :, r:] = float("nan"), float("nan")
    assert_within(ck.lora_add(x, ck.LoraAdapters(a, b, sc, rk), index, base=y), *ref)


@pytest.mark.parametrize("M", [30, 270, 1070])
def test_lora_strided_in_place_and_isolated_rows(M):
    K, N = 192, 96
    x, a, b, sc, rk, index, y = lora_case(M, K, N, 24, 3, seed=M)
    adapters = ck.LoraAdapters(a, b, sc, rk)
    want = ck.lora_add(x, adapters, index, base=y)
    wide = torch.full((M, K + 16), float("nan"), device=DEV, dtype=torch.bfloat16)
    wide[:, :K] = x
    space = torch.full((M, N + 8), 5.0, device=DEV, dtype=torch.bfloat16)
    space[:, :N] = y
    got = ck.lora_add(wide[:, :K], adapters, index, base=space[:, :N], out=space[:, :N])
    assert torch.equal(bits(got), bits(want)) and (space[:, N:] == 5.0).all()
    x[4], x[9, 3] = float("nan"), INF
    index[4], index[9] = 0, 1
    rk[:] = 24
    sick = ck.lora_add(x, adapters, index, base=y)
    x[4], x[9, 3] = 0.0, 0.0
    well = ck.lora_add(x, adapters, index, base=y)
    rest = [m for m in range(M) if m not in (4, 9)]
    assert torch.equal(bits(sick[rest]), bits(well[rest]))
    assert torch.isnan(sick[4]).all() and not torch.isfinite(sick[9].float()).any()


def test_lora_same_bits_again_in_graphs_and_on_other_streams():
    for M in (20, 400, 1400):
        x, a, b, sc, rk, index, y = lora_case(M, 640, 208, 32, 5, seed=M)
        adapters = ck.LoraAdapters(a, b, sc, rk)
        other = torch.flip(index, (0,)).contiguous()
        want = [ck.lora_add(x, adapters, i, base=y) for i in (index, other)]
        assert torch.equal(bits(ck.lora_add(x, adapters, index, base=y)), bits(want[0]))
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = ck.lora_add(x, adapters, other, base=y)
        side.synchronize()
        assert torch.equal(bits(got), bits(want[1]))
        held = index.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = ck.lora_add(x, adapters, held, base=y)
        for i in (1, 0, 1):
            held.copy_((index, other)[i])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(bits(got), bits(want[i]))


def test_lora_no_rows():
    x, a, b, sc, rk, index, y = lora_case(4, 64, 32, 8, 2, seed=1)
    assert ck.lora_add(x[:0], ck.LoraAdapters(a, b), index[:0], base=y[:0]).shape == (0, 32)


def test_lora_slots_beyond_32_bit_offsets():
    M, K, N, R, L = 3, 16384, 64, 256, 600
    _, a, b, _, _, _, y = lora_case(M, K, N, R, 1, seed=2)
    x = torch.randn((M, K), device=DEV, generator=gen(3)).bfloat16()
    big_a = torch.empty((L, R, K), dtype=torch.bfloat16, device=DEV)
    big_b = torch.empty((L, N, R), dtype=torch.bfloat16, device=DEV)
    assert big_a.numel() > 2 ** 31
    big_a[L - 1], big_b[L - 1] = a[0], b[0]
    index = torch.tensor([L - 1, -1, L - 1], dtype=torch.int32, device=DEV)
    out = ck.lora_add(x, ck.LoraAdapters(big_a, big_b), index, base=y)
    assert_within(out, *ref_lora(x, a, b, None, None, torch.where(index >= 0, 0, -1), y))


def test_bindings_refuse_what_does_not_fit():
    x, a, b, sc, rk, index, y = lora_case(8, 128, 48, 16, 2, seed=4)
    adapters = ck.LoraAdapters(a, b, sc, rk)
    space = torch.empty(ck.lora_workspace_bytes(8, 128, 16, 2) - 256, dtype=torch.uint8, device=DEV)
    with pytest.raises(ck.CKError, match="workspace"):
        ck.lora_add(x, adapters, index, base=y, workspace=space)
    for bad in (dict(index=index.long()), dict(index=index[:7]), dict(x=x.float()), dict(x=x[:, :64]),
                dict(base=y[:7]), dict(base=y.cpu()), dict(x=x[:1].expand(8, 128)), dict(out=y[:, :32])):
        args = dict(x=x, index=index, base=y, out=None)
        args.update(bad)
        with pytest.raises(ValueError):
            ck.lora_add(args["x"], adapters, args["index"], base=args["base"], out=args["out"])
    with pytest.raises(ValueError):
        ck.LoraAdapters(a, b[:, :, :8].contiguous())
    with pytest.raises(ValueError):
        ck.lora_add(x, adapters, index, base=y, out=torch.as_strided(y, (8, 48), (48, 1), 0)[:, :48].t().contiguous().t())
    tensors = expert_weights(4, 128, 64, True, seed=5)
    experts = ck.MoeExperts(*tensors)
    l = torch.randn((8, 4), device=DEV)
    for bad in (dict(x=x[:7]), dict(l=l.half()), dict(l=l[:, :3]), dict(l=l[0]), dict(l=l.t().contiguous().t())):
        args = dict(x=x, l=l)
        args.update(bad)
        with pytest.raises(ValueError):
            ck.moe(args["x"], args["l"], experts, 2)
    with pytest.raises(ck.CKError):
        ck.moe(x, l, experts, 33)
    with pytest.raises(ValueError):
        ck.moe(x, l, experts, 0)
    with pytest.raises(ValueError):
        ck.MoeExperts(*tensors[:3], tensors[3][:, :64], *tensors[4:])
    with pytest.raises(ValueError):
        ck.moe_experts(x, torch.zeros((8, 2), dtype=torch.int64, device=DEV), torch.zeros((8, 2), device=DEV), experts)
    with pytest.raises(ValueError):
        ck.moe_route(l.half(), 2)
