"""What is measured of the operators that choose weights row by row: the
mixture-of-experts router, the whole mixture-of-experts layer on packed uint4
experts, and the low-rank adapters of many requests beside a shared projection.

`run` computes a case either in plain torch operations in fp32 (`own` false) or
through the library's entry points (`own` true), on the same prepared inputs; the
library's result buffers and workspace are kept from step to step, as a serving loop does.
`exact` is the definition in fp64.
"""
import math

import torch

own = False

DEV = "cuda:0"
INF = float("inf")


def listed():
    return [
        # One token through a small layer: the latency of a decode step.
        dict(name="moe_one_token_small", op="moe", tokens=1, hidden=2048, inter=768, experts=32, k=2,
             logits="bf16", renormalize=True, zeros=True),
        # One token of an ordinary layer, eight experts.
        dict(name="moe_one_token", op="moe", tokens=1, hidden=3840, inter=1280, experts=64, k=8,
             logits="fp32", renormalize=True, zeros=True),
        # A small decode batch (or one request's drafted tokens).
        dict(name="moe_batch_8", op="moe", tokens=8, hidden=3840, inter=1280, experts=64, k=8,
             logits="bf16", renormalize=True, zeros=False),
        # Odd everything: tokens, experts, group counts; softmax over all experts kept as it is.
        dict(name="moe_odd_37", op="moe", tokens=37, hidden=2112, inter=832, experts=60, k=5,
             logits="fp32", renormalize=False, zeros=True),
        # The largest decode batch: most experts of a wide layer are active.
        dict(name="moe_batch_64", op="moe", tokens=64, hidden=3840, inter=1280, experts=128, k=8,
             logits="fp32", renormalize=True, zeros=True),
        # The router alone, in a decode step and over a prompt (some experts masked off).
        dict(name="route_batch_5", op="route", tokens=5, experts=60, k=4, logits="bf16", renormalize=False,
             masked=0),
        dict(name="route_prompt", op="route", tokens=8192, experts=256, k=8, logits="fp32", renormalize=True,
             masked=37),
        # One decode row and its adapter.
        dict(name="lora_one_row", op="lora", rows=1, K=3840, N=3840, rank=16, adapters=4, order="mixed",
             none=0.0, ranks=False, base=True),
        # A decode batch of many requests, each with its own adapter or none, of unlike ranks.
        dict(name="lora_batch_32", op="lora", rows=32, K=3840, N=10240, rank=16, adapters=32, order="mixed",
             none=0.15, ranks=True, base=True),
        # An odd batch of short prompts on a few adapters.
        dict(name="lora_odd_301", op="lora", rows=301, K=10240, N=3840, rank=40, adapters=7, order="segments",
             none=0.1, ranks=True, base=True),
        # The largest: packed prompts of many requests.
        dict(name="lora_prompt", op="lora", rows=8192, K=3840, N=10240, rank=64, adapters=8, order="segments",
             none=0.1, ranks=False, base=True),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return min(hi, max(lo, int(v) // step * step))


def draw(rng):
    op = rng.choice(("moe", "moe", "route", "lora", "lora"))
    if op == "moe":
        E = _log(rng, 8, 128)
        return dict(op=op, tokens=_log(rng, 1, 64), hidden=_log(rng, 512, 3840, 64), inter=_log(rng, 192, 1280, 64),
                    experts=E, k=rng.randint(1, 8), logits=rng.choice(("bf16", "fp32")),
                    renormalize=rng.random() < 0.5, zeros=rng.random() < 0.7)
    if op == "route":
        E = _log(rng, 8, 256)
        return dict(op=op, tokens=_log(rng, 1, 8192), experts=E, k=rng.randint(1, 8),
                    logits=rng.choice(("bf16", "fp32")), renormalize=rng.random() < 0.5,
                    masked=rng.choice((0, E // 3)))
    return dict(op=op, rows=_log(rng, 1, 8192), K=_log(rng, 512, 3840, 64), N=_log(rng, 512, 10240, 16),
                rank=8 * rng.randint(1, 8), adapters=_log(rng, 1, 8), order=rng.choice(("mixed", "segments")),
                none=rng.choice((0.0, 0.2)), ranks=rng.random() < 0.5, base=rng.random() < 0.8)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _packed_weight(g, E, N, K, zeros):
    packed = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    s = torch.empty((E, K // 64, N), device=DEV).uniform_(0.002, 0.02, generator=g).to(torch.bfloat16)
    z = torch.empty((E, K // 64, N), device=DEV).normal_(0.0, 0.01, generator=g).to(torch.bfloat16) if zeros else None
    return packed, s, z


def _logits(g, T, E, kind, masked=0):
    l = torch.randn((T, E), device=DEV, generator=g)
    if masked:  # the same experts are off for every token (a failed or drained device)
        off = torch.randperm(E, device=DEV, generator=g)[:masked]
        l[:, off] = -INF
    return l.to(torch.bfloat16) if kind == "bf16" else l


def _rank_of(case, l):
    """Ranks of a mixed set of adapters: full, half, and an odd one."""
    R = case["rank"]
    return (R, R // 2, R - 3)[l % 3] if case["ranks"] else R


def _slots(case):
    """The ids and weights that a serving loop keeps from step to step."""
    shape = (case["tokens"], case["k"])
    return (torch.empty(shape, dtype=torch.int32, device=DEV), torch.empty(shape, dtype=torch.float32, device=DEV))


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    if case["op"] == "route":
        st["logits"] = _logits(g, case["tokens"], case["experts"], case["logits"], case["masked"])
        st["k"] = case["k"]
        if own:
            import packed_int4_convrot_amd as ck
            st["ck"] = ck
            st["slots"] = _slots(case)
    elif case["op"] == "moe":
        T, H, I, E = case["tokens"], case["hidden"], case["inter"], case["experts"]
        st["x"] = torch.randn((T, H), device=DEV, generator=g).to(torch.bfloat16)
        st["logits"] = _logits(g, T, E, case["logits"])
        st["k"] = case["k"]
        st["w1"] = _packed_weight(g, E, 2 * I, H, case["zeros"])
        st["w2"] = _packed_weight(g, E, H, I, case["zeros"])
        if own:
            import packed_int4_convrot_amd as ck
            st["ck"] = ck
            st["experts"] = ck.MoeExperts(*st["w1"], *st["w2"])
            st["slots"] = _slots(case)
            st["out"] = torch.empty_like(st["x"])
            st["space"] = torch.empty(ck.moe_workspace_bytes(T, I, E, case["k"]), dtype=torch.uint8, device=DEV)
    else:
        M, K, N, R, L = case["rows"], case["K"], case["N"], case["rank"], case["adapters"]
        st["x"] = torch.randn((M, K), device=DEV, generator=g).to(torch.bfloat16)
        st["a"] = (torch.randn((L, R, K), device=DEV, generator=g) / K ** 0.5).to(torch.bfloat16)
        st["b"] = (torch.randn((L, N, R), device=DEV, generator=g) * 0.2).to(torch.bfloat16)
        st["scaling"] = torch.empty((L,), device=DEV).uniform_(0.25, 2.0, generator=g)
        st["ranks"] = torch.tensor([_rank_of(case, l) for l in range(L)], dtype=torch.int32, device=DEV)
        if case["order"] == "mixed":
            idx = torch.randint(0, L, (M,), device=DEV, generator=g)
            idx = torch.where(torch.rand((M,), device=DEV, generator=g) < case["none"], -1, idx)
        else:  # packed requests: runs of rows of random lengths, two for each adapter on average
            runs = min(M, 2 * L)
            starts = torch.rand((M,), device=DEV, generator=g).argsort()[:runs].sort().values
            of_run = torch.randint(0, L, (runs + 1,), device=DEV, generator=g)
            of_run = torch.where(torch.rand((runs + 1,), device=DEV, generator=g) < case["none"], -1, of_run)
            idx = of_run[torch.searchsorted(starts, torch.arange(M, device=DEV), right=True)]
        st["index"] = idx.to(torch.int32)
        st["base"] = torch.randn((M, N), device=DEV, generator=g).to(torch.bfloat16) if case["base"] else None
        if own:
            import packed_int4_convrot_amd as ck
            st["ck"] = ck
            st["adapters"] = ck.LoraAdapters(st["a"], st["b"], scaling=st["scaling"],
                                             ranks=st["ranks"] if case["ranks"] else None)
            st["out"] = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
            st["space"] = torch.empty(ck.lora_workspace_bytes(M, K, R, L), dtype=torch.uint8, device=DEV)
    return st


# -------------------------------------------------------------- plain forms

def _plain_route(logits, k, renormalize):
    l = logits.float()
    l = torch.where(torch.isnan(l), -INF, l)
    v, order = torch.sort(l, dim=1, descending=True, stable=True)
    sel, ids = v[:, :k], order[:, :k].to(torch.int32)
    if sel.shape[1] < k:  # fewer experts than slots
        pad = (0, k - sel.shape[1])
        sel, ids = torch.nn.functional.pad(sel, pad, value=-INF), torch.nn.functional.pad(ids, pad, value=-1)
    m = v[:, :1]
    ids = torch.where(sel == -INF, -1, ids)

    def ex(t):
        e = torch.where(m == INF, (t == INF).float(), torch.exp(t - m))
        return torch.where(t == -INF, 0.0, e)
    e = ex(sel)
    den = (e if renormalize else ex(v)).sum(dim=1, keepdim=True)
    return ids, torch.where(den > 0, e / den, 0.0)


def _plain_weight(packed, s, z):
    """fp32 [E, N, K] of packed uint4 weights."""
    q = torch.stack((packed & 15, packed >> 4), dim=-1).flatten(-2).float() - 8.0
    E, N, K = q.shape
    q = q.view(E, N, K // 64, 64) * s.float().transpose(1, 2).unsqueeze(-1)
    if z is not None:
        q += z.float().transpose(1, 2).unsqueeze(-1)
    return q.view(E, N, K)


def _plain_moe(st):
    case, x = st["case"], st["x"].float()
    ids, w = _plain_route(st["logits"], st["k"], case["renormalize"])
    T, k, E, I = x.shape[0], st["k"], case["experts"], case["inter"]
    if T * k <= E:  # the chosen experts' weights, slot by slot
        at = ids.clamp(min=0).flatten().long()
        pick = lambda t: None if t is None else t[at]  # noqa: E731
        w1, w2 = (_plain_weight(*(pick(t) for t in st[n])) for n in ("w1", "w2"))
        y = torch.matmul(w1, x.repeat_interleave(k, dim=0).unsqueeze(-1))
        g, u = y[:, :I], y[:, I:]
        y = torch.matmul(w2, g / (1.0 + torch.exp(-g)) * u).view(T, k, -1)
        out = torch.where(ids.unsqueeze(-1) >= 0, w.unsqueeze(-1) * y, 0.0).sum(dim=1)
    else:  # every expert for every token, and the chosen ones' weights
        w1, w2 = _plain_weight(*st["w1"]), _plain_weight(*st["w2"])
        y = torch.matmul(x.unsqueeze(0), w1.transpose(1, 2))
        g, u = y[..., :I], y[..., I:]
        y = torch.matmul(g / (1.0 + torch.exp(-g)) * u, w2.transpose(1, 2))
        dense = torch.zeros((T, E + 1), device=x.device).scatter(1, torch.where(ids < 0, E, ids).long(), w)[:, :E]
        out = (y * dense.t().unsqueeze(-1)).sum(dim=0)
    return out.to(torch.bfloat16), ids, w


def _plain_lora(st):
    x, a, b, idx = st["x"].float(), st["a"].float(), st["b"].float(), st["index"].long()
    L, R, K = a.shape
    N, M = b.shape[1], x.shape[0]
    live = torch.arange(R, device=x.device) < st["ranks"][:, None]                      # [L, R]
    a = torch.where(live.unsqueeze(-1), a, 0.0).reshape(L * R, K)
    b = torch.where(live.unsqueeze(1), b, 0.0).permute(0, 2, 1).reshape(L * R, N)
    v = torch.matmul(x, a.t()).view(M, L, R) * st["scaling"][:, None]
    mine = (torch.arange(L, device=x.device) == idx[:, None]).unsqueeze(-1)
    y = torch.matmul(torch.where(mine, v, 0.0).reshape(M, L * R), b)
    if st["base"] is not None:
        y = y + st["base"].float()
    return y.to(torch.bfloat16)


def run(state):
    case = state["case"]
    if own:
        ck = state["ck"]
        if case["op"] == "route":
            return ck.moe_route(state["logits"], state["k"], case["renormalize"], *state["slots"])
        if case["op"] == "moe":
            return ck.moe(state["x"], state["logits"], state["experts"], state["k"], case["renormalize"],
                          state["out"], *state["slots"], workspace=state["space"])
        return ck.lora_add(state["x"], state["adapters"], state["index"], base=state["base"], out=state["out"],
                           workspace=state["space"])
    if case["op"] == "route":
        return _plain_route(state["logits"], state["k"], case["renormalize"])
    return _plain_moe(state) if case["op"] == "moe" else _plain_lora(state)


# ------------------------------------------------------------- what it costs

def work(case):
    if case["op"] == "route":
        T, E, k = case["tokens"], case["experts"], case["k"]
        return dict(bytes=T * E * (2 if case["logits"] == "bf16" else 4) + 8 * T * k, flops=3 * T * E)
    if case["op"] == "moe":
        T, H, I, E, k = case["tokens"], case["hidden"], case["inter"], case["experts"], min(case["k"], case["experts"])
        used = E * (1 - (1 - k / E) ** T)  # distinct experts that T tokens choose, on average
        per = 3 * H * I / 2 + 3 * H * I / 64 * (4 if case["zeros"] else 2)
        return dict(bytes=used * per + T * H * 4 + T * E * (2 if case["logits"] == "bf16" else 4) + 8 * T * case["k"],
                    flops=6 * H * I * T * k)
    M, K, N, L = case["rows"], case["K"], case["N"], case["adapters"]
    picks = M if case["order"] == "mixed" else min(M, 2 * L) + 1
    used = 1 - (1 - (1 - case["none"]) / L) ** picks
    ranks = [_rank_of(case, l) for l in range(L)]
    rows = M * (1 - case["none"])
    return dict(bytes=rows * K * 2 + M * N * (4 if case["base"] else 2) + 4 * M + used * sum(ranks) * (K + N) * 2,
                flops=2 * rows * sum(ranks) / L * (K + N))


# ------------------------------------------------------- the definition, fp64

def _exact_route(logits, k, renormalize):
    l = logits.double().nan_to_num(nan=-INF, posinf=INF, neginf=-INF)
    T, E = l.shape
    place = torch.empty((T, E), dtype=torch.int64, device=l.device)
    lower = torch.tril(torch.ones((E, E), dtype=torch.bool, device=l.device), -1)  # [j, i]: i < j
    for t0 in range(0, T, 512):  # how many come before expert j: a larger logit, or the same at a lower index
        c = l[t0:t0 + 512]
        before = (c[:, None, :] > c[:, :, None]) | ((c[:, None, :] == c[:, :, None]) & lower)
        place[t0:t0 + 512] = before.sum(dim=2)
    ids = torch.full((T, k), -1, dtype=torch.int64, device=l.device)
    t, j = ((place < k) & (l > -INF)).nonzero(as_tuple=True)
    ids[t, place[t, j]] = j
    top = l.max(dim=1, keepdim=True).values
    p = torch.where(top == INF, (l == INF).double(), torch.exp(l - top))
    p = torch.where(l == -INF, 0.0, p)
    w = torch.where(ids >= 0, p.gather(1, ids.clamp(min=0)), 0.0)
    den = (w if renormalize else p).sum(dim=1, keepdim=True)
    return ids.to(torch.int32), torch.where(den > 0, w / den, 0.0)


def _exact_weight(packed, s, z, e):
    q = torch.empty((packed.shape[1], 2 * packed.shape[2]), dtype=torch.float64, device=packed.device)
    q[:, 0::2] = (packed[e] % 16).double() - 8
    q[:, 1::2] = torch.div(packed[e], 16, rounding_mode="floor").double() - 8
    q *= s[e].double().t().repeat_interleave(64, dim=1)
    return q if z is None else q + z[e].double().t().repeat_interleave(64, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(st["logits"], case["k"], case["renormalize"])
    if case["op"] == "moe":
        ids, w = _exact_route(st["logits"], case["k"], case["renormalize"])
        x, I = st["x"].double(), case["inter"]
        out = torch.zeros_like(x)
        for e in range(case["experts"]):
            t, slot = (ids == e).nonzero(as_tuple=True)
            if t.numel():
                y = x[t] @ _exact_weight(*st["w1"], e).t()
                h = y[:, :I] * torch.sigmoid(y[:, :I]) * y[:, I:]
                out.index_add_(0, t, (h @ _exact_weight(*st["w2"], e).t()) * w[t, slot, None])
        return out, ids, w
    out = torch.zeros((case["rows"], case["N"]), dtype=torch.float64, device=DEV)
    for l in range(case["adapters"]):
        rows, r = (st["index"] == l).nonzero().flatten(), _rank_of(case, l)
        v = st["x"][rows].double() @ st["a"][l, :r].double().t()
        out[rows] = float(st["scaling"][l]) * (v @ st["b"][l, :, :r].double().t())
    return out if st["base"] is None else out + st["base"].double()
