"""Operators measured beside the MoE layer: grouped routing, the norms around the block, adapters.

Each case is one call as a serving program makes it between two layers.  With
``own`` false ``run`` computes the operator in elementary torch operations, in
32 bits (the router's logits and scores in 64, as its contract asks); with
``own`` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one request's next token through a 256-expert sigmoid router with groups
        dict(name="route_token", op="route", dtype="bf16", T=1, d=7168, E=256, k="8", k_max=8, score="sigmoid",
             groups=8, keep=4, rule="top2", renorm=True, scale=2.5, masked=0),
        # a decode batch of requests with their own budgets
        dict(name="route_decode", op="route", dtype="bf16", T=128, d=7168, E=256, k="4 8", k_max=8, score="sigmoid",
             groups=8, keep=4, rule="top2", renorm=True, scale=2.5, masked=0),
        # a prefill batch of the same layer
        dict(name="route_prefill", op="route", dtype="bf16", T=4096, d=7168, E=256, k="4 8", k_max=8,
             score="sigmoid", groups=8, keep=4, rule="top2", renorm=True, scale=2.5, masked=0),
        # softmax scores without renormalisation, an odd batch in float32, some experts out of service
        dict(name="route_softmax_f32", op="route", dtype="f32", T=777, d=2048, E=96, k="0 1 3 6", k_max=6,
             score="softmax", groups=3, keep=2, rule="max", renorm=False, scale=1.0, masked=5),
        # residual add and the norm before the block, one token
        dict(name="norm_token", op="norm", dtype="bf16", T=1, d=7168, kind="rms", post=False, gate="none",
             alpha=1.0, offset=0.0, bias=False),
        # norms on both sides of a block with a channel gate and a residual scale, prefill
        dict(name="norm_prefill", op="norm", dtype="bf16", T=8192, d=2048, kind="rms", post=True, gate="channel",
             alpha=0.5, offset=1.0, bias=False),
        # layer norms with bias and a gate per token at a width that no vector load divides
        dict(name="norm_layer_odd", op="norm", dtype="f32", T=1021, d=1531, kind="layer", post=True, gate="token",
             alpha=1.0, offset=0.0, bias=True),
        # the layer's combine with both norms and the residual, decode
        dict(name="combine_decode", op="combine", dtype="bf16", T=128, d=7168, k="4 8", k_max=8, shared=True,
             kind="rms", post=True, gate="none", alpha=1.0, offset=0.0, bias=False),
        # the same for a prefill batch
        dict(name="combine_prefill", op="combine", dtype="bf16", T=4096, d=7168, k="4 8", k_max=8, shared=True,
             kind="rms", post=True, gate="channel", alpha=1.0, offset=0.0, bias=False),
        # a decode batch, a token per request, each with one of 32 adapters on a dense down projection
        dict(name="adapt_decode", op="adapt", dtype="bf16", T=128, K=2048, N=7168, R=16, L=32, G=1, k_max=1,
             runs=False),
        # a prefill batch of few requests, each a run of tokens
        dict(name="adapt_prefill", op="adapt", dtype="bf16", T=4096, K=2048, N=7168, R=32, L=8, G=1, k_max=1,
             runs=True),
        # adapters of every expert's down projection over the permuted rows of a decode batch
        dict(name="adapt_experts", op="adapt", dtype="bf16", T=256, K=768, N=2048, R=16, L=4, G=128, k_max=8,
             runs=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "norm", "combine", "adapt"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(max(2, 8 // groups), 320 // groups)
        keep = rng.randint(max(1, groups // 2), groups)
        d = 128 * rng.randint(2, 56)
        T = _log_int(rng, 1, min(4096, 4096 * 256 // E))
        k_max = rng.randint(1, min(12, keep * (E // groups)))
        return dict(op=op, dtype=dtype, T=T, d=d, E=E, k="%d %d" % (rng.randint(0, k_max), k_max), k_max=k_max,
                    score=rng.choice(["sigmoid", "softmax"]), groups=groups, keep=keep,
                    rule=rng.choice(["top2", "max"]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), masked=rng.choice([0, 0, min(3, E // 4)]))
    if op == "norm":
        d = rng.choice([_log_int(rng, 64, 8192), 8 * _log_int(rng, 16, 1024)])
        T = _log_int(rng, 1, min(8192, 8192 * 2048 // d))
        return dict(op=op, dtype=dtype, T=T, d=d, kind=rng.choice(["rms", "layer"]), post=rng.random() < 0.6,
                    gate=rng.choice(["none", "channel", "token", "full"]), alpha=rng.choice([1.0, 0.5, 0.22]),
                    offset=rng.choice([0.0, 1.0]), bias=rng.random() < 0.5)
    if op == "combine":
        d = 128 * rng.randint(2, 56)
        T = _log_int(rng, 1, min(4096, 2048 * 7168 // d))
        k_max = rng.randint(1, 10)
        return dict(op=op, dtype=dtype, T=T, d=d, k="%d %d" % (rng.randint(0, k_max), k_max), k_max=k_max,
                    shared=rng.random() < 0.5, kind=rng.choice(["rms", "layer"]), post=rng.random() < 0.5,
                    gate=rng.choice(["none", "channel", "token", "full"]), alpha=rng.choice([1.0, 0.5]),
                    offset=rng.choice([0.0, 1.0]), bias=rng.random() < 0.3)
    R = rng.choice([8, 16, 24, 32, 64])
    if rng.random() < 0.6:  # a dense projection
        K, N = 8 * rng.randint(16, 512), 8 * rng.randint(16, 896)
        T = _log_int(rng, 1, min(4096, 2048 * 7168 // max(K, N)))
        L = rng.randint(1, max(1, min(32, 256 * 1024 // (R * max(T, 128)))))
        return dict(op=op, dtype=dtype, T=T, K=K, N=N, R=R, L=L, G=1, k_max=1, runs=rng.random() < 0.5)
    K, N = 128 * rng.randint(1, 8), 128 * rng.randint(1, 16)
    k_max = rng.randint(1, 8)
    T = _log_int(rng, 1, 1024 // k_max)
    return dict(op=op, dtype=dtype, T=T, K=K, N=N, R=min(R, 32), L=rng.randint(1, 6), G=rng.randint(8, 128),
                k_max=k_max, runs=rng.random() < 0.5)


def _choices(c):
    """The budgets that requests of the case ask for."""
    return [int(v) for v in c["k"].split()]


def work(case):
    c, s = case, 2 if case["dtype"] == "bf16" else 4
    T = c["T"]
    if c["op"] == "route":
        A = T * sum(_choices(c)) / len(_choices(c))
        return {"bytes": T * c["d"] * s + c["E"] * c["d"] * s + c["E"] * 4 + T * 8 + A * 8,
                "flops": 2 * T * c["E"] * c["d"]}
    if c["op"] in ("norm", "combine"):
        d = c["d"]
        vec = d * s * ((1 + c["bias"]) * (1 + c["post"]) + (c["gate"] == "channel"))
        vec += {"token": T, "full": T * d}.get(c["gate"], 0) * s
        if c["op"] == "norm":
            return {"bytes": 4 * T * d * s + vec, "flops": 10 * T * d}
        A = T * sum(_choices(c)) / len(_choices(c))
        return {"bytes": A * d * s + (3 + c["shared"]) * T * d * s + vec + A * 8 + T * 4,
                "flops": 2 * A * d + 10 * T * d}
    # adapters: x and y once, the matrices that some row uses once
    rows = T * (1 + c["k_max"]) / 2 if c["G"] > 1 else T
    pairs = c["G"] * c["L"] * (1 - (1 - 1 / (c["G"] * c["L"])) ** (0.9 * rows))
    return {"bytes": rows * (c["K"] + 2 * c["N"]) * s + pairs * c["R"] * (c["K"] + c["N"]) * s + rows * 8,
            "flops": 2 * 0.9 * rows * c["R"] * (c["K"] + c["N"])}


# -------------------------------------------------------------------- inputs

def _budgets(c, gen):
    pick = torch.tensor(_choices(c), dtype=torch.int32, device="cuda")
    return pick[torch.randint(0, len(pick), (c["T"],), generator=gen, device="cuda")]


def _offsets(k):
    off = torch.zeros(k.numel() + 1, dtype=torch.int32, device=k.device)
    off[1:] = torch.cumsum(k, 0)
    return off


def prepare(case, seed):
    c, dt = case, _DT[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *n, std=1.0: (torch.randn(*n, generator=gen, device="cuda") * std).to(dt)
    T = c["T"]
    s = {"c": c}
    if c["op"] == "route":
        E, A = c["E"], max(T * c["k_max"], 1)
        s["x"], s["w"] = randn(T, c["d"]), randn(E, c["d"], std=c["d"] ** -0.5)
        s["bias"] = (torch.rand(E, generator=gen, device="cuda") - 0.5) * (0.1 if c["score"] == "sigmoid" else 0.5 / E)
        if c["masked"]:
            s["bias"][torch.randperm(E, generator=gen, device="cuda")[:c["masked"]]] = -math.inf
        s["k"] = _budgets(c, gen)
        s["tok_off"] = torch.zeros(T + 1, dtype=torch.int32, device="cuda")
        s["ids"] = torch.full((A,), -1, dtype=torch.int32, device="cuda")
        s["wts"] = torch.zeros(A, device="cuda")
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    if c["op"] in ("norm", "combine"):
        d = c["d"]
        s["resid"] = randn(T, d)
        for name in ("post", "pre"):
            s[name + "_w"] = randn(d, std=0.1) + (1 - c["offset"])
            s[name + "_b"] = randn(d, std=0.1) if c["bias"] else None
        shape = {"none": None, "channel": (d,), "token": (T,), "full": (T, d)}[c["gate"]]
        s["gate"] = randn(*shape, std=0.5) if shape else None
        s["resid_out"], s["x_out"] = torch.empty(T, d, dtype=dt, device="cuda"), torch.empty(T, d, dtype=dt, device="cuda")
        if c["op"] == "norm":
            s["y"] = randn(T, d)
            return s
        A = max(T * c["k_max"], 1)
        k = _budgets(c, gen)
        s["tok_off"] = _offsets(k)
        s["y_perm"] = randn(A, d)
        # the rows of the A assignments, in some order of the first A rows
        n = int(k.sum())
        s["inv_perm"] = torch.full((A,), -1, dtype=torch.int32, device="cuda")
        s["inv_perm"][:n] = torch.randperm(n, generator=gen, device="cuda").int()
        s["topk_w"] = torch.rand(A, generator=gen, device="cuda") / max(c["k_max"], 1)
        s["y_shared"] = randn(T, d) if c["shared"] else None
        return s
    G, L, R, K, N = c["G"], c["L"], c["R"], c["K"], c["N"]
    rows = T * c["k_max"]
    s["a"], s["b"] = randn(L, G, R, K, std=K ** -0.5), randn(L, G, N, R, std=R ** -0.5)
    s["ranks"] = torch.full((L,), R, dtype=torch.int32, device="cuda")
    s["ranks"][L // 2:] = max(1, R // 2)  # adapters of two ranks in one stack
    s["scales"] = torch.rand(L, generator=gen, device="cuda") + 0.5
    if c["runs"]:  # tokens of a request follow each other
        edges = torch.sort(torch.randint(0, T + 1, (max(1, L - 1),), generator=gen, device="cuda")).values
        ids = torch.bucketize(torch.arange(T, device="cuda"), edges, right=True) % L
    else:
        ids = torch.randint(0, L, (T,), generator=gen, device="cuda")
        ids[torch.rand(T, generator=gen, device="cuda") < 0.1] = -1  # requests of the base model
    s["ids"] = ids.int()
    s["row_tok"] = s["expert_off"] = None
    if G > 1:  # permuted rows, as the dispatch leaves them: by expert, then by token
        k = torch.randint(1, c["k_max"] + 1, (T,), generator=gen, device="cuda").clamp(max=G)
        order = torch.rand(T, G, generator=gen, device="cuda").argsort(1)
        taken = torch.zeros(T, G, dtype=torch.bool, device="cuda")
        taken.scatter_(1, order, torch.arange(G, device="cuda")[None] < k[:, None])
        tok = taken.t().nonzero()[:, 1].int()
        s["row_tok"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
        s["row_tok"][:tok.numel()] = tok
        s["expert_off"] = _offsets(taken.sum(0).int())
    s["x"], s["y"] = randn(rows, K), randn(rows, N)
    s["out"] = torch.zeros(rows, N, dtype=dt, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms

def _plain_route(s):
    c = s["c"]
    T, E, g = c["T"], c["E"], c["groups"]
    dev = s["x"].device
    l = (s["x"].double() @ s["w"].double().t()).float().double()
    score = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
    key = score + s["bias"].double()
    live = key > -math.inf
    # value of a group: its largest key, or the sum of its two largest, of the experts in service
    by = torch.where(live, key, -math.inf).view(T, g, E // g).sort(2, descending=True).values
    value = by[..., 0]
    if c["rule"] == "top2" and E // g > 1:
        value = value + torch.where(by[..., 1] > -math.inf, by[..., 1], 0.0)
    rank = torch.sort(value, dim=1, descending=True, stable=True).indices
    kept = torch.zeros(T, g, dtype=torch.bool, device=dev).scatter_(
        1, rank, (torch.arange(g, device=dev) < c["keep"]).expand(T, g).contiguous())
    live &= kept.repeat_interleave(E // g, 1)
    order = torch.sort(torch.where(live, key, -math.inf), dim=1, descending=True, stable=True).indices[:, :c["k_max"]]
    k = s["k"].long()
    use = torch.arange(c["k_max"], device=dev) < k[:, None]
    ok = use & live.gather(1, order)
    w = torch.where(ok, score.gather(1, order), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    off = _offsets(s["k"])
    # token t's entries from off[t] on; what is not used goes to a place behind the last one
    at = torch.where(use, off[:-1, None].long() + torch.arange(c["k_max"], device=dev), s["ids"].numel())
    ids = torch.cat([s["ids"], s["ids"][:1]]).scatter(0, at.flatten(), torch.where(ok, order, -1).int().flatten())
    wts = torch.cat([s["wts"], s["wts"][:1]]).scatter(0, at.flatten(), (w * c["scale"]).float().flatten())
    return off, ids[:-1], wts[:-1]


def _plain_norm(v, w, b, c):
    if c["kind"] == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * (w.float() + c["offset"])
    return v if b is None else v + b.float()


def _plain_chain(s, y):
    c = s["c"]
    if c["post"]:
        y = _plain_norm(y, s["post_w"], s["post_b"], c)
    if s["gate"] is not None:
        y = y * (s["gate"].float()[:, None] if c["gate"] == "token" else s["gate"].float())
    r = s["resid"].float() + c["alpha"] * y
    x = _plain_norm(r, s["pre_w"], s["pre_b"], c)
    return r.to(s["resid"].dtype), x.to(s["resid"].dtype)


def _plain_combine(s):
    c = s["c"]
    off, dev = s["tok_off"].long(), s["resid"].device
    j = torch.arange(c["k_max"], device=dev)
    at = (off[:-1, None] + j).clamp(max=s["inv_perm"].numel() - 1)
    use = j < (off[1:] - off[:-1])[:, None]
    w = torch.where(use, s["topk_w"][at], 0.0)
    rows = torch.where(use, s["inv_perm"][at].long(), 0)
    y = torch.bmm(w[:, None], s["y_perm"][rows].float())[:, 0]
    return y if s["y_shared"] is None else y + s["y_shared"].float()


def _plain_adapt(s):
    c = s["c"]
    T, G, L, R, rows = c["T"], c["G"], c["L"], c["R"], s["x"].shape[0]
    dev = s["x"].device
    r = torch.arange(rows, device=dev)
    tok = r if s["row_tok"] is None else s["row_tok"].long()
    ad = s["ids"].long()[tok]
    has = (ad >= 0) & (ad < L)
    one = ad.clamp(0, L - 1)
    live = torch.arange(R, device=dev) < s["ranks"][:, None]  # [L, R]
    factor = torch.where(has, s["scales"][one], 0.0)[:, None]
    x = s["x"].float()
    if G == 1:  # the product with every adapter, then each row's own
        mine = (torch.arange(L, device=dev) == one[:, None])[:, :, None] & live
        v = torch.where(mine, (x @ s["a"].float().view(L * R, -1).t()).view(rows, L, R), 0.0) * factor[..., None]
        delta = v.view(rows, L * R) @ s["b"][:, 0].float().transpose(1, 2).reshape(L * R, -1)
        written = torch.ones(rows, 1, dtype=torch.bool, device=dev)
    else:
        g = torch.bucketize(r, s["expert_off"][1:].long(), right=True).clamp(max=G - 1)
        v = torch.where(live[one], torch.bmm(s["a"][one, g].float(), x[..., None])[..., 0], 0.0) * factor
        delta = torch.bmm(s["b"][one, g].float(), v[..., None])[..., 0]
        written = (r < s["expert_off"][-1])[:, None]
    return torch.where(written, (s["y"].float() + delta).to(s["y"].dtype), s["out"])


# ----------------------------------------------------------------------- run

def _handle(s):
    """What a program keeps between calls: descriptors and workspaces."""
    if "handle" in s:
        return s["handle"]
    import mixture_experts_layer_token_amd as moe
    c = s["c"]
    dt, T = _DT[c["dtype"]], c["T"]
    if c["op"] == "route":
        desc = moe.make_desc(T, c["d"], c["E"], 128, c["k_max"], dtype=dt, routed_scale=c["scale"])
        rule = moe.make_route_rule(score=c["score"], n_group=c["groups"], topk_group=c["keep"],
                                   group_score=c["rule"], renorm=c["renorm"])
        s["handle"] = (moe, desc, rule, moe.alloc_workspace(desc, moe.MOE_OP_ROUTE_GROUPED))
    elif c["op"] in ("norm", "combine"):
        nd = moe.make_norm_desc(T, c["d"], dtype=dt, kind=c["kind"], eps=1e-6, alpha=c["alpha"],
                                w_offset=c["offset"], gate=c["gate"], post=c["post"])
        desc = moe.make_desc(T, c["d"], c["k_max"], 128, c["k_max"], dtype=dt) if c["op"] == "combine" else None
        s["handle"] = (moe, desc, nd)
    else:
        ad = moe.make_adapter_desc(T, s["x"].shape[0], c["K"], c["N"], c["R"], c["L"], c["G"], dtype=dt)
        s["handle"] = (moe, ad, moe.alloc_adapt_workspace(ad))
    return s["handle"]


def _own(s):
    c, h = s["c"], _handle(s)
    moe = h[0]
    if c["op"] == "route":
        moe.moe_route_grouped(h[1], h[2], s["x"], s["w"], None, s["bias"], s["k"], s["tok_off"], s["ids"], s["wts"],
                              s["status"], h[3])
        return s["tok_off"], s["ids"], s["wts"]
    if c["op"] == "norm":
        moe.moe_norm(h[2], s["y"], s["resid"], s["post_w"] if c["post"] else None, s["post_b"] if c["post"] else None,
                     s["gate"], s["pre_w"], s["pre_b"], s["resid_out"], s["x_out"])
        return s["resid_out"], s["x_out"]
    if c["op"] == "combine":
        moe.moe_combine_norm(h[1], h[2], s["y_perm"], s["y_shared"], s["tok_off"], s["topk_w"], s["inv_perm"],
                             s["resid"], s["post_w"] if c["post"] else None, s["post_b"] if c["post"] else None,
                             s["gate"], s["pre_w"], s["pre_b"], s["resid_out"], s["x_out"])
        return s["resid_out"], s["x_out"]
    moe.moe_adapt(h[1], s["x"], None, s["a"], s["b"], s["ranks"], s["scales"], s["ids"], s["row_tok"],
                  s["expert_off"], s["y"], s["out"], h[2])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    op = state["c"]["op"]
    if op == "route":
        return _plain_route(state)
    if op == "norm":
        return _plain_chain(state, state["y"].float())
    if op == "combine":
        return _plain_chain(state, _plain_combine(state))
    return _plain_adapt(state)


# --------------------------------------------------- the definitions, 64 bits

def _host(t):
    return None if t is None else (t.double() if t.is_floating_point() else t.long()).cpu().numpy()


def _exact_route(c, h):
    T, E, per = c["T"], c["E"], c["E"] // c["groups"]
    logit = (h["x"] @ h["w"].T).astype(np.float32).astype(np.float64)
    ids, wts = h["ids"].copy(), h["wts"].copy()
    at = 0
    for t in range(T):
        l = logit[t]
        if c["score"] == "sigmoid":
            p = 1.0 / (1.0 + np.exp(-l))
        else:
            p = np.exp(l - l.max())
            p /= p.sum()
        key = p + h["bias"]
        pool = [e for e in range(E) if key[e] > -np.inf]
        if c["groups"] > 1:
            value = {}
            for g in sorted({e // per for e in pool}):
                top = np.sort(key[[e for e in pool if e // per == g]])[::-1]
                value[g] = top[:2 if c["rule"] == "top2" else 1].sum()
            kept = set(sorted(value, key=lambda g: (-value[g], g))[:c["keep"]])
            pool = [e for e in pool if e // per in kept]
        best = sorted(pool, key=lambda e: (-key[e], e))[:int(h["k"][t])]
        total = p[best].sum() if c["renorm"] else 1.0
        for j in range(int(h["k"][t])):
            ids[at + j] = best[j] if j < len(best) else -1
            wts[at + j] = c["scale"] * (p[best[j]] / total if total > 0 else 0.0) if j < len(best) else 0.0
        at += int(h["k"][t])
    return np.concatenate([[0], np.cumsum(h["k"])]).astype(np.int32), ids.astype(np.int32), wts


def _exact_norm(v, w, b, c):
    mean = v.mean(axis=1, keepdims=True) if c["kind"] == "layer" else 0.0
    v = (v - mean) / np.sqrt(np.square(v - mean).mean(axis=1, keepdims=True) + 1e-6) * (c["offset"] + w)
    return v + (0.0 if b is None else b)


def _exact_chain(c, h):
    if c["op"] == "norm":
        y = h["y"]
    else:
        y = np.zeros_like(h["resid"]) if h["y_shared"] is None else h["y_shared"].copy()
        off = h["tok_off"]
        for j in range(c["k_max"]):
            t = np.nonzero(off[1:] - off[:-1] > j)[0]
            y[t] += h["topk_w"][off[t] + j, None] * h["y_perm"][h["inv_perm"][off[t] + j]]
    if c["post"]:
        y = _exact_norm(y, h["post_w"], h["post_b"], c)
    if c["gate"] != "none":
        y = y * (h["gate"][:, None] if c["gate"] == "token" else h["gate"])
    r = h["resid"] + c["alpha"] * y
    return r, _exact_norm(r, h["pre_w"], h["pre_b"], c)


def _exact_adapt(c, h):
    off = np.array([0, c["T"]]) if c["G"] == 1 else h["expert_off"]
    out = h["out"].copy()
    for g in range(c["G"]):
        rows = np.arange(off[g], off[g + 1])
        owner = h["ids"][rows if h["row_tok"] is None else h["row_tok"][rows]]
        out[rows] = h["y"][rows]
        for ad in np.unique(owner[owner >= 0]):
            at, r = rows[owner == ad], h["ranks"][ad]
            out[at] += h["scales"][ad] * (h["x"][at] @ h["a"][ad, g, :r].T) @ h["b"][ad, g, :, :r].T
    return out


def exact(case, seed):
    state = prepare(case, seed)
    h = {name: _host(t) for name, t in state.items() if t is None or isinstance(t, torch.Tensor)}
    if case["op"] == "route":
        return _exact_route(case, h)
    if case["op"] in ("norm", "combine"):
        return _exact_chain(case, h)
    return _exact_adapt(case, h)
