"""CPU oracle of the operators around the MoE layer: grouped routing, the norms
before and behind the block, per-request low-rank adapters (numpy, float64).

TEST INFRASTRUCTURE ONLY, like moe_oracle.py.  Plain definitions, token by token
or row by row; pinned by tests/test_block_pins.py against closed forms, torch's
float64 layer norm, the plain router's oracle and merged weight matrices.
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import router_logits


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def expert_scores(logits, score: str) -> np.ndarray:
    """sigmoid or softmax of float32 logits [T, E], in float64."""
    l = _f64(logits)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        p = np.exp(l - l.max(axis=1, keepdims=True))
        return p / p.sum(axis=1, keepdims=True)


def group_values(keys, n_group: int, group_score: str) -> np.ndarray:
    """Value of each group of one token's keys [E] (-inf: no expert in service)."""
    out = []
    for part in np.split(_f64(keys), n_group):
        best = np.sort(part[part > -np.inf])[::-1]  # NaN compares false
        n = 2 if group_score == "top2" else 1
        out.append(best[:n].sum() if best.size else -np.inf)
    return np.array(out)


def route_grouped(x, w_router, router_bias, select_bias, budgets, *, score: str, n_group: int = 1,
                  topk_group: int = 1, group_score: str = "top2", renorm: bool = True, scale: float = 1.0):
    """budgets: the executed k_t.  Returns dict(tok_off, ids, w, keys)."""
    l = router_logits(x, w_router, router_bias)
    s = expert_scores(l, score)
    c = s if select_bias is None else s + _f64(select_bias)[None, :]
    E = l.shape[1]
    ids, w = [], []
    for t, k in enumerate(np.asarray(budgets, dtype=np.int64)):
        val = group_values(c[t], n_group, group_score)
        kept = np.argsort(-val, kind="stable")[:topk_group]
        pool = [e for e in range(E) if c[t, e] > -np.inf and e // (E // n_group) in kept]
        best = sorted(pool, key=lambda e: (-c[t, e], e))[:k]
        p = s[t, best]
        total = p.sum() if renorm else 1.0
        ids += best + [-1] * (int(k) - len(best))
        w += [scale * v / total if total > 0 else 0.0 for v in p] + [0.0] * (int(k) - len(best))
    off = np.concatenate([[0], np.cumsum(np.asarray(budgets, dtype=np.int64))])
    return dict(tok_off=off, ids=np.array(ids, dtype=np.int64), w=np.array(w), keys=c)


def norm(v, w=None, b=None, *, kind: str = "rms", eps: float = 1e-6, w_offset: float = 0.0) -> np.ndarray:
    v = _f64(v)
    if kind == "layer":
        v = v - v.mean(axis=-1, keepdims=True)
    o = v / np.sqrt((v * v).mean(axis=-1, keepdims=True) + eps)
    if w is not None:
        o = o * (w_offset + _f64(w))
    return o if b is None else o + _f64(b)


def norm_chain(y, resid, *, post=None, gate=None, pre=None, alpha: float = 1.0, **kw):
    """post, pre: (weight, bias) or None for no norm.  gate: broadcastable to [T, d].
    Returns (r, x); x is None without pre."""
    r = 0.0 if resid is None else _f64(resid)
    if y is not None:
        p = _f64(y) if post is None else norm(y, *post, **kw)
        r = r + alpha * (p if gate is None else _f64(gate) * p)
    return r, None if pre is None else norm(r, *pre, **kw)


def combine(y_perm, y_shared, tok_off, w, inv_perm, T: int, d: int) -> np.ndarray:
    out = np.zeros((T, d)) if y_shared is None else _f64(y_shared).copy()
    for t in range(T):
        for j in range(int(tok_off[t]), int(tok_off[t + 1])):
            if inv_perm[j] >= 0:
                out[t] += float(w[j]) * _f64(y_perm[inv_perm[j]])
    return out


def adapt(y, x, a, b, adapter_ids, *, ranks=None, scales=None, row_tok=None, x_rows=None, expert_off=None) -> np.ndarray:
    """Rows from expert_off[-1] on keep y."""
    out = _f64(y).copy()
    L, G, R, _ = a.shape
    n = len(out) if expert_off is None else int(expert_off[-1])
    for r in range(n):
        tok = r if row_tok is None else int(row_tok[r])
        xr = r if x_rows is None else int(x_rows[r])
        if not 0 <= tok < len(adapter_ids) or not 0 <= xr < len(x) or not 0 <= adapter_ids[tok] < L:
            continue
        i = int(adapter_ids[tok])
        g = 0 if expert_off is None else int(np.searchsorted(expert_off, r, side="right")) - 1
        k = R if ranks is None else int(np.clip(ranks[i], 0, R))
        v = _f64(a[i, g, :k]) @ _f64(x[xr])
        out[r] += (1.0 if scales is None else float(scales[i])) * (_f64(b[i, g, :, :k]) @ v)
    return out
