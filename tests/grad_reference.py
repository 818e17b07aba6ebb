"""The training operators in float64 on the CPU, written from their
formulas one token or one expert at a time, and the routing they start
from.  Nothing here uses the package."""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def route(logits, k, capacity, choice):
    """Routing of float64 logits [T, E] as the layer defines it: a dict of
    topk_idx, topk_w, slot_of (lists of tensors' types: int64 / float64),
    slot_token, offsets, counts, f."""
    T, E = logits.shape
    p = torch.softmax(logits, 1)
    if choice:
        k, C = E, capacity
        idx = torch.arange(E).expand(T, E).contiguous()
        w = p.clone()
        slot = torch.full((T, E), -1)
        token = torch.full((E * C,), -1)
        for e in range(E):
            order = torch.sort(logits[:, e], descending=True, stable=True)[1]
            for r, t in enumerate(sorted(order[:C].tolist())):
                slot[t, e] = e * C + r
                token[e * C + r] = t
        counts = torch.full((E,), T)
        kept = torch.full((E,), C)
    else:
        order = torch.sort(logits, dim=1, descending=True, stable=True)[1]
        idx = order[:, :k].contiguous()
        w = torch.softmax(torch.gather(logits, 1, idx), 1)
        counts = torch.bincount(idx.reshape(-1), minlength=E)
        kept = counts if capacity < 0 else counts.clamp(max=capacity)
        start = (kept.cumsum(0) - kept).tolist()
        room, used = kept.tolist(), [0] * E
        slot = torch.full((T, k), -1)
        token = torch.full((T * k,), -1)
        for t in range(T):
            for j in range(k):
                e = int(idx[t, j])
                if used[e] < room[e]:
                    slot[t, j] = start[e] + used[e]
                    token[start[e] + used[e]] = t
                    used[e] += 1
    offsets = torch.zeros(E + 1, dtype=torch.int64)
    offsets[1:] = kept.cumsum(0)
    return {"topk_idx": idx, "topk_w": w, "slot_of": slot,
            "slot_token": token, "offsets": offsets, "counts": counts,
            "kept": kept, "f": counts.double() / (T * slot.shape[1])}


def dispatch(r, x, n_shared, fill):
    """Expert-sorted rows; rows in no use hold ``fill``."""
    rows = torch.full((r["slot_token"].numel(), x.shape[1]), fill, dtype=F64)
    for t in range(x.shape[0]):
        for s in r["slot_of"][t].tolist():
            if s >= 0:
                rows[s] = x[t]
    return torch.cat([rows, x]) if n_shared else rows


def combine(r, ys, T, n_shared, weighted=True):
    R = r["slot_token"].numel()
    y = torch.zeros(T, ys.shape[1], dtype=F64)
    for t in range(T):
        for j, s in enumerate(r["slot_of"][t].tolist()):
            if s >= 0:
                y[t] += (r["topk_w"][t, j] if weighted else 1.0) * ys[s]
    return y + ys[R:] if n_shared else y


def combine_grad(r, dy, ys, n_shared, fill):
    T, k = r["slot_of"].shape
    rows = torch.full((r["slot_token"].numel(), dy.shape[1]), fill, dtype=F64)
    dw = torch.zeros(T, k, dtype=F64)
    for t in range(T):
        for j, s in enumerate(r["slot_of"][t].tolist()):
            if s >= 0:
                rows[s] = r["topk_w"][t, j] * dy[t]
                dw[t, j] = (dy[t] * ys[s]).sum()
    return (torch.cat([rows, dy]) if n_shared else rows), dw


def activation(act, z, u):
    if act == "gelu":
        return z * torch.special.ndtr(z)
    a = z * torch.sigmoid(z)
    return a * u if act == "swiglu" else a


def expert(act, x, w, shared=False):
    """One expert (or the shared one) on rows x, from a dict of weights."""
    s = "s" if shared else ""

    def lin(v, n):
        b = w.get("b" + s + n)
        return v @ w["w" + s + n].t() + (0 if b is None else b)

    z = lin(x, "1")
    u = lin(x, "3") if act == "swiglu" else None
    return lin(activation(act, z, u), "2")


def loss(w, x, dy, r, act, choice, n_shared, alpha, aux, z):
    """sum dy * y + aux * l_aux + z * z-loss, differentiable in x and the
    weights, the selection and the counts held (float64 autograd)."""
    T, E = x.shape[0], w["w_router"].shape[0]
    logits = x @ w["w_router"].t()
    if w.get("b_router") is not None:
        logits = logits + w["b_router"]
    if w.get("expert_bias") is not None:
        logits = logits - w["expert_bias"]
    p = torch.softmax(logits, 1)
    if choice:
        rw = p
    else:
        rw = torch.softmax(torch.gather(logits, 1, r["topk_idx"]), 1)
    y = torch.zeros(T, x.shape[1], dtype=F64)
    for e in range(E):
        t, j = ((r["topk_idx"] == e) & (r["slot_of"] >= 0)) \
            .nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        one = {n: (v[e] if n[1:] in ("1", "2", "3") and v is not None else v)
               for n, v in w.items()}
        y = y.index_add(0, t, rw[t, j][:, None] * expert(act, x[t], one))
    if n_shared:
        y = y + expert(act, x, w, shared=True)
    l_aux = alpha * E * (r["f"] * p.mean(0)).sum()
    zl = torch.logsumexp(logits, 1).square().mean()
    return (dy * y).sum() + aux * l_aux + z * zl


def router_loss(w, x, dw, r, choice, alpha, aux, z):
    """sum dw * topk_w + the losses, differentiable."""
    E = w["w_router"].shape[0]
    logits = x @ w["w_router"].t()
    if w.get("b_router") is not None:
        logits = logits + w["b_router"]
    if w.get("expert_bias") is not None:
        logits = logits - w["expert_bias"]
    p = torch.softmax(logits, 1)
    rw = p if choice else torch.softmax(
        torch.gather(logits, 1, r["topk_idx"]), 1)
    l_aux = alpha * E * (r["f"] * p.mean(0)).sum()
    zl = torch.logsumexp(logits, 1).square().mean()
    return (dw * rw).sum() + aux * l_aux + z * zl


def clip(tensors, max_norm):
    norm = math.sqrt(math.fsum(float(t.double().square().sum())
                               for t in tensors))
    f = min(1.0, max_norm / (norm + 1e-6))
    return norm, [t.double() * f for t in tensors]
