"""The balance loss and the gradients of combine and router in float64, with error bounds in roundings of float32 (U)."""
import torch

from tests._layer_ref import U


def balance(logits, ids, weight, offset=None, mask=None):
    """Loss, counts [S, E] and gradient with their bounds, sequence by sequence, for float64 logits on the CPU."""
    T, E = logits.shape
    k = ids.shape[1]
    offset = [0, T] if offset is None else list(offset)
    S = len(offset) - 1
    live = [mask is None or bool(mask[t]) for t in range(T)]
    count = torch.zeros(S, E, dtype=torch.int64)
    tokens = []
    for s in range(S):
        tokens.append([t for t in range(offset[s], offset[s + 1]) if live[t]])
        for t in tokens[s]:
            for e in ids[t].tolist():
                if 0 <= e < E:
                    count[s, e] += 1
    used = sum(len(t) > 0 for t in tokens)
    loss, dloss = 0.0, 0.0
    d, db = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    for s in range(S):
        n = len(tokens[s])
        if not n:
            continue
        x = logits[tokens[s]]
        f = count[s].double() / (k * n)
        top = x.amax(1, keepdim=True)
        all_out = top == -float("inf")
        e = torch.where(all_out, torch.zeros_like(x), torch.exp(x - torch.where(all_out, torch.zeros_like(top), top)))
        p = e / torch.where(all_out, torch.ones_like(top), e.sum(1, keepdim=True))
        dot = (p * f).sum(1, keepdim=True)
        # a p is off by its exponent's rounding (the distance from the maximum), expf, the sum of E terms and a division
        far = torch.where(torch.isfinite(x), top - x, torch.zeros_like(x))
        rel = U * (far + E + 32)
        worst = rel.amax(1, keepdim=True) + U * E
        factor = weight * E / (n * used)
        loss += factor * float(dot.sum())
        dloss += abs(factor) * float((dot * (worst + 8 * U)).sum())
        d[tokens[s]] = factor * p * (f - dot)
        db[tokens[s]] = abs(factor) * p * ((rel + 8 * U) * (f - dot).abs() + 4 * U * f + (worst + 4 * U) * dot) * 1.01
    return dict(loss=loss, dloss=dloss, count=count, d=d, db=db)


def combine_backward(dy, out, pair_row, w):
    """(d_w, bound, d_out, bound, rows written) for float64 dy [T, H], out [., H], w [T, k]."""
    T, k = pair_row.shape
    d_w, b = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    d_out, bo = torch.zeros_like(out), torch.zeros_like(out)
    for t in range(T):
        for j in range(k):
            r = int(pair_row[t, j])
            if r >= 0:
                d_w[t, j] = (dy[t] * out[r]).sum()
                b[t, j] = (dy.shape[1] + 1) * U * (dy[t] * out[r]).abs().sum()
                d_out[r] = w[t, j] * dy[t]
                bo[r] = U * d_out[r].abs()
    return d_w, b, d_out, bo


def route_backward(x, wr, ids, w, d_w, d_in, split):
    """Gradients of the router in float64: each with its bound. split: x is bf16, and d_x takes its operands in fp16, scaled by
    a power of two for each token of d_logits and each column of the weight that puts the largest value into [2^14, 2^15). Half
    a step of fp16 is 2^-11 of a value down to 2^-14, and 2^-25 below, which is 2^-39 of that largest value at most. So with
    a' = a (1 + d) + s, |d| <= 2^-11, |s| <= 2^-39 max|a|, and b' alike, |a' b' - a b| is at most
    (2^-10 + 2^-22) |a b| + 1.01 (|s_a| |b| + |s_b| |a|) + |s_a s_b|."""
    T, H = x.shape
    E = wr.shape[0]
    dl = torch.zeros(T, E, dtype=torch.float64) if d_in is None else d_in.clone()
    db = torch.zeros_like(dl)
    if d_w is not None:
        k = ids.shape[1]
        s = (w * d_w).sum(1, keepdim=True)
        m = (w * d_w).abs().sum(1, keepdim=True)
        c = w * (d_w - s)
        e = w * ((k + 4) * U * (d_w.abs() + m))
        for j in range(k):
            for t in range(T):
                if 0 <= ids[t, j] < E:
                    dl[t, ids[t, j]] += c[t, j]
                    db[t, ids[t, j]] += e[t, j]
        db += (k + 1) * U * (dl.abs() + db)
    part = 2.0 ** -10 + 2.0 ** -22 if split else 0.0
    d_x = dl @ wr
    bx = ((E + 2) * U + part) * ((dl.abs() + db) @ wr.abs()) + db @ wr.abs()
    if split and T:
        low = 2.0 ** -39
        sa, sb = low * (dl.abs() + db).amax(1, keepdim=True), low * wr.abs().amax(0, keepdim=True)
        bx = bx + 1.01 * (sa * wr.abs().sum(0) + sb * (dl.abs() + db).sum(1, keepdim=True)) + E * sa * sb
    d_wr = dl.T @ x
    bw = (T + 2) * U * ((dl.abs() + db).T @ x.abs()) + db.T @ x.abs()
    return dict(d_logits=(dl, db), d_x=(d_x, bx), d_w_router=(d_wr, bw),
                d_bias=(dl.sum(0), db.sum(0) + (T + 2) * U * (dl.abs() + db).sum(0)))
