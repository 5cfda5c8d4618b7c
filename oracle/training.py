"""Float64 restatement of the training-step operators: embedding lookup and
gradient, matrix products grouped by expert, and distillation from a teacher's
top logits (with the values the library defines for masked rows)."""
import numpy as np


def embedding_lookup(W, ids, scale=1.0):
    W, ids = np.asarray(W, np.float64), np.asarray(ids)
    out = np.zeros((len(ids), W.shape[1]))
    ok = (ids >= 0) & (ids < W.shape[0])
    out[ok] = scale * W[ids[ok]]
    return out


def embedding_grad(dY, ids, vocab, scale=1.0, start=None):
    dY = np.asarray(dY, np.float64)
    out = np.zeros((vocab, dY.shape[1])) if start is None else np.array(start, np.float64)
    ids = np.asarray(ids)
    keep = (ids >= 0) & (ids < vocab)
    np.add.at(out, ids[keep], scale * dY[keep])
    return out


def _groups(offsets):
    return [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(len(offsets) - 1)]


def expert_linear(X, W, offsets):
    X, W = np.asarray(X, np.float64), np.asarray(W, np.float64)
    Y = np.zeros((X.shape[0], W.shape[1]))
    for e, a, b in _groups(offsets):
        Y[a:b] = X[a:b] @ W[e].T
    return Y


def expert_linear_dgrad(dY, W, offsets):
    dY, W = np.asarray(dY, np.float64), np.asarray(W, np.float64)
    dX = np.zeros((dY.shape[0], W.shape[2]))
    for e, a, b in _groups(offsets):
        dX[a:b] = dY[a:b] @ W[e]
    return dX


def expert_linear_wgrad(dY, X, offsets, start=None):
    dY, X = np.asarray(dY, np.float64), np.asarray(X, np.float64)
    dW = np.zeros((len(offsets) - 1, dY.shape[1], X.shape[1])) if start is None else np.array(start, np.float64)
    for e, a, b in _groups(offsets):
        dW[e] += dY[a:b].T @ X[a:b]
    return dW


def distill_topk(logits, idx, teacher, temperature=1.0, row_weight=None, grad_scale=1.0):
    """(loss per row, gradient by the logits, q, z) with z = (s - max s) / T."""
    S, t = np.asarray(logits, np.float64), np.asarray(teacher, np.float64)
    n, V = S.shape
    T = float(temperature)
    w = np.ones(n) if row_weight is None else np.asarray(row_weight, np.float64)
    loss, grad, Q, Z = np.zeros(n), np.zeros((n, V)), np.zeros((n, V)), np.zeros((n, V))
    with np.errstate(all="ignore"):
        for r in range(n):
            keep = [(int(i), x) for i, x in zip(idx[r], t[r]) if 0 <= i < V and x != -np.inf]
            if w[r] == 0 or not keep:
                continue
            at = np.array([i for i, _ in keep])
            tt = np.array([x for _, x in keep])
            tt = (tt - tt.max()) / T
            p = np.exp(tt) / np.exp(tt).sum()
            if np.all(S[r] == -np.inf):
                q, logq = np.zeros(V), np.full(V, -np.inf)
            else:
                Z[r] = (S[r] - S[r].max()) / T
                log_z = np.log(np.exp(Z[r]).sum())
                logq = Z[r] - log_z
                q = np.exp(logq)
            terms = [pk * (np.log(pk) - logq[i]) for pk, i in zip(p, at) if pk != 0]
            loss[r] = w[r] * T * T * np.sum(terms)
            g = q.copy()
            np.add.at(g, at, -p)
            grad[r] = grad_scale * w[r] * T * g
            Q[r] = q
    return loss, grad, Q, Z
