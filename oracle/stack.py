"""Oracle of what a stack needs around its layers, in fp64 NumPy: the residual norm, the log
probabilities of a row of logits and the divergence from a teacher's entries, with their gradients.

Written from the definitions, row by row where that is plainer.
"""

import numpy as np


def add_norm(h, w, eps):
    """The norm of rows h (already added and rounded)."""
    return h / np.sqrt(np.mean(h * h, -1, keepdims=True) + eps) * w


def add_norm_backward(h, w, eps, dy, d_res):
    """(dh, dw)."""
    r = 1 / np.sqrt(np.mean(h * h, -1, keepdims=True) + eps)
    dn = dy * w
    return d_res + r * (dn - h * r * r * np.mean(dn * h, -1, keepdims=True)), np.sum(dy * h * r, 0)


def log_softmax(z):
    """Of one row; -inf where a row holds nothing else."""
    m = z.max()
    if m == -np.inf:
        return np.full_like(z, -np.inf)
    with np.errstate(divide="ignore", invalid="ignore"):
        return z - m - np.log(np.sum(np.exp(z - m)))


def entropy(logq):
    some = logq > -np.inf
    return -np.sum(np.exp(logq[some]) * logq[some])


def top(x, k):
    """Indices of the k largest of a row, equal ones by ascending index."""
    return np.lexsort((np.arange(x.size), -x))[:k]


def logprobs_backward(logits, scale, target, g, f):
    """Gradient of g log q[target] + f entropy with respect to one row's logits."""
    logq = log_softmax(logits * scale)
    if logq.max() == -np.inf:
        return np.zeros_like(logits)
    q = np.exp(logq)
    d = -g * q
    if target is not None:
        d[target] += g
    some = logq > -np.inf
    d[some] -= f * q[some] * (logq[some] + entropy(logq))
    return scale * d


def teacher(ids, values, vocab, scale, given):
    """(ids, log p) of the entries that are there."""
    there = (ids >= 0) & (ids < vocab)
    ids, values = ids[there], values[there]
    if given or not ids.size or values.max() == -np.inf:
        return ids, values
    return ids, log_softmax(values * scale)


def distill(logits, scale, ids, values, given):
    """The divergence of one row."""
    logq = log_softmax(logits * scale)
    loss = 0.0
    for i, logp in zip(*teacher(ids, values, logits.size, scale, given)):
        if logp > -np.inf:
            loss += np.exp(logp) * (logp - logq[i])
    return loss


def distill_backward(logits, scale, ids, values, given, g):
    logq = log_softmax(logits * scale)
    if logq.max() == -np.inf:
        return np.zeros_like(logits)
    d = np.zeros_like(logits)
    for i, logp in zip(*teacher(ids, values, logits.size, scale, given)):
        d += np.exp(logp) * np.exp(logq)
        d[i] -= np.exp(logp)
    return g * scale * d
