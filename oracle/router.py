"""Router, balance loss and their gradient (oracle side), in float64.

The definitions are this library's own (the pages route with given IDs and
weights). A logit of -inf or NaN takes its expert out of the row; +inf counts
as the largest finite fp32. t_e = exp(l_e) (softmax) or the logistic function
of l_e (sigmoid); scores are the logits, or t_e + bias_e; the topk largest are
chosen in descending order, ties to the lower expert; weights are
scale * t_j over the sum of t over the chosen (renorm), over all experts
(softmax), or over 1 (sigmoid). The balance loss is
coef * E * sum_e (count_e / (T topk)) * (mean over the T rows of p_te).

Written row by row over plain Python loops where the order matters (choice,
counts); ``loss_of_logits`` is the scalar that the gradient tests difference.
"""

import numpy as np

FMAX = float(np.finfo(np.float32).max)


def clean(logits):
    l = np.array(logits, dtype=np.float64)
    l[np.isnan(l)] = -np.inf
    return np.minimum(l, FMAX)


def _log_strength(l, scoring):
    """log t_e; -inf for an expert that takes no part."""
    if scoring == "softmax":
        return l
    with np.errstate(invalid="ignore"):
        out = -np.logaddexp(0.0, -l)
    out[np.isneginf(l)] = -np.inf
    return out


def _normalised(logt):
    """t over its sum, for a vector of log t (all zero if there is none)."""
    m = np.max(logt) if logt.size else -np.inf
    if np.isneginf(m):
        return np.zeros_like(logt)
    t = np.exp(logt - m)
    return t / t.sum()


def route_topk(logits, topk, scoring="softmax", renorm=True, scale=1.0, bias=None, row_mask=None):
    l = clean(logits)
    T, E = l.shape
    ids = np.full((T, topk), -1, dtype=np.int64)
    w = np.zeros((T, topk))
    for t in range(T):
        if row_mask is not None and not row_mask[t]:
            continue
        score = l[t].copy()
        if bias is not None:
            live = ~np.isneginf(l[t])
            score[live] = 1.0 / (1.0 + np.exp(-l[t][live])) + np.asarray(bias, np.float64)[live]
            score[np.isnan(score)] = -np.inf
        left = [e for e in range(E) if score[e] > -np.inf]
        chosen = []
        while left and len(chosen) < topk:
            best = max(left, key=lambda e: (score[e], -e))
            chosen.append(best)
            left.remove(best)
        if not chosen:
            continue
        logt = _log_strength(l[t], scoring)
        if renorm:
            v = _normalised(logt[chosen])
        elif scoring == "softmax":
            v = _normalised(logt)[chosen]
        else:
            v = np.exp(logt[chosen])
        ids[t, :len(chosen)] = chosen
        w[t, :len(chosen)] = scale * v
    return ids, w


def balance(logits, ids, scoring="softmax", coef=1.0):
    l = clean(logits)
    T, E = l.shape
    topk = ids.shape[1]
    count = np.zeros(E, dtype=np.int64)
    prob = np.zeros(E)
    tokens = 0
    for t in range(T):
        mine = [int(e) for e in ids[t] if 0 <= e < E]
        if not mine:
            continue
        tokens += 1
        for e in mine:
            count[e] += 1
        prob += _normalised(_log_strength(l[t], scoring))
    if tokens == 0:
        return {"loss": 0.0, "count": count, "prob": prob, "tokens": 0}
    prob /= tokens
    loss = coef * E * float(np.sum(count / (tokens * topk) * prob))
    return {"loss": loss, "count": count, "prob": prob, "tokens": tokens}


def backward(logits, ids, dw=None, scoring="softmax", renorm=True, scale=1.0, with_balance=False,
             coef=1.0, dloss=1.0, count=None, tokens=None):
    """d/dl of sum dw_j w_j + dloss * loss (counts held constant)."""
    l = clean(logits)
    T, E = l.shape
    topk = ids.shape[1]
    if with_balance and count is None:
        b = balance(logits, ids, scoring, coef)
        count, tokens = b["count"], b["tokens"]
    out = np.zeros((T, E))
    for t in range(T):
        at = [j for j in range(topk) if 0 <= ids[t, j] < E]
        if not at:
            continue
        logt = _log_strength(l[t], scoring)
        live = ~np.isneginf(l[t])
        # d log t / d l
        h = np.where(live, 1.0, 0.0)
        if scoring == "sigmoid":
            h = np.where(live, np.exp(-np.logaddexp(0.0, np.where(live, l[t], 0.0))), 0.0)
        g = np.zeros(E)  # gradient with respect to log t
        e = np.array([int(ids[t, j]) for j in at])
        if dw is not None:
            d = np.where(live[e], np.asarray(dw, np.float64)[t, at], 0.0)
            if renorm:
                q = _normalised(logt[e])
                np.add.at(g, e, scale * q * (d - np.sum(q * d)))
            elif scoring == "softmax":
                p = _normalised(logt)
                np.add.at(g, e, scale * p[e] * d)
                g -= p * scale * np.sum(p[e] * d)
            else:
                np.add.at(g, e, scale * np.exp(logt[e]) * d)
        if with_balance and tokens > 0:
            p = _normalised(logt)
            f = count / (tokens * topk)
            g += dloss * coef * E / tokens * p * (f - np.sum(f * p))
        out[t] = g * h
    return out


def loss_of_logits(logits, ids, dw, scoring, renorm, scale, coef, dloss, count, tokens):
    """The scalar whose gradient ``backward`` is, as a function of the logits
    with the IDs, counts and number of rows held constant."""
    l = clean(logits)
    T, E = l.shape
    topk = ids.shape[1]
    total = 0.0
    for t in range(T):
        at = [j for j in range(topk) if 0 <= ids[t, j] < E]
        if not at:
            continue
        e = [int(ids[t, j]) for j in at]
        tt = np.exp(l[t]) if scoring == "softmax" else 1.0 / (1.0 + np.exp(-l[t]))
        if renorm:
            w = scale * tt[e] / np.sum(tt[e])
        elif scoring == "softmax":
            w = scale * tt[e] / np.sum(tt)
        else:
            w = scale * tt[e]
        total += float(np.sum(np.asarray(dw, np.float64)[t, at] * w))
        if tokens > 0:
            total += dloss * coef * E * float(np.sum(count / (tokens * topk) * tt / tt.sum())) / tokens
    return total
