"""The routing gate, the balance loss and their gradients, in float64.

Row by row and straight from the definitions in include/nvfp4moe.h; nothing
is shared with the kernels.
"""
import numpy as np

SOFTMAX, SIGMOID, SQRT_SOFTPLUS = 0, 1, 2


def scores(x, score):
    """Scores of logits x [..., E] (float64); -inf gives 0, a row of -inf gives zeros."""
    x = np.asarray(x, np.float64)
    if score == SOFTMAX:
        top = x.max(-1, keepdims=True)
        e = np.exp(x - np.where(np.isfinite(top), top, 0.0))
        s = e.sum(-1, keepdims=True)
        return np.divide(e, s, out=np.zeros_like(e), where=s > 0)
    if score == SIGMOID:
        return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))
    return np.sqrt(np.logaddexp(x, 0.0))


def score_slopes(x, score):
    """d score / d x of the scores that depend on one logit alone."""
    s = scores(x, score)
    if score == SIGMOID:
        return s * scores(-np.asarray(x, np.float64), SIGMOID)  # 1 - s would have lost its digits where s is near 1
    low = np.maximum(np.where(np.isfinite(x), x, -1e9), -700.0)
    full = scores(low, SIGMOID) / (2.0 * scores(low, score))
    return np.where(np.isfinite(x), full, 0.0)


def keys(x, score, bias=None, n_group=1, topk_group=1):
    """The keys of one row that the choice goes by; -inf where an expert cannot be chosen."""
    x = np.asarray(x, np.float64)
    if bias is None and n_group == 1:
        return x.copy()
    key = scores(x, score)
    if bias is not None:
        key = key + np.asarray(bias, np.float64)
    key = np.where(x > -np.inf, key, -np.inf)
    if n_group > 1:
        size = len(x) // n_group
        value = []
        for g in range(n_group):
            two = sorted((v for v in key[g * size:(g + 1) * size] if v > -np.inf), reverse=True)[:2]
            value.append(sum(two) if two else -np.inf)
        keep = sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group]
        for g in range(n_group):
            if g not in keep:
                key[g * size:(g + 1) * size] = -np.inf
    return key


def gate_topk(logits, k, score, bias=None, mask=None, n_group=1, topk_group=1, renormalize=True, scale=1.0):
    T, E = logits.shape
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        if mask is not None and mask[t] == 0:
            continue
        key = keys(logits[t], score, bias, n_group, topk_group)
        order = [e for e in sorted(range(E), key=lambda e: (-key[e], e)) if key[e] > -np.inf][:k]
        ids[t, :len(order)] = order
        w[t] = weights(logits[t], ids[t], score, renormalize, scale)
    return ids, w


def weights(x, ids, score, renormalize, scale):
    """Weights of one row's choices ids (any ids outside [0, E) give 0)."""
    E = len(x)
    x = np.asarray(x, np.float64)
    ok = (ids >= 0) & (ids < E)
    xl = np.where(ok, x[np.clip(ids, 0, E - 1)], -np.inf)
    if score == SOFTMAX and renormalize:
        if not np.isfinite(xl.max()):
            return np.zeros(len(ids))
        e = np.exp(xl - xl.max())
        return scale * e / e.sum()
    s = scores(x, score)[np.clip(ids, 0, E - 1)] * (xl > -np.inf)
    if renormalize:
        return scale * s / s.sum() if s.sum() > 0 else np.zeros(len(ids))
    return scale * s


def spans(T, cu):
    return [(0, T)] if cu is None else [(int(cu[b]), int(cu[b + 1])) for b in range(len(cu) - 1)]


def live_tokens(logits, mask):
    live = (np.asarray(logits, np.float64) > -np.inf).any(1)
    return live if mask is None else live & (np.asarray(mask) != 0)


def balance_loss(logits, ids, score, mask=None, cu=None):
    """(loss [2], counts [B, E], tokens [B + 2])."""
    T, E = logits.shape
    k = ids.shape[1]
    live = live_tokens(logits, mask)
    sp = spans(T, cu)
    counts = np.zeros((len(sp), E), np.int64)
    tokens, terms, z = [], [], []
    for b, (lo, hi) in enumerate(sp):
        share = np.zeros(E)
        n = 0
        for t in range(lo, hi):
            if not live[t]:
                continue
            n += 1
            for e in ids[t]:
                if 0 <= e < E:
                    counts[b, e] += 1
            s = scores(logits[t], score)
            if s.sum() > 0:
                share += s / s.sum()
            x = np.asarray(logits[t], np.float64)
            z.append((x.max() + np.log(np.exp(x - x.max()).sum())) ** 2)
        tokens.append(n)
        if n:
            terms.append(E * (counts[b] / (n * k) * share / n).sum())
    loss = np.array([np.mean(terms) if terms else 0.0, np.mean(z) if z else 0.0])
    return loss, counts.astype(np.int32), np.array(tokens + [sum(tokens), len(terms)], np.int32)


def gate_backward(logits, ids, score, renormalize=True, scale=1.0, mask=None, d_w=None, d_loss=None, counts=None,
                  tokens=None, cu=None):
    T, E = logits.shape
    k = ids.shape[1]
    live = live_tokens(logits, mask)
    dx = np.zeros((T, E))
    seq = np.full(T, -1)
    for b, (lo, hi) in enumerate(spans(T, cu)):
        seq[lo:hi] = b
    for t in range(T):
        if not live[t]:
            continue
        x = np.asarray(logits[t], np.float64)
        s = scores(x, score)
        ds = np.zeros(E)
        if d_w is not None:
            c = scale * np.asarray(d_w[t], np.float64)
            good = [j for j in range(k) if 0 <= ids[t, j] < E and x[ids[t, j]] > -np.inf]
            if score == SOFTMAX and renormalize:
                w = weights(x, ids[t], score, True, 1.0)
                dot = sum(c[j] * w[j] for j in good)
                for j in good:
                    dx[t, ids[t, j]] += w[j] * (c[j] - dot)
            else:
                total = sum(s[ids[t, j]] for j in good)
                dot = sum(c[j] * s[ids[t, j]] for j in good)
                for j in good:
                    if not renormalize:
                        ds[ids[t, j]] += c[j]
                    elif total > 0:
                        ds[ids[t, j]] += (c[j] - dot / total) / total
        if d_loss is not None and seq[t] >= 0:
            n, seqs = float(tokens[seq[t]]), float(tokens[-1])
            dq = float(d_loss[0]) * E * counts[seq[t]] / (seqs * n * n * k)
            if s.sum() > 0:
                q = s / s.sum()
                ds += (dq - (dq * q).sum()) / s.sum()
            p = scores(x, SOFTMAX)
            lse = x.max() + np.log(np.exp(x - x.max()).sum())
            dx[t] += float(d_loss[1]) * 2.0 * lse * p / float(tokens[-2])
        if score == SOFTMAX:
            dx[t] += s * (ds - (ds * s).sum())
        else:
            dx[t] += ds * score_slopes(x, score)
    return dx
