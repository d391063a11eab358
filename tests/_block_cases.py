"""Inputs and helpers shared by the tests of the operators around the expert FFN."""
import numpy as np
import torch

import oracle.gate as G

DEV = "cuda:0"
EPS32 = 2.0 ** -24       # half a step of float32, relative
HALF_BF16 = 2.0 ** -8    # half a step of BF16, relative


def to_dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def as_stored(a, dtype):
    """float64 values of `a` after rounding to dtype ('f32' or 'bf16')."""
    t = torch.from_numpy(np.asarray(a, np.float32))
    return (t.to(torch.bfloat16) if dtype == "bf16" else t).double().numpy()


def torch_dtype(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def guarded(shape, dtype, fill):
    """A tensor of this shape inside a larger one, and a check that its surroundings kept their fill."""
    n = int(np.prod(shape))
    pad = 256 // torch.empty((), dtype=dtype).element_size()
    whole = torch.full((n + 2 * pad,), fill, dtype=dtype, device=DEV)
    mid = whole[pad:pad + n].view(*shape)

    def intact():
        torch.cuda.synchronize()
        return bool((whole[:pad] == fill).all() and (whole[pad + n:] == fill).all())
    return mid, intact


def gate_logits(case, seed):
    """Logits [T, E] of a kind, as float64 of what the given dtype stores."""
    T, E = case["T"], case["E"]
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, E)) * 1.5 + rng.standard_normal(E) * 0.5
    kind = case.get("kind", "plain")
    if kind == "ties":                       # few distinct values, whole rows equal
        x = np.round(x * 2) / 2
        x[::3] = 0.25
    elif kind == "holes":                    # experts a token must not use, rows without any, the type's lowest value
        x[rng.random((T, E)) < 0.6] = -np.inf
        x[::5] = -np.inf
        if T > 1:
            x[1, :] = -np.inf
            x[1, E // 2] = 0.5
        low = float(torch.finfo(torch_dtype(case["dtype"])).min)
        x[rng.random((T, E)) < 0.05] = low
    elif kind == "wide":                     # scores from underflow to saturation
        x = x * 12
    return as_stored(x, case["dtype"])


def grad_bound(x, ids, c, score, renormalize, mask, d_loss, counts, tokens, seq):
    """Per element: what float32 rounding may leave in d_logits. 64 half steps of the sum of the absolute values of
    the terms (some 20 operations each rounding once, exp and log within 2 steps), and the rounding of the argument
    x - max of an exponential, |x - max| half steps."""
    T, E = x.shape
    out = np.zeros((T, E))
    for t in range(T):
        fin = x[t][x[t] > -np.inf]
        if not len(fin):
            continue
        span = min(100.0, fin.max() - fin.min())
        s = G.scores(x[t], score)
        slope = s if score == G.SOFTMAX else np.abs(G.score_slopes(x[t], score))
        a = np.zeros(E)
        row = 0.0
        if c is not None:
            good = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E and x[t, ids[t, j]] > -np.inf]
            big = max([abs(c[t, j]) for j in good], default=0.0)
            if score == G.SOFTMAX and renormalize:
                w = G.weights(x[t], ids[t], score, True, 1.0)
                for j in good:
                    a[ids[t, j]] += w[j] * 2 * big
            else:
                total = sum(s[ids[t, j]] for j in good) if renormalize else 1.0
                for j in good:
                    if total > 0:
                        a[ids[t, j]] += 2 * big / total * slope[ids[t, j]]
                        row += big * s[ids[t, j]] / total
        if score == G.SOFTMAX:
            a += s * row
        if d_loss is not None and seq[t] >= 0 and s.sum() > 0:
            n = float(tokens[seq[t]])
            dq = abs(d_loss[0]) * E * counts[seq[t]] / (float(tokens[-1]) * n * n * ids.shape[1]) if n else np.zeros(E)
            a += (dq + (dq * s).sum() / s.sum()) / s.sum() * slope
            p = G.scores(x[t], G.SOFTMAX)
            a += abs(d_loss[1]) * 2 * (abs(fin.max()) + np.log(E) + 1) * p / max(1.0, float(tokens[-2]))
        out[t] = (64 + 2 * span) * EPS32 * a
    return out
