"""The expert layer with BF16 activations on NVFP4 weights, in float64 (weights given as the values they stand for)."""
import numpy as np

from .formats import bf16_to_f64, f32_to_bf16
from .int8 import silu_mul


def forward(x, ids, w, start, w1, w2, add=None):
    """x float64 [T, H], ids [T, k], w float32 [T, k], w1 [L, 2I, H], w2 [L, H, I] float64 (global scales in them) ->
    (out float64 [T, H], scale float64 [T, H]: the sum of the magnitudes of its terms, h as the layer rounds it)."""
    T, H = x.shape
    L, I = len(w1), w1.shape[1] // 2
    out = np.zeros((T, H)) if add is None else np.array(add, np.float64)
    size = np.abs(out)
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j]) - start
            if not 0 <= e < L:
                continue
            gu = w1[e] @ x[t]
            h = bf16_to_f64(f32_to_bf16(silu_mul(gu[:I], gu[I:]).astype(np.float32)))
            out[t] += float(w[t, j]) * (w2[e] @ h)
            size[t] += abs(float(w[t, j])) * (np.abs(w2[e]) @ np.abs(h))
    return out, size
