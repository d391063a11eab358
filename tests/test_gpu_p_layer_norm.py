"""Layer norm and its gradients against the float64 oracle.

Tolerances are float32 half steps (2^-24) of a result's terms, as for the block
norms: a row sum passes through at most 32 additions in the thread, 6 in the wave
and 16 over the waves, and enters through a root and a reciprocal: 96 half steps;
a column sum over T tokens adds T / 256 + 64. The mean m of a row is off by at
most 64 half steps of mean |r'|, and deviations are taken from m: that much is
added to their size before what the correction leaves is counted. A BF16 result
adds half a BF16 step (2^-8) of itself.
"""
import numpy as np
import pytest
import torch

import oracle.layer_norm as LN
from _block_cases import DEV, EPS32, HALF_BF16, as_stored, guarded, to_dev, torch_dtype

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_quantized_moe_amd as nv
    return nv


def case(T, H, x="bf16", res="bf16", w=True, b=True, kind="plain"):
    return dict(T=T, H=H, x=x, res=res, w=w, b=b, kind=kind)


CASES = [
    case(1, 8), case(1, 7168), case(3, 16, "f32", "f32"), case(5, 520, "bf16", "f32"), case(67, 2888, "f32", "bf16", b=False),
    case(300, 1032, w=False), case(9, 8192, "f32", None), case(4, 8200, "bf16", "f32"), case(3, 16384, "f32", "f32"),
    case(2, 16384, "bf16", None, w=False, b=False), case(19, 128), case(130, 512, "f32", "f32", kind="far"),
    case(40, 7168, "f32", None, kind="far"), case(8, 96, kind="constant"), case(33, 4096, res="f32"), case(515, 64, "f32", "f32"),
    case(64, 1000, kind="sizes"), case(777, 136, "bf16", "bf16"), case(1030, 2048, "bf16", "f32"), case(2100, 72, "f32", None),
]
IDS = [f"{i}-T{c['T']}-H{c['H']}-{c['x']}-{c['res']}-{c['kind']}" for i, c in enumerate(CASES)]


def inputs(c, seed):
    rng = np.random.default_rng(seed)
    T, H = c["T"], c["H"]
    x, r = rng.standard_normal((T, H)) + 0.3, rng.standard_normal((T, H)) * 2 + rng.standard_normal((T, 1))
    if c["kind"] == "far":        # rows whose mean is up to 10^6 deviations from 0
        off = 10.0 ** rng.uniform(0, 6, (T, 1))
        x, r = x + off, r + off
    elif c["kind"] == "constant":  # eps alone keeps these rows finite
        x[::2] = 0.5
        r[::2] = 4.0
    elif c["kind"] == "sizes":    # rows of very different size, one dominating element, the first one at that
        x, r = (v * 10.0 ** rng.uniform(-9, 9, (T, 1)) for v in (x, r))
        r[:, 0] *= 1e3
    p = dict(x=as_stored(x, c["x"]), residual=None if c["res"] is None else as_stored(r, c["res"]))
    p["w"] = as_stored(1 + 0.2 * rng.standard_normal(H), "f32") if c["w"] else None
    p["b"] = as_stored(0.5 * rng.standard_normal(H), "f32") if c["b"] else None
    p["scale"] = 1.0 if c["res"] is None else 0.75
    return p, rng


def put(a, dtype="f32"):
    return None if a is None else to_dev(a.astype(np.float32), torch_dtype(dtype))


def close(got, ref, tol, dtype, what):
    got = got.double().cpu().numpy()
    tol = tol + 2.0 ** -126
    if dtype == "bf16":
        tol = tol * (1 + HALF_BF16) + HALF_BF16 * np.abs(ref)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (what, int(bad.sum()), float(np.max(np.abs(got - ref) / tol)))


def y_tolerance(r, w, b):
    """(y, what float32 may leave in it) of stored rows r."""
    y = LN.forward(r, w, b, EPS)
    n, rho, c = LN.normalized(r, EPS)
    off = 64 * EPS32 * np.abs(r).mean(1, keepdims=True)              # of m
    dev = np.abs(c) + off + (np.abs(c) + off).mean(1, keepdims=True)  # an element's deviation and the correction's terms
    var = (c * c).mean(1, keepdims=True)
    rel = (var + off * off + off * np.abs(c).mean(1, keepdims=True)) / (var + EPS)
    w_abs = 1.0 if w is None else np.abs(w)
    return y, 96 * EPS32 * (rho * dev * w_abs + rel * np.abs(n) * w_abs + np.abs(y))


@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_forward(nv, c):
    p, _ = inputs(c, 1)
    T, H = c["T"], c["H"]
    y, y_ok = guarded((T, H), torch_dtype(c["x"]), 9.0)
    x, w, b = put(p["x"], c["x"]), put(p["w"]), put(p["b"])
    if c["res"] is None:
        got_r, got_y = nv.moe_layer_norm(x, None, w, b, eps=EPS, y=y)
        assert got_r is x
    else:
        out, out_ok = guarded((T, H), torch_dtype(c["res"]), 9.0)
        got_r, got_y = nv.moe_layer_norm(x, put(p["residual"], c["res"]), w, b, 0.75, EPS, residual_out=out, y=y)
        assert out_ok()
        ref, terms = LN.update(p["x"], p["residual"], 0.75)
        close(got_r, ref, 3 * EPS32 * terms, c["res"], "residual_out")
    assert y_ok()
    close(got_y, *y_tolerance(got_r.double().cpu().numpy(), p["w"], p["b"]), c["x"], "y")


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_codes_are_the_quantizers(nv, c, rule):
    p, _ = inputs(c, 3)
    T, H = c["T"], c["H"]
    args = [put(p["x"], c["x"]), put(p["residual"], c["res"]) if c["res"] else None, put(p["w"]), put(p["b"])]
    Hp = nv.mxfp4_padded(H)
    q, q_ok = guarded((T, Hp // 2), torch.uint8, 0x5A)
    s, s_ok = guarded((Hp // 128, T, 4), torch.uint8, 0x5A)
    r, y, _, _ = nv.moe_layer_norm(*args, scale=p["scale"], mx_rule=rule, y_q=q, y_scale=s)
    assert q_ok() and s_ok()
    r2, y2 = nv.moe_layer_norm(*args, scale=p["scale"])
    assert torch.equal(r, r2) and torch.equal(y, y2)
    want = nv.mxfp4_quantize(y, rule=rule)
    assert torch.equal(q, want[0]) and torch.equal(s, want[1])


@pytest.mark.parametrize("c", CASES, ids=IDS)
@pytest.mark.parametrize("with_res", [True, False])
def test_backward(nv, c, with_res):
    p, rng = inputs(c, 2)
    T, H = c["T"], c["H"]
    xt, rt = c["x"], c["res"] or c["x"]
    r = as_stored(LN.update(p["x"], p["residual"], p["scale"])[0], rt)
    d_y = as_stored(rng.standard_normal((T, H)), xt)
    d_r = as_stored(rng.standard_normal((T, H)), rt) if with_res else None
    bufs = dict(d_x=guarded((T, H), torch_dtype(xt), 5.0))
    if c["res"]:
        bufs["d_residual"] = guarded((T, H), torch_dtype(rt), 5.0)
    for n in "wb":
        if p[n] is not None:
            bufs["d_" + n] = guarded((H,), torch.float32, 5.0)
    ws, ws_ok = guarded((nv.moe_layer_norm_backward_ws_bytes(T, H),), torch.uint8, 0xA5)
    got = nv.moe_layer_norm_backward(put(d_y, xt), put(d_r, rt) if with_res else None, put(r, rt), put(p["w"]), put(p["b"]),
                                     p["scale"], EPS, residual=c["res"] is not None, ws=ws, **{n: v[0] for n, v in bufs.items()})
    assert all(v[1]() for v in bufs.values()) and ws_ok()
    assert {n for n, v in got.items() if v is not None} == set(bufs)
    ref = LN.backward(d_y, d_r, r, p["w"], p["scale"], EPS)
    # a row's mean off by `off`: its deviations, and what is multiplied by them, are larger by that share
    c_abs = np.abs(r - r.mean(1, keepdims=True)).mean(1, keepdims=True)
    off = 64 * EPS32 * np.abs(r).mean(1, keepdims=True)
    var = ((r - r.mean(1, keepdims=True)) ** 2).mean(1, keepdims=True)
    share = 1 + off / np.maximum(c_abs, 1e-300) + off * off / (var + EPS) if c["kind"] == "far" else 1.0
    far = float(np.max(share)) ** 2 if c["kind"] == "far" else 1.0
    for n in bufs:
        value, terms = ref[n]
        steps = 192 if n in ("d_x", "d_residual") else 192 + T / 256 + 64
        close(got[n], value, steps * EPS32 * terms * (share ** 2 if n in ("d_x", "d_residual") else far),
              {"d_x": xt, "d_residual": rt}.get(n, "f32"), n)


def test_gradients_against_differences(nv):
    """Of the calls themselves, float32 rows, along random directions."""
    T, H = 6, 200
    p, rng = inputs(case(T, H, "f32", "f32"), 5)
    d = {n: rng.standard_normal(p[n].shape) for n in ("x", "residual", "w", "b")}
    dy, dro = rng.standard_normal((T, H)), rng.standard_normal((T, H))

    def loss(h):
        v = {n: p[n] + h * d[n] for n in d}
        r, y = nv.moe_layer_norm(put(v["x"]), put(v["residual"]), put(v["w"]), put(v["b"]), 0.75, EPS)
        return float((y.double().cpu().numpy() * dy).sum() + (r.double().cpu().numpy() * dro).sum())
    r, _ = nv.moe_layer_norm(put(p["x"]), put(p["residual"]), put(p["w"]), put(p["b"]), 0.75, EPS)
    g = nv.moe_layer_norm_backward(put(dy), put(dro), r, put(p["w"]), put(p["b"]), 0.75, EPS)
    want = sum(float((g["d_" + n].double().cpu().numpy() * d[n]).sum()) for n in d)
    h = 2.0 ** -7
    got = (8 * (loss(h) - loss(-h)) - (loss(2 * h) - loss(-2 * h))) / (12 * h)
    # differences: rounding 2^-24 of about 4 T H terms of size 4 over 12 h / 18, and the fifth derivative times h^4
    assert abs(got - want) <= 18 * EPS32 * 16 * T * H / (12 * h) + 40 * h ** 4 * T * H


def test_not_finite(nv):
    """A row with an infinity or NaN is NaN, its neighbours are what they were."""
    x = torch.randn(9, 256, device=DEV).bfloat16()
    w, b = torch.randn(256, device=DEV), torch.randn(256, device=DEV)
    clean = nv.moe_layer_norm(x, None, w, b)[1]
    x[2, 5], x[6, 255] = float("inf"), float("nan")
    _, y, q, s = nv.moe_layer_norm(x, None, w, b, mx_rule=nv.MX_SCALE_FLOOR)
    rest = [t for t in range(9) if t not in (2, 6)]
    assert torch.equal(y[rest], clean[rest]) and torch.isnan(y[2]).all() and torch.isnan(y[6]).all()
    assert (s[:, [2, 6]] == 255).all() and (s[:, rest] != 255).all()


def test_in_place_and_empty(nv):
    p, _ = inputs(case(40, 1024), 6)
    x, r, w, b = put(p["x"], "bf16"), put(p["residual"], "bf16"), put(p["w"]), put(p["b"])
    r1, y1 = nv.moe_layer_norm(x, r, w, b, 0.75)
    d_y, d_r = torch.randn_like(x), torch.randn_like(r)
    g1 = nv.moe_layer_norm_backward(d_y, d_r, r1, w, b, 0.75)
    g2 = nv.moe_layer_norm_backward(d_y, d_r, r1, w, b, 0.75, d_x=d_y, d_residual=d_r)
    assert torch.equal(g1["d_x"], d_y) and torch.equal(g1["d_residual"], d_r)
    assert torch.equal(g1["d_w"], g2["d_w"]) and torch.equal(g1["d_b"], g2["d_b"])
    nv.moe_layer_norm(x, r, w, b, 0.75, residual_out=r, y=x)
    assert torch.equal(r, r1) and torch.equal(x, y1)
    empty, one = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV), torch.ones(64, device=DEV)
    for res in (None, empty):
        out = nv.moe_layer_norm(empty, res, one, one, 1.0 if res is None else 0.5, mx_rule=0)
        assert out[0].shape == out[1].shape == (0, 64) and out[2].shape == (0, 64) and out[3].shape == (1, 0, 4)
        g = nv.moe_layer_norm_backward(empty, None, empty, one, one, 1.0 if res is None else 0.5, residual=res is not None)
        assert not g["d_w"].any() and not g["d_b"].any()


def test_refused(nv):
    x = torch.zeros(4, 64, device=DEV)
    w = torch.zeros(64, device=DEV)
    for call in (lambda: nv.moe_layer_norm(x, None, w, w, scale=0.5), lambda: nv.moe_layer_norm(x, None, w, residual_out=x),
                 lambda: nv.moe_layer_norm(x, x[:3]), lambda: nv.moe_layer_norm(x, x, w[:8].clone()),
                 lambda: nv.moe_layer_norm(x, x, w.bfloat16()), lambda: nv.moe_layer_norm(x.half()),
                 lambda: nv.moe_layer_norm_backward(x, None, x.bfloat16(), w, residual=False),
                 lambda: nv.moe_layer_norm_backward(x, None, x, w, scale=2.0, residual=False),
                 lambda: nv.moe_layer_norm_backward(x, None, x, w, residual=False, d_residual=x),
                 lambda: nv.moe_layer_norm_backward(x, x.bfloat16(), x, w),
                 # outputs of what the call does not make
                 lambda: nv.moe_layer_norm(x, y_q=torch.zeros(4, 64, dtype=torch.uint8, device=DEV)),
                 lambda: nv.moe_layer_norm(x, y_scale=torch.zeros(1, 4, 4, dtype=torch.uint8, device=DEV)),
                 lambda: nv.moe_layer_norm_backward(x, None, x, d_w=w), lambda: nv.moe_layer_norm_backward(x, None, x, w, d_b=w)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(RuntimeError):   # a tensor where a truth value belongs
        nv.moe_layer_norm_backward(x, None, x, w, residual=x)
    with pytest.raises(nv.NVFP4Error):
        nv.moe_layer_norm(x, mx_rule=2)
    with pytest.raises(nv.NVFP4Error):
        nv.moe_layer_norm(torch.zeros(4, 60, device=DEV))


def test_equal_on_every_run_and_in_a_graph(nv):
    p, _ = inputs(case(777, 2888, "bf16", "f32"), 8)
    x, r, w, b = put(p["x"], "bf16"), put(p["residual"]), put(p["w"]), put(p["b"])
    o = dict(r=torch.empty_like(r), y=torch.empty_like(x), dx=torch.empty_like(x), dr=torch.empty_like(r),
             dw=torch.empty_like(w), db=torch.empty_like(w))
    ws = torch.empty(nv.moe_layer_norm_backward_ws_bytes(777, 2888), dtype=torch.uint8, device=DEV)
    d_y = torch.randn_like(x)

    def step():
        nv.moe_layer_norm(x, r, w, b, 0.75, residual_out=o["r"], y=o["y"])
        nv.moe_layer_norm_backward(d_y, None, o["r"], w, b, 0.75, d_x=o["dx"], d_residual=o["dr"], d_w=o["dw"],
                                   d_b=o["db"], ws=ws)

    def snap():
        torch.cuda.synchronize()
        return {n: t.clone() for n, t in o.items()}
    step()
    first = snap()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        for t in o.values():
            t.fill_(-3)
        ws.fill_(0xA5)
        graph.replay()
        again = snap()
        assert all(torch.equal(first[n], again[n]) for n in o)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    again = snap()
    assert all(torch.equal(first[n], again[n]) for n in o)
