"""The block norms and their gradients against the float64 oracle.

Float32 arithmetic: tolerances are half steps (2^-24) times the sum of the
absolute values of a result's terms. A row sum passes through at most 32
additions in the thread, 6 in the wave and 16 over the waves, and enters
through a square root and a reciprocal; 96 half steps cover the chain. A
column sum over T tokens adds T / 256 + 64 in a row. A BF16 result adds half a
BF16 step (2^-8) of itself.
"""
import numpy as np
import pytest
import torch

import oracle.norm as N
from _block_cases import DEV, EPS32, HALF_BF16, as_stored, guarded, to_dev, torch_dtype

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_quantized_moe_amd as nv
    return nv


def case(T, H, x="bf16", res="bf16", gate="channel", post=True, pre=True, kind="plain", **kw):
    return dict(T=T, H=H, x=x, res=res, gate=gate, post=post, pre=pre, kind=kind, **kw)


CASES = [
    case(1, 8), case(1, 7168), case(3, 16, "f32", "f32", None, False), case(5, 520, "bf16", "f32", "token"),
    case(67, 2888, "f32", "bf16", "token", False), case(300, 1032, gate="token"), case(9, 8192, gate=None),
    case(4, 8200, "bf16", "f32"), case(3, 16384, "f32", "f32"), case(2, 16384), case(19, 128, pre=False),
    case(21, 264, "f32", "f32", None, False, pre=False), case(130, 512, kind="extreme"), case(8, 96, kind="zeros"),
    case(33, 4096, res="f32", residual=False), case(515, 64, "f32", "f32", "channel"),
]
IDS = [f"{i}-T{c['T']}-H{c['H']}-{c['x']}-{c['res']}-{c['gate']}" for i, c in enumerate(CASES)]


def inputs(c, seed):
    rng = np.random.default_rng(seed)
    T, H = c["T"], c["H"]
    x, r = rng.standard_normal((T, H)), rng.standard_normal((T, H)) * 2
    if c["kind"] == "extreme":   # rows of very different size, one dominating element
        x *= 10.0 ** rng.uniform(-9, 9, (T, 1))
        r *= 10.0 ** rng.uniform(-9, 9, (T, 1))
        x[:, 3] *= 1e3
    elif c["kind"] == "zeros":   # eps alone keeps these rows finite
        x[::2] = 0
        r[::2] = 0
    p = dict(x=as_stored(x, c["x"]), residual=as_stored(r, c["res"]) if c.get("residual", True) else None)
    p["w_pre"] = as_stored(1 + 0.2 * rng.standard_normal(H), "f32") if c["pre"] else None
    p["w_post"] = as_stored(0.5 + 0.2 * rng.standard_normal(H), "f32") if c["post"] else None
    shape = {"channel": (H,), "token": (T, 1)}
    p["gate"] = as_stored(rng.standard_normal(shape[c["gate"]]), "f32") if c["gate"] else None
    return p, rng


def f32_dev(a):
    return None if a is None else to_dev(a.astype(np.float32))


def close(got, ref, terms, steps, dtype, what):
    got = got.double().cpu().numpy()
    tol = steps * EPS32 * terms + 2.0 ** -126
    if dtype == "bf16":
        tol = tol * (1 + HALF_BF16) + HALF_BF16 * np.abs(ref)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (what, int(bad.sum()), float(np.max(np.abs(got - ref) / tol)))


@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_forward(nv, c):
    p, _ = inputs(c, 1)
    T, H = c["T"], c["H"]
    out, out_ok = guarded((T, H), torch_dtype(c["res"]), 9.0)
    y, y_ok = guarded((T, H), torch_dtype(c["x"]), 9.0)
    x = to_dev(p["x"].astype(np.float32), torch_dtype(c["x"]))
    r = None if p["residual"] is None else to_dev(p["residual"].astype(np.float32), torch_dtype(c["res"]))
    got_r, got_y = nv.moe_block_norm(x, r, f32_dev(p["w_pre"]), f32_dev(p["w_post"]), f32_dev(p["gate"]), scale=0.75,
                                     eps=1e-6, residual_out=out, y=y if c["pre"] else None)
    assert out_ok() and y_ok()
    ref, terms = N.update(p["x"], p["residual"], p["w_post"], p["gate"], 0.75, 1e-6)
    close(got_r, ref, terms, 96, c["res"], "residual_out")
    if c["pre"]:
        ref = N.normalize(got_r.double().cpu().numpy(), p["w_pre"], 1e-6)  # y is defined from r' as stored
        close(got_y, ref, np.abs(ref), 96, c["x"], "y")
    else:
        assert got_y is None


@pytest.mark.parametrize("c", CASES, ids=IDS)
@pytest.mark.parametrize("with_res", [True, False])
def test_backward(nv, c, with_res):
    if not with_res and not c["pre"]:
        pytest.skip("refused: nothing to differentiate")
    p, rng = inputs(c, 2)
    T, H = c["T"], c["H"]
    r, _ = N.update(p["x"], p["residual"], p["w_post"], p["gate"], 0.75, 1e-6)
    r = as_stored(r, c["res"])
    d_y = as_stored(rng.standard_normal((T, H)), c["x"]) if c["pre"] else None
    d_r = as_stored(rng.standard_normal((T, H)), c["res"]) if with_res else None
    xt, rt = torch_dtype(c["x"]), torch_dtype(c["res"])
    bufs = dict(d_x=guarded((T, H), xt, 5.0), d_residual=guarded((T, H), rt, 5.0))
    for n in ("w_pre", "w_post", "gate"):
        if p[n] is not None:
            bufs["d_" + n] = guarded(p[n].shape, torch.float32, 5.0)
    ws = torch.full((nv.moe_block_norm_backward_ws_bytes(T, H),), 0xA5, dtype=torch.uint8, device=DEV)
    put = lambda a, t: None if a is None else to_dev(a.astype(np.float32), t)  # noqa: E731
    got = nv.moe_block_norm_backward(put(d_y, xt), put(d_r, rt), put(p["x"], xt), put(r, rt), f32_dev(p["w_pre"]),
                                     f32_dev(p["w_post"]), f32_dev(p["gate"]), scale=0.75, eps=1e-6, ws=ws,
                                     **{n: b[0] for n, b in bufs.items()})
    assert all(b[1]() for b in bufs.values())
    ref = N.backward(d_y, d_r, p["x"], r, p["w_pre"], p["w_post"], p["gate"], 0.75, 1e-6)
    assert {n for n, v in got.items() if v is not None} == set(ref)
    for n, (value, terms) in ref.items():
        steps = 192 if n in ("d_x", "d_residual") else 192 + T / 256 + 64
        close(got[n], value, terms, steps, {"d_x": c["x"], "d_residual": c["res"]}.get(n, "f32"), n)


@pytest.mark.parametrize("T,H,res,scale", [(1, 32, "bf16", 1.0), (37, 7168, "bf16", 1.0), (70, 416, "f32", 0.02),
                                           (5, 8224, "bf16", 30.0), (2, 16384, "f32", 1.0)])
def test_nvfp4_output_equals_the_static_quantizer(nv, T, H, res, scale):
    c = case(T, H, "bf16", res)
    p, _ = inputs(c, 4)
    gs = torch.tensor([4.5 / 2688 * scale], device=DEV)  # scale < 1: blocks saturate
    q, q_ok = guarded((T, H // 2), torch.uint8, 0x5A)
    sf, sf_ok = guarded((T, H // 16), torch.uint8, 0x5A)
    args = (to_dev(p["x"].astype(np.float32), torch.bfloat16), to_dev(p["residual"].astype(np.float32), torch_dtype(res)),
            f32_dev(p["w_pre"]), f32_dev(p["w_post"]), f32_dev(p["gate"]))
    r, y, _, _ = nv.moe_block_norm(*args, scale=0.75, gs=gs, y_q=q, y_sf=sf)
    assert q_ok() and sf_ok()
    r2, y2 = nv.moe_block_norm(*args, scale=0.75)
    assert torch.equal(r, r2) and torch.equal(y.view(torch.int16), y2.view(torch.int16))
    ref_q, ref_sf = nv.nvfp4_quantize_static(y, gs)
    assert torch.equal(q, ref_q) and torch.equal(sf, ref_sf)


def test_in_place_and_empty(nv):
    p, _ = inputs(case(40, 1024), 6)
    x, r = to_dev(p["x"].astype(np.float32), torch.bfloat16), to_dev(p["residual"].astype(np.float32), torch.bfloat16)
    w, wp = f32_dev(p["w_pre"]), f32_dev(p["w_post"])
    r1, y1 = nv.moe_block_norm(x, r, w, wp)
    d_y, d_r = torch.randn_like(x), torch.randn_like(r)
    g1 = nv.moe_block_norm_backward(d_y, d_r, x, r1, w, wp)
    g2 = nv.moe_block_norm_backward(d_y, d_r, x, r1, w, wp, d_x=d_y, d_residual=d_r)
    assert torch.equal(g1["d_x"], d_y) and torch.equal(g1["d_residual"], d_r)
    assert all(torch.equal(g1[n], g2[n]) for n in ("d_w_pre", "d_w_post"))
    nv.moe_block_norm(x, r, w, wp, residual_out=r, y=x)
    assert torch.equal(r, r1) and torch.equal(x, y1)
    empty = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    out, y = nv.moe_block_norm(empty, empty, torch.ones(64, device=DEV))
    assert out.shape == y.shape == (0, 64)
    g = nv.moe_block_norm_backward(empty, None, empty, empty, torch.ones(64, device=DEV))
    assert not g["d_w_pre"].any()


def test_equal_on_every_run_and_in_a_graph(nv):
    p, _ = inputs(case(777, 2888, "bf16", "f32"), 8)
    x, r = to_dev(p["x"].astype(np.float32), torch.bfloat16), f32_dev(p["residual"])
    w, wp, g = f32_dev(p["w_pre"]), f32_dev(p["w_post"]), f32_dev(p["gate"])
    b = dict(r=torch.empty_like(r), y=torch.empty_like(x), dx=torch.empty_like(x), dr=torch.empty_like(r),
             a=torch.empty_like(w), b=torch.empty_like(w), c=torch.empty_like(w))
    ws = torch.empty(nv.moe_block_norm_backward_ws_bytes(777, 2888), dtype=torch.uint8, device=DEV)
    d_y = torch.randn_like(x)

    def step():
        nv.moe_block_norm(x, r, w, wp, g, residual_out=b["r"], y=b["y"])
        nv.moe_block_norm_backward(d_y, None, x, b["r"], w, wp, g, d_x=b["dx"], d_residual=b["dr"], d_w_pre=b["a"],
                                   d_w_post=b["b"], d_gate=b["c"], ws=ws)

    def snap():
        torch.cuda.synchronize()
        return {n: t.clone() for n, t in b.items()}

    step()
    first = snap()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        for t in b.values():
            t.fill_(-3)
        ws.fill_(0xA5)
        graph.replay()
        again = snap()
        assert all(torch.equal(first[n], again[n]) for n in b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    again = snap()
    assert all(torch.equal(first[n], again[n]) for n in b)
