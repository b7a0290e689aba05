"""The gated feed-forward block's forward and backward on the GPU, against its formulas in fp64.

Every comparison is element by element with a bound that is derived, not tuned:
 - a rounding to bf16 is off by at most 2^-8 of the value (half a step);
 - an fp32 sum of K products by at most K 2^-23 of the sum of their magnitudes (each addition of
   the tensor cores may truncate: twice the bound of rounding to nearest);
 - the activation's fast exp and quotient by at most 2^-18 of |g| (1 + |u|).
The kernels round h, du and dg to bf16 before the products that read them, and each result once.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

R16 = 2.0 ** -8
R32 = 2.0 ** -23
ACT = 2.0 ** -18


def _layer(**kw):
    from mixture_experts_layer_block_b200.native import MoELayer
    return MoELayer(256, 128, 8, 2, 16, 16, **kw)


def _inputs(T, H, D, seed=0, sigma_x=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape, s=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * s).to(torch.bfloat16)

    wts = {"Ws_up": r(D, H, s=1.2 / H ** 0.5), "Ws_gate": r(D, H, s=1.2 / H ** 0.5), "Ws_down": r(H, D, s=1.0 / D ** 0.5)}
    return r(T, H, s=sigma_x), wts, r(T, H)


def _forward_reference(x, wts):
    """out, u, g in fp64, and how far each may be off before its own rounding."""
    x, up, gate, down = x.double(), *(wts[n].double() for n in ("Ws_up", "Ws_gate", "Ws_down"))
    H, D = x.shape[1], up.shape[0]
    u, g = x @ up.T, x @ gate.T
    eu, eg = (H * R32 * (x.abs() @ w.abs().T) for w in (up, gate))
    s = torch.sigmoid(u)
    h = u * s * g
    eh = 1.1 * g.abs() * eu + (u * s).abs() * eg + eu * eg + ACT * g.abs() * (1 + u.abs())
    eh = eh + R16 * (h.abs() + eh)
    out = h @ down.T
    eo = eh @ down.abs().T + D * R32 * (h.abs() @ down.abs().T)
    return out, u, g, eo, eu, eg


def _backward_reference(dout, x, u, g, wts):
    """{name: (gradient, how far it may be off before its own rounding)} from the given u and g."""
    dout, x, u, g = dout.double(), x.double(), u.double(), g.double()
    up, gate, down = (wts[n].double() for n in ("Ws_up", "Ws_gate", "Ws_down"))
    (T, H), D = x.shape, up.shape[0]
    s = torch.sigmoid(u)
    a, da = u * s, s * (1 + u * (1 - s))
    dh = dout @ down
    e = H * R32 * (dout.abs() @ down.abs())
    du, dg, h = dh * g * da, dh * a, a * g

    def rounded(v, err):
        return err + R16 * (v.abs() + err)

    act = ACT * (1 + u.abs())
    edu = rounded(du, e * (g * da).abs() + (dh.abs() + e) * g.abs() * act)
    edg = rounded(dg, e * a.abs() + (dh.abs() + e) * act)
    eh = rounded(h, g.abs() * act)
    dx = du @ up + dg @ gate
    edx = edu @ up.abs() + edg @ gate.abs() + 2 * D * R32 * (du.abs() @ up.abs() + dg.abs() @ gate.abs())

    def weight(d, ed, b):
        return d.T @ b, ed.T @ b.abs() + T * R32 * (d.abs().T @ b.abs())

    return {"x": (dx, edx), "Ws_up": weight(du, edu, x), "Ws_gate": weight(dg, edg, x),
            "Ws_down": (dout.T @ h, dout.abs().T @ eh + T * R32 * (dout.abs().T @ h.abs()))}


def _close(got, ref, err, name):
    err = err + (R16 * (ref.abs() + err) if got.dtype == torch.bfloat16 else 0) + 1e-30
    bad = ~((got.double() - ref).abs() <= err)
    assert not bool(bad.any()), (name, int(bad.sum()), float(((got.double() - ref).abs() / err).max()))


# one token to several m-tiles; sizes off every tile, chunk and 64-wide block; the smallest sizes
SHAPES = [(1, 256, 128), (5, 264, 136), (16, 2048, 512), (17, 264, 136), (31, 8, 8), (64, 1024, 72), (127, 72, 1024),
          (128, 512, 256), (129, 2048, 512), (257, 328, 1032), (333, 2048, 200), (515, 2048, 512), (1030, 520, 1544),
          # few tokens and long sums over few tiles
          (5, 264, 2048), (16, 2568, 2048), (9, 24, 4104), (2, 8, 8),
          # rows spread over tiles that none of them fills; K split with the narrowest tiles; one K block
          (777, 1024, 520), (20, 7168, 64), (40, 64, 2056), (200, 4104, 72), (513, 72, 72), (900, 264, 64)]


@pytest.mark.parametrize("T,H,D", SHAPES)
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_forward(T, H, D, out_dtype):
    layer = _layer()
    x, wts, _ = _inputs(T, H, D, seed=T + H + D)
    # results in the middle of larger buffers: what lies around them stays
    buf = torch.full((T + 4, H), 7.0, dtype=out_dtype, device="cuda")
    ub, gb = (torch.full((T + 4, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out, u, g = buf[2:T + 2], ub[2:T + 2], gb[2:T + 2]
    assert layer.ffn_forward(x, wts, out, u=u, g=g) is out
    ref, ru, rg, eo, eu, eg = _forward_reference(x, wts)
    _close(u, ru, eu, "u")
    _close(g, rg, eg, "g")
    _close(out, ref, eo, "out")
    for b in (buf, ub, gb):
        assert bool((b[:2] == 7).all()) and bool((b[T + 2:] == 7).all())
    # without u and g: the same bits
    again = torch.empty_like(out)
    layer.ffn_forward(x, wts, again)
    assert torch.equal(again, out)
    assert layer.status() == (0, 0)
    layer.close()


@pytest.mark.parametrize("T,H,D", SHAPES)
@pytest.mark.parametrize("grad_dtype", [torch.bfloat16, torch.float32])
def test_backward(T, H, D, grad_dtype):
    layer = _layer()
    x, wts, dout = _inputs(T, H, D, seed=T + 3 * H + D)
    u, g = (x.float() @ wts["Ws_up"].float().T).bfloat16(), (x.float() @ wts["Ws_gate"].float().T).bfloat16()
    buf = torch.full((T + 4, H), 7.0, dtype=torch.bfloat16, device="cuda")
    grads = {"x": buf[2:T + 2], **{n: torch.full_like(w, float("nan"), dtype=grad_dtype) for n, w in wts.items()}}
    layer.ffn_backward(dout, x, u, g, wts, grads)
    ref = _backward_reference(dout, x, u, g, wts)
    for n in grads:
        _close(grads[n], *ref[n], n)
    assert bool((buf[:2] == 7).all()) and bool((buf[T + 2:] == 7).all())
    # each gradient on its own has the same bits; those not asked for are not written
    for n in grads:
        one = {m: (torch.full_like(grads[m], 3.0) if m == n else None) for m in grads}
        layer.ffn_backward(dout, x, u, g, wts, one)
        assert torch.equal(one[n], grads[n]), n
    assert layer.status() == (0, 0)
    layer.close()


@pytest.mark.parametrize("T,H,D", [(9, 264, 136), (300, 512, 328)])
def test_backward_adds_to_fp32_gradients(T, H, D):
    layer = _layer()
    x, wts, dout = _inputs(T, H, D, seed=5)
    u, g = (x.float() @ wts["Ws_up"].float().T).bfloat16(), (x.float() @ wts["Ws_gate"].float().T).bfloat16()
    once = {n: torch.empty_like(w, dtype=torch.float32) for n, w in wts.items()}
    layer.ffn_backward(dout, x, u, g, wts, once)
    start = {n: torch.randn_like(v) for n, v in once.items()}
    both = {n: v.clone() for n, v in start.items()}
    layer.ffn_backward(dout, x, u, g, wts, both, accumulate=True)
    for n in both:  # one fp32 addition each
        assert torch.equal(both[n], start[n] + once[n]), n
    layer.close()


def test_gradients_against_differences():
    """L = sum(out * dout) moves by the gradient times the step, at sizes where a bf16 forward
    resolves the difference: the directional derivative of each input against the fp64 forward."""
    layer = _layer()
    T, H, D = 40, 136, 72
    x, wts, dout = _inputs(T, H, D, seed=11)
    out = torch.empty_like(x)
    u, g = (torch.empty(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    layer.ffn_forward(x, wts, out, u=u, g=g)
    grads = {"x": torch.empty_like(x), **{n: torch.empty_like(w, dtype=torch.float32) for n, w in wts.items()}}
    layer.ffn_backward(dout, x, u, g, wts, grads)
    at = {"x": x.double(), **{n: w.double() for n, w in wts.items()}}

    def loss(p):
        a, b = p["x"] @ p["Ws_up"].T, p["x"] @ p["Ws_gate"].T
        return float((((a * torch.sigmoid(a)) * b) @ p["Ws_down"].T * dout.double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(3)
    for n in at:
        d = torch.randn(at[n].shape, generator=gen, device="cuda", dtype=torch.float64)
        step = 1e-4 / float(d.abs().max())
        diff = (loss({**at, n: at[n] + step * d}) - loss({**at, n: at[n] - step * d})) / (2 * step)
        # u, g, h, du, dg, dx each carry at most one bf16 rounding (six of 2^-8), on terms of either
        # sign: bounded by the sum of the magnitudes
        size = float((grads[n].double().abs() * d.abs()).sum())
        assert abs(float((grads[n].double() * d).sum()) - diff) <= 6 * R16 * size, n
    layer.close()


@pytest.mark.parametrize("T", [9, 200])
def test_bad_values_stay_in_their_row(T):
    """An infinite or NaN token spoils its own row of out, u, g and dx and no other; very large
    pre-activations of either sign saturate the activation without NaN."""
    layer = _layer()
    H, D = 264, 136
    x, wts, dout = _inputs(T, H, D, seed=2)
    clean = torch.empty_like(x)
    layer.ffn_forward(x, wts, clean)
    x2 = x.clone()
    x2[3, 5], x2[T - 1, 0], x2[6] = float("inf"), float("nan"), x[6] * 3000
    out = torch.empty_like(x)
    u, g = (torch.empty(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    layer.ffn_forward(x2, wts, out, u=u, g=g)
    keep = [t for t in range(T) if t not in (3, 6, T - 1)]
    assert torch.equal(out[keep], clean[keep])
    assert bool(torch.isnan(out[T - 1]).all())
    assert bool(torch.isfinite(out[6]).all())
    grads = {"x": torch.empty_like(x)}
    layer.ffn_backward(dout, x2, u, g, wts, grads)
    assert bool(torch.isfinite(grads["x"][keep + [6]]).all())
    assert layer.status() == (0, 0)
    layer.close()


def test_no_tokens():
    layer = _layer()
    x, wts, _ = _inputs(0, 64, 32)
    out = torch.empty(0, 64, device="cuda")
    layer.ffn_forward(x, wts, out)
    e = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        grads = {"x": torch.empty_like(x), **{n: torch.full_like(w, 9.0, dtype=dtype) for n, w in wts.items()}}
        layer.ffn_backward(x, x, e, e, wts, grads)
        assert all(bool((grads[n] == 0).all()) for n in wts)
    grads = {n: torch.full_like(w, 9.0, dtype=torch.float32) for n, w in wts.items()}
    layer.ffn_backward(x, x, e, e, wts, grads, accumulate=True)
    assert all(bool((grads[n] == 9).all()) for n in wts)
    layer.close()


@pytest.mark.parametrize("T", [7, 150])
def test_training_step_captured_and_replayed(T):
    """Forward and backward captured in one graph with buffers of its own, replayed on new inputs
    beside eager calls of the same handle on another stream: all equal the eager results."""
    layer = _layer()
    H, D = 520, 264
    x, wts, dout = _inputs(T, H, D, seed=1)
    out, u, g = torch.empty_like(x), *(torch.empty(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    grads = {"x": torch.empty_like(x), **{n: torch.empty_like(w) for n, w in wts.items()}}

    def step(x, dout, out, u, g, grads):
        layer.ffn_forward(x, wts, out, u=u, g=g)
        layer.ffn_backward(dout, x, u, g, wts, grads)

    step(x, dout, out, u, g, grads)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(x, dout, out, u, g, grads)
    side = torch.cuda.Stream()
    for seed in (21, 22):
        x1, _, d1 = _inputs(T, H, D, seed=seed)
        x.copy_(x1)
        dout.copy_(d1)
        e_out, e_u, e_g = torch.empty_like(x), torch.empty_like(u), torch.empty_like(g)
        e_grads = {n: torch.empty_like(v) for n, v in grads.items()}
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            step(x1, d1, e_out, e_u, e_g, e_grads)
        torch.cuda.synchronize()
        assert torch.equal(out, e_out) and torch.equal(u, e_u) and torch.equal(g, e_g)
        for n in grads:
            assert torch.equal(grads[n], e_grads[n]), n
    assert layer.status() == (0, 0)
    layer.close()


def test_workspace_of_the_stated_size_is_enough_and_not_exceeded():
    layer = _layer()
    for T, H, D in ((3, 264, 136), (60, 1032, 264), (700, 520, 72)):
        x, wts, dout = _inputs(T, H, D, seed=4)
        u, g = (torch.empty(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        for back in (False, True):
            need = layer.ffn_workspace_bytes(T, H, D, back)
            buf = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
            if back:
                layer.ffn_backward(dout, x, u, g, wts, {"x": torch.empty_like(x), **{n: torch.empty_like(w) for n, w in wts.items()}},
                                   workspace=buf[256:need + 256])
            else:
                layer.ffn_forward(x, wts, torch.empty_like(x), u=u, g=g, workspace=buf[256:need + 256])
            assert bool((buf[:256] == 0x5A).all()) and bool((buf[need + 256:] == 0x5A).all())
            with pytest.raises(ValueError):
                layer.ffn_forward(x, wts, torch.empty_like(x), workspace=buf[:max(0, layer.ffn_workspace_bytes(T, H, D) - 1)])
    layer.close()


def test_stream_argument():
    layer = _layer()
    x, wts, _ = _inputs(50, 264, 136, seed=8)
    ref, out = torch.empty_like(x), torch.empty_like(x)
    layer.ffn_forward(x, wts, ref)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    layer.ffn_forward(x, wts, out, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    layer.close()


def test_matches_the_layers_shared_expert():
    """The layer's W_shared(x) term: a layer forward whose router weighs one zero expert gives the
    block's output (both round h to bf16; the layer also rounds the block's row)."""
    from mixture_experts_layer_block_b200 import native
    H, D, T = 256, 128, 40
    layer = native.MoELayer(H, 64, 2, 1, 16, T, inter_shared=D)
    x, wts, _ = _inputs(T, H, D, seed=6)
    w = dict(wts, W_router=torch.zeros(2, H, dtype=torch.bfloat16, device="cuda"),
             W_up=torch.zeros(2, 64, H, dtype=torch.bfloat16, device="cuda"),
             W_gate=torch.zeros(2, 64, H, dtype=torch.bfloat16, device="cuda"),
             W_down=torch.zeros(2, H, 64, dtype=torch.bfloat16, device="cuda"))
    whole, block = torch.empty(T, H, device="cuda"), torch.empty(T, H, device="cuda")
    layer.forward(x, w, whole)
    layer.ffn_forward(x, wts, block)
    ref, _, _, eo, _, _ = _forward_reference(x, wts)
    _close(block, ref, eo, "block")
    err = eo + R16 * (ref.abs() + eo)
    assert bool(((whole.double() - ref).abs() <= err).all())
    layer.close()


def test_two_streams_at_once():
    """Calls of one handle on two streams overlap, each with a workspace of its own, and agree with the
    same calls one after another."""
    layer = _layer()
    cases = [(300, 520, 264), (12, 1024, 512)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    data, refs, got = [], [], []
    for i, (T, H, D) in enumerate(cases):
        x, wts, dout = _inputs(T, H, D, seed=30 + i)
        u, g = (torch.empty(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ref = {"out": torch.empty_like(x), "x": torch.empty_like(x), **{n: torch.empty_like(w) for n, w in wts.items()}}
        layer.ffn_forward(x, wts, ref["out"], u=u, g=g)
        layer.ffn_backward(dout, x, u, g, wts, {n: v for n, v in ref.items() if n != "out"})
        data.append((x, wts, dout, u, g))
        refs.append(ref)
        got.append([{n: torch.empty_like(v) for n, v in ref.items()} for _ in range(8)])
    torch.cuda.synchronize()
    for rep in range(8):
        for i, st in enumerate(streams):
            x, wts, dout, u, g = data[i]
            layer.ffn_forward(x, wts, got[i][rep]["out"], stream=st)
            layer.ffn_backward(dout, x, u, g, wts, {n: v for n, v in got[i][rep].items() if n != "out"}, stream=st)
    torch.cuda.synchronize()
    for i in range(2):
        for rep in range(8):
            for n, v in refs[i].items():
                assert torch.equal(got[i][rep][n], v), (i, rep, n)
    assert layer.status() == (0, 0)
    layer.close()


def test_offsets_past_32_bits():
    """More than 2^31 elements of x, out, dx and dout: rows at both ends against fp64, and the weight
    gradients against fp64 sums over all rows."""
    layer = _layer()
    T, H, D = 5 * 2 ** 19 + 77, 1024, 64
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    _, wts, _ = _inputs(1, H, D, seed=3)
    dout = torch.empty_like(x).normal_(generator=gen)
    out, dx = torch.empty_like(x), torch.empty_like(x)
    u, g = (torch.empty(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    layer.ffn_forward(x, wts, out, u=u, g=g)
    grads = {"x": dx, "Ws_up": torch.empty(D, H, device="cuda")}
    layer.ffn_backward(dout, x, u, g, wts, grads)
    rows = torch.cat([torch.arange(0, 300), torch.arange(2 ** 21 - 200, 2 ** 21 + 200), torch.arange(T - 300, T)]).cuda()
    ref, ru, rg, eo, eu, eg = _forward_reference(x[rows], wts)
    _close(out[rows], ref, eo, "out")
    _close(u[rows], ru, eu, "u")
    _close(g[rows], rg, eg, "g")
    back = _backward_reference(dout[rows], x[rows], u[rows], g[rows], wts)
    _close(dx[rows], *back["x"], "x")
    # W_up's gradient in slices; its fp32 sum of T products is off by at most T 2^-23 of their magnitudes'
    dw, mag = (torch.zeros(D, H, dtype=torch.float64, device="cuda") for _ in range(2))
    for r in range(0, T, 1 << 17):
        c = slice(r, min(T, r + (1 << 17)))
        uu, gg = u[c].double(), g[c].double()
        s = torch.sigmoid(uu)
        du = (dout[c].double() @ wts["Ws_down"].double()) * gg * (s * (1 + uu * (1 - s)))
        dw += du.T @ x[c].double()
        mag += du.abs().T @ x[c].double().abs()
    assert bool(((grads["Ws_up"].double() - dw).abs() <= (R16 * 1.1 + T * R32) * mag).all())
    # and closer on the whole: independent roundings of T terms (2^-8 each) leave about 2^-8 / sqrt(T) of
    # the magnitudes' sum, and truncated additions a drift below 2^-12 of it
    assert float((grads["Ws_up"].double() - dw).norm() / dw.norm()) < 0.02
    assert layer.status() == (0, 0)
    layer.close()


@pytest.mark.parametrize("T", [8, 40])
def test_overlapping_results_are_refused(T):
    from mixture_experts_layer_block_b200 import native
    H, D = 64, 64
    layer = _layer()
    x, wts, dout = _inputs(T, H, D, seed=2)
    buf = torch.zeros(4 * T, D, dtype=torch.bfloat16, device="cuda")
    u, g, out = buf[:T], buf[T:2 * T], buf[2 * T:3 * T]  # side by side: allowed
    layer.ffn_forward(x, wts, out, u=u, g=g)
    ref = torch.empty_like(x)
    layer.ffn_forward(x, wts, ref)
    assert torch.equal(out, ref)

    def forward(out=out, u=u, g=g, ws=None):
        layer.ffn_forward(x, wts, out, u=u, g=g, workspace=ws)

    grads = {"x": torch.empty_like(x), **{n: torch.empty_like(w) for n, w in wts.items()}}

    def backward(dout=dout, ws=None, **kw):
        layer.ffn_backward(dout, x, u, g, wts, dict(grads, **kw), workspace=ws)

    big = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    inside = big[:2 * T * H].view(torch.bfloat16).view(T, H)
    for call in (lambda: forward(out=x), lambda: forward(u=u, g=u), lambda: forward(out=buf[T + 1:2 * T + 1]),
                 lambda: forward(out=wts["Ws_up"][:T]), lambda: forward(out=inside, ws=big),
                 lambda: backward(x=dout), lambda: backward(x=x), lambda: backward(x=u),
                 lambda: backward(Ws_up=grads["Ws_gate"]), lambda: backward(Ws_down=wts["Ws_down"]),
                 lambda: backward(x=inside, ws=big)):
        with pytest.raises(native.MoEError) as err:
            call()
        assert err.value.code == native.MOE_ERR_INVALID_ARG
    backward()
    backward(dout=x)  # an input may serve twice
    assert layer.status() == (0, 0)
    layer.close()


def test_a_long_kernel_in_front_is_not_on_the_clock():
    """The waits' limit counts from the end of the kernel in front: behind one of about a millisecond
    that lets its successor in early, a limit of 0.2 ms is enough for a small call."""
    from mixture_experts_layer_block_b200.native import MoELayer
    layer = MoELayer(256, 128, 8, 2, 16, 16, timeout_ns=200_000)
    x, wts, dout = _inputs(40, 264, 136, seed=8)
    u, g = (torch.empty(40, 136, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ref, out = torch.empty_like(x), torch.empty_like(x)
    dx, dref = torch.empty_like(x), torch.empty_like(x)
    layer.ffn_forward(x, wts, ref, u=u, g=g)
    layer.ffn_backward(dout, x, u, g, wts, {"x": dref})
    long = torch.zeros(1 << 18, 1 << 14, dtype=torch.bfloat16, device="cuda")  # 8 GB: more than 1 ms to read
    assert layer.status() == (0, 0)
    for _ in range(3):
        layer.quantize_int4(long)
        layer.ffn_forward(x, wts, out)
        layer.quantize_int4(long)
        layer.ffn_backward(dout, x, u, g, wts, {"x": dx})
    assert layer.status() == (0, 0)
    assert torch.equal(out, ref) and torch.equal(dx, dref)
    layer.close()


@pytest.mark.parametrize("what", ["up", "down", "dh", "gradients"])
def test_a_wait_that_runs_out_is_reported(what):
    """Sums so long that the epilogue's wait for the first tile (a quarter of a millisecond, or 35 us where
    the 2048 blocks of a gradient's sum are split 16 ways) passes a limit of 5 us: the call drains what it had in
    flight and returns, the status says so and is cleared, and the next call is right."""
    from mixture_experts_layer_block_b200.native import MOE_ERR_DEVICE_TIMEOUT, MoELayer
    # 74 tiles of one product, each one sum of 1024 blocks of 64 whose K is not split; dx of 2048 blocks
    T, H, D = {"up": (37 * 256, 1 << 16, 256), "down": (37 * 256, 512, 1 << 16), "dh": (37 * 256, 1 << 16, 512),
               "gradients": (37 * 256, 512, 1 << 16)}[what]
    layer = MoELayer(256, 128, 8, 2, 16, 16, timeout_ns=5_000)
    x, dout = (torch.zeros(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    u, g = (torch.zeros(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wts = {"Ws_up": torch.zeros(D, H, dtype=torch.bfloat16, device="cuda"),
           "Ws_gate": torch.zeros(D, H, dtype=torch.bfloat16, device="cuda"),
           "Ws_down": torch.zeros(H, D, dtype=torch.bfloat16, device="cuda")}
    if what in ("up", "down"):
        layer.ffn_forward(x, wts, dout)
    else:
        layer.ffn_backward(dout, x, u, g, wts, {"x": torch.empty_like(x), **{n: torch.empty_like(w) for n, w in wts.items()}})
    rc, st = layer.status()
    assert rc == MOE_ERR_DEVICE_TIMEOUT and st & (1 << 30)
    assert layer.status() == (0, 0)
    x, wts, _ = _inputs(20, 64, 64, seed=1)
    out = torch.empty(20, 64, device="cuda")
    patient = _layer()
    patient.ffn_forward(x, wts, out)
    assert patient.status() == (0, 0)
    ref, _, _, eo, _, _ = _forward_reference(x, wts)
    _close(out, ref, eo, "out")
    layer.close()
    patient.close()


def _a_call_that_runs_out(layer):
    """Arguments of a forward whose first tile sums 4096 blocks of 64 (a millisecond)."""
    T, H, D = 37 * 256, 1 << 18, 256
    assert layer.ffn_workspace_bytes(T, H, D) == 2 * T * D  # K is not split
    wts = {"Ws_up": torch.zeros(D, H, dtype=torch.bfloat16, device="cuda"),
           "Ws_gate": torch.zeros(D, H, dtype=torch.bfloat16, device="cuda"),
           "Ws_down": torch.zeros(H, D, dtype=torch.bfloat16, device="cuda")}
    return torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), wts, torch.empty(T, H, dtype=torch.bfloat16, device="cuda")


def test_a_handle_whose_wait_ran_out_works_again():
    """Until the status is read, further calls return and the timeout stays to be reported; after it the same
    handle's calls are right, forward and backward, and nothing is left to report."""
    from mixture_experts_layer_block_b200.native import MOE_ERR_DEVICE_TIMEOUT, MoELayer
    layer = MoELayer(256, 128, 8, 2, 16, 16, timeout_ns=200_000)
    long = _a_call_that_runs_out(layer)
    x, wts, dout = _inputs(200, 264, 136, seed=1)
    out = torch.empty(200, 264, device="cuda")
    u, g = (torch.empty(200, 136, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    grads = {"x": torch.empty_like(x), **{n: torch.empty_like(w) for n, w in wts.items()}}
    for _ in range(2):
        layer.ffn_forward(*long)
        layer.ffn_forward(x, wts, out, u=u, g=g)
        layer.ffn_backward(dout, x, u, g, wts, grads)
        rc, st = layer.status()
        assert rc == MOE_ERR_DEVICE_TIMEOUT and st & (1 << 30)
        for t in (out, u, g, *grads.values()):
            t.fill_(float("nan"))
        layer.ffn_forward(x, wts, out, u=u, g=g)
        ref, ru, rg, eo, eu, eg = _forward_reference(x, wts)
        _close(out, ref, eo, "out")
        _close(u, ru, eu, "u")
        _close(g, rg, eg, "g")
        layer.ffn_backward(dout, x, u, g, wts, grads)
        for n, (r, e) in _backward_reference(dout, x, u, g, wts).items():
            _close(grads[n], r, e, n)
        assert layer.status() == (0, 0)
    layer.close()


def test_the_status_covers_every_stream():
    """A wait that runs out on one stream, behind tens of milliseconds of other work, is reported although the
    handle's last call, on another stream, was over long before."""
    from mixture_experts_layer_block_b200.native import MOE_ERR_DEVICE_TIMEOUT, MoELayer
    layer = MoELayer(256, 128, 8, 2, 16, 16, timeout_ns=200_000)
    long = _a_call_that_runs_out(layer)
    x, wts, _ = _inputs(4, 264, 136, seed=1)
    out = torch.empty_like(x)
    busy = torch.zeros(1 << 32, dtype=torch.uint8, device="cuda")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    layer.ffn_forward(x, wts, out, stream=b)
    torch.cuda.synchronize()
    with torch.cuda.stream(a):
        for _ in range(20):  # 1.3 ms each at least
            busy.add_(1)
    layer.ffn_forward(*long, stream=a)
    layer.ffn_forward(x, wts, out, stream=b)
    rc, st = layer.status()
    assert rc == MOE_ERR_DEVICE_TIMEOUT and st & (1 << 30)
    assert layer.status() == (0, 0)
    layer.close()


def test_the_layers_counters_wait_for_the_layer():
    """What the layer's last forward left is read behind that forward, not behind a later call of the block on
    another stream."""
    from mixture_experts_layer_block_b200 import configs, inputs as gen
    from mixture_experts_layer_block_b200.native import MoELayer
    w = configs.TINY
    inp = {k: (v.cuda() if v is not None else None) for k, v in gen.make_inputs(w).items()}
    layer = MoELayer.for_workload(w)
    out = torch.empty((w.T, w.H), device="cuda")
    layer.forward(inp["x"], inp, out)
    tasks = layer.query(3)
    x, wts, _ = _inputs(4, 264, 136, seed=1)
    busy = torch.zeros(1 << 32, dtype=torch.uint8, device="cuda")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    layer.forward(inp["x"][:1].contiguous(), inp, out[:1])
    assert layer.query(3) < tasks
    with torch.cuda.stream(a):
        for _ in range(20):
            busy.add_(1)
    layer.forward(inp["x"], inp, out, stream=a)
    layer.ffn_forward(x, wts, torch.empty_like(x), stream=b)
    assert layer.query(3) == tasks
    torch.cuda.synchronize()
    layer.close()


def _product(a, b, ea=None):
    """a b in fp64, and how far an fp32 sum of the rounded a may be off: additions of zeros are exact, so that only
    the nonzero terms count."""
    terms = (a != 0).double() @ (b != 0).double()
    err = terms * R32 * (a.abs() @ b.abs())
    return a @ b, err if ea is None else err + ea @ b.abs()


@pytest.mark.parametrize("T,H,D", [(1, 1 << 20, 8), (16, 8, 1 << 20), (17, 1 << 20, 8), (40, 8, 1 << 20), (1 << 24, 8, 8),
                                   (1 << 22, 16, 24)])
def test_the_largest_extents(T, H, D):
    """The longest rows, columns and batches that the block takes. What a long sum runs over is mostly zero, at random
    places, so that its bound stays narrow."""
    layer = _layer()
    g = torch.Generator(device="cuda").manual_seed(H + D)

    def r(*shape, keep=1.0, s=1.0):
        v = torch.randn(shape, generator=g, device="cuda") * s
        if keep < 1:
            v *= torch.rand(shape, generator=g, device="cuda") < keep
        return v.to(torch.bfloat16)

    few = 1024.0
    x, dout = (r(T, H, keep=few / H) if H > few else r(T, H) for _ in range(2))
    if T > few:  # whole tokens
        for v in (x, dout):
            v *= (torch.rand(T, 1, generator=g, device="cuda") < few / T).to(torch.bfloat16)
        x[-1], dout[-1] = 1.0, -1.0
    wts = {"Ws_up": r(D, H, s=0.1 if H > few else 0.4), "Ws_gate": r(D, H, s=0.1 if H > few else 0.4),
           "Ws_down": r(H, D, keep=few / D, s=0.1) if D > few else r(H, D, s=0.3)}
    out = torch.empty(T, H, device="cuda")
    u, gate = (torch.empty(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    layer.ffn_forward(x, wts, out, u=u, g=gate)
    assert layer.status() == (0, 0)
    up, gw, down = (wts[n].double() for n in ("Ws_up", "Ws_gate", "Ws_down"))
    xd, dd = x.double(), dout.double()
    ru, eu = _product(xd, up.T)
    rg, eg = _product(xd, gw.T)
    _close(u, ru, eu, "u")
    _close(gate, rg, eg, "g")
    s = torch.sigmoid(ru)
    h = ru * s * rg
    eh = 1.1 * rg.abs() * eu + (ru * s).abs() * eg + eu * eg + ACT * rg.abs() * (1 + ru.abs())
    _close(out, *_product(h, down.T, eh + R16 * (h.abs() + eh)), "out")
    del out, ru, rg, eu, eg, s, h, eh

    grads = {"x": torch.empty_like(x), **{n: torch.empty_like(w, dtype=torch.float32) for n, w in wts.items()}}
    layer.ffn_backward(dout, x, u, gate, wts, grads)
    assert layer.status() == (0, 0)
    ud, gd = u.double(), gate.double()
    s = torch.sigmoid(ud)
    a, da = ud * s, s * (1 + ud * (1 - s))
    dh, e = _product(dd, down)
    act = ACT * (1 + ud.abs())

    def rounded(v, err):
        return v, err + R16 * (v.abs() + err)

    du, edu = rounded(dh * gd * da, e * (gd * da).abs() + (dh.abs() + e) * gd.abs() * act)
    dg, edg = rounded(dh * a, e * a.abs() + (dh.abs() + e) * act)
    h, eh = rounded(a * gd, gd.abs() * act)
    del s, a, da, dh, e, act
    # dx is one sum over both weights
    _close(grads["x"], *_product(torch.cat((du, dg), 1), torch.cat((up, gw)), torch.cat((edu, edg), 1)), "x")
    _close(grads["Ws_up"], *_product(du.T, xd, edu.T), "Ws_up")
    _close(grads["Ws_gate"], *_product(dg.T, xd, edg.T), "Ws_gate")
    ref, err = _product(dd.T, h)
    _close(grads["Ws_down"], ref, err + dd.T.abs() @ eh, "Ws_down")
    layer.close()
