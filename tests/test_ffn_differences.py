"""The feed-forward block's gradients against differences of its fp64 loss L = sum(out * dout).

For each input p the change of L along d is compared with sum(grad * d). The direction is the fp64 gradient
itself (by autograd), so that the derivative is the sum of its squares and nothing cancels; the bound is taken
from the reference, not from the gradient under test.

The bound is derived. x and the up and gate weights lie on grids on which u and g are whole numbers of 1/8
below 32: bf16 holds them exactly (8 bits), so that the saved pre-activations are the true ones. What is rounded:
 - h, du and dg once to bf16: each is off by at most 2^-8 of itself, besides the error of what it is made of: dh's
   fp32 sum of H products (H 2^-23 of their magnitudes) and the activation's intrinsics (2^-18 of its factors);
 - a gradient once, where it is bf16: 2^-8 of itself; and its fp32 sums, K 2^-23 of their magnitudes.
All of it enters sum(grad * d) linearly: an error e[t, j] of du moves sum(dW_up * d) by e[t, j] (x d^T)[t, j].
The central difference's own error, (step of 1e-4 of the largest entry)^2 of third derivatives, is far below.
"""
import pytest
import torch

R16, R32, ACT = 2.0 ** -8, 2.0 ** -23, 2.0 ** -18
NAMES = ("x", "Ws_up", "Ws_gate", "Ws_down")


def _inputs(T, H, D, seed, device):
    g = torch.Generator().manual_seed(seed)

    def r(*shape, s=1.0):
        return (torch.randn(shape, generator=g) * s).to(torch.bfloat16)

    def grid(*shape, most, step):
        return (torch.randint(-most, most + 1, shape, generator=g) * step).to(torch.bfloat16)

    p = {"x": grid(T, H, most=1, step=1.0), "Ws_up": grid(D, H, most=1, step=0.125), "Ws_gate": grid(D, H, most=1, step=0.125),
         "Ws_down": r(H, D, s=D ** -0.5)}
    return {n: v.to(device) for n, v in p.items()}, r(T, H).to(device)


def _pre(p):
    """u and g, exact in bf16."""
    u, g = p["x"].double() @ p["Ws_up"].double().T, p["x"].double() @ p["Ws_gate"].double().T
    assert torch.equal(u.bfloat16().double(), u) and torch.equal(g.bfloat16().double(), g)
    return u, g


def _loss(p, dout):
    u, g = p["x"] @ p["Ws_up"].T, p["x"] @ p["Ws_gate"].T
    return ((u * torch.sigmoid(u) * g) @ p["Ws_down"].T * dout).sum()


def _directions(p, dout):
    at = {n: p[n].double().requires_grad_(True) for n in NAMES}
    return dict(zip(NAMES, torch.autograd.grad(_loss(at, dout.double()), [at[n] for n in NAMES])))


def _allowed(n, d, p, dout, u, g, bf16):
    """How far sum(grad * d) may be from the derivative of L along d."""
    x, up, gate, down, dout = (v.double() for v in (*(p[m] for m in NAMES), dout))
    (T, H), D = x.shape, up.shape[0]
    s = torch.sigmoid(u)
    a, da = u * s, s * (1 + u * (1 - s))
    dh = dout @ down
    e = H * R32 * (dout.abs() @ down.abs())
    act = ACT * (1 + u.abs())

    def rounded(v, err):
        return err + R16 * (v.abs() + err)

    edu = rounded(dh * g * da, e * (g * da).abs() + (dh.abs() + e) * g.abs() * act)
    edg = rounded(dh * a, e * a.abs() + (dh.abs() + e) * act)
    eh = rounded(a * g, g.abs() * act)
    if n == "x":
        grad = (dh * g * da) @ up + (dh * a) @ gate
        out = (edu * (d @ up.T).abs()).sum() + (edg * (d @ gate.T).abs()).sum()
        sums = 2 * D * R32 * ((dh * g * da).abs() @ up.abs() + (dh * a).abs() @ gate.abs())
    elif n == "Ws_down":
        grad = dout.T @ (a * g)
        out = (eh * (dout @ d).abs()).sum()
        sums = T * R32 * (dout.abs().T @ (a * g).abs())
    else:
        v, ev = (dh * g * da, edu) if n == "Ws_up" else (dh * a, edg)
        grad = v.T @ x
        out = (ev * (x @ d.T).abs()).sum()
        sums = T * R32 * (v.abs().T @ x.abs())
    out = out + (sums * d.abs()).sum()
    if bf16:
        out = out * (1 + R16) + R16 * (grad * d).abs().sum()
    return float(out)


def _wrong(grads, p, dout):
    """{input: (distance of sum(grad * d) from the difference, what is allowed)} of the gradients given."""
    u, g = _pre(p)
    at = {n: p[n].double() for n in NAMES}
    result = {}
    for n, d in _directions(p, dout).items():
        step = 1e-4 / float(d.abs().max())
        diff = float(_loss({**at, n: at[n] + step * d}, dout.double()) - _loss({**at, n: at[n] - step * d}, dout.double())) / (2 * step)
        got = float((grads[n].double() * d).sum())
        result[n] = (abs(got - diff), _allowed(n, d, p, dout, u, g, grads[n].dtype == torch.bfloat16) + 1e-6 * abs(diff))
    return result


def _formula(p, dout, u, g, dtype, da=None, drop=False, half=1.0):
    """The gradients as the kernels round them, with a mistake if one is asked for."""
    x, up, gate, down, dout = (v.double() for v in (*(p[m] for m in NAMES), dout))
    s = torch.sigmoid(u)
    dh = dout @ down
    du = (dh * g * (s * (1 + u * (1 - s)) if da is None else da(u))).bfloat16().double()
    dg = (dh * u * s).bfloat16().double()
    h = (u * s * g).bfloat16().double()
    return {"x": (du @ up + (0 if drop else dg @ gate)).to(torch.bfloat16), "Ws_up": (half * du.T @ x).to(dtype), "Ws_gate": (dg.T @ x).to(dtype),
            "Ws_down": (dout.T @ h).to(dtype)}


SHAPES = [(40, 136, 72), (9, 72, 136), (150, 264, 200)]


@pytest.mark.parametrize("T,H,D", SHAPES)
def test_the_check_passes_the_formula_and_fails_mistakes(T, H, D):
    """The bound is narrow enough to tell the gradients from near misses, in each input that they touch."""
    p, dout = _inputs(T, H, D, T, "cpu")
    u, g = _pre(p)
    for dtype in (torch.float32, torch.bfloat16):
        assert all(off <= most for off, most in _wrong(_formula(p, dout, u, g, dtype), p, dout).values())
        for kw, hurt in ((dict(drop=True), ("x",)),                                    # dx without the gate's term
                         (dict(da=torch.sigmoid), ("x", "Ws_up")),                    # the derivative's second term left out
                         (dict(da=lambda u: torch.sigmoid(u) * (1 + u)), ("x", "Ws_up")),  # its last factor left out
                         (dict(half=0.98), ("Ws_up",))):                               # two percent too small
            wrong = _wrong(_formula(p, dout, u, g, dtype, **kw), p, dout)
            assert all(wrong[n][0] > wrong[n][1] for n in hurt), (kw, wrong)
        other = _formula(p, dout, u, g, dtype)
        other["Ws_gate"] = other["Ws_gate"][torch.randperm(D, generator=torch.Generator().manual_seed(1))]
        off, most = _wrong(other, p, dout)["Ws_gate"]
        assert off > most


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,D", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients(T, H, D, dtype):
    from mixture_experts_layer_block_b200.native import MoELayer
    layer = MoELayer(256, 128, 8, 2, 16, 16)
    p, dout = _inputs(T, H, D, T, "cuda")
    wts = {n: p[n] for n in NAMES[1:]}
    u, g = (torch.empty(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    layer.ffn_forward(p["x"], wts, torch.empty_like(p["x"]), u=u, g=g)
    ru, rg = _pre(p)
    assert torch.equal(u.double(), ru) and torch.equal(g.double(), rg)  # sums of 1/8s: exact in fp32 too
    grads = {"x": torch.empty_like(p["x"]), **{n: torch.empty_like(w, dtype=dtype) for n, w in wts.items()}}
    layer.ffn_backward(dout, p["x"], u, g, wts, grads)
    wrong = _wrong(grads, p, dout)
    assert all(off <= most for off, most in wrong.values()), wrong
    assert layer.status() == (0, 0)
    layer.close()
