"""Tokens whose router logits are NaN: every choice still names an expert (so that no index leaves its
table), the token's own output is NaN, and the other tokens keep theirs bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("E,k", [(8, 8), (64, 4), (256, 8), (300, 32), (1024, 3)])
def test_choices_name_experts(E, k):
    """NaN comes last, by expert index; the rest as without it."""
    from mixture_experts_layer_block_b200.native import MoELayer
    T = 40
    layer = MoELayer(64, 32, E, k, 16, T)
    g = torch.Generator().manual_seed(E)
    logits = torch.randint(-3, 4, (T, E), generator=g).float()  # ties too
    logits[0] = NAN
    logits[1] = -INF
    logits[2, 1:] = NAN
    logits[3, ::2] = NAN
    logits[4, : E - 1] = NAN
    logits[5] = torch.where(torch.rand(E, generator=g) < 0.5, torch.tensor(NAN), torch.tensor(-INF))
    logits[6, 0] = -NAN
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    layer.gate_topk(logits.cuda(), k, ids, w)
    for t in range(T):
        row = logits[t].tolist()
        order = sorted(range(E), key=lambda e: (row[e] != row[e], 0.0 if row[e] != row[e] else -row[e], e))
        assert ids[t].tolist() == order[:k], t
        best = [row[e] for e in order[:k]]
        assert bool(torch.isnan(w[t]).all()) == (any(v != v for v in best) or best[0] == -INF), t
    layer.close()


@pytest.mark.parametrize("E,k,T,flags", [(16, 4, 12, 0), (16, 4, 12, 1024), (16, 4, 40, 0), (8, 2, 300, 0), (8, 2, 300, 8),
                                         (300, 8, 12, 0), (300, 8, 100, 0)])
def test_layer_forward(E, k, T, flags):
    from mixture_experts_layer_block_b200.native import MoELayer
    H, D, Ds = 256, 128, 128
    g = torch.Generator(device="cuda").manual_seed(E + T)

    def r(*shape, s=0.05):
        return (torch.randn(shape, generator=g, device="cuda") * s).to(torch.bfloat16)

    wts = {"W_router": r(E, H), "W_up": r(E, D, H), "W_gate": r(E, D, H), "W_down": r(E, H, D), "Ws_up": r(Ds, H),
           "Ws_gate": r(Ds, H), "Ws_down": r(H, Ds)}
    layer = MoELayer(H, D, E, k, 16, T, inter_shared=Ds, flags=flags)
    x = r(T, H, s=1.0)
    clean, out = (torch.empty(T, H, device="cuda") for _ in range(2))
    layer.forward(x, wts, clean)
    x[5], x[T - 1, 3] = NAN, NAN
    layer.forward(x, wts, out)
    assert layer.status() == (0, 0)
    keep = [t for t in range(T) if t not in (5, T - 1)]
    assert torch.equal(out[keep], clean[keep])
    assert bool(torch.isnan(out[[5, T - 1]]).all())
    layer.close()


@pytest.mark.parametrize("T", [12, 300])
def test_mxfp8_forward(T):
    """MXFP8 tokens go the same ways; what a NaN becomes in E4M3 is its own."""
    from mixture_experts_layer_block_b200.native import MOE_FLAG_MXFP8, MoELayer
    H, D, E, k = 256, 128, 16, 4
    g = torch.Generator(device="cuda").manual_seed(T)

    def r(*shape, s=0.05):
        return (torch.randn(shape, generator=g, device="cuda") * s).to(torch.bfloat16)

    wts = {"W_router": r(E, H), "W_up": r(E, D, H), "W_gate": r(E, D, H), "W_down": r(E, H, D)}
    layer = MoELayer(H, D, E, k, 16, T, flags=MOE_FLAG_MXFP8)
    wq = layer.quantize_experts_mxfp8(wts)
    x = r(T, H, s=1.0)
    clean, out = (torch.empty(T, H, device="cuda") for _ in range(2))
    layer.forward_mxfp8(x, wts["W_router"], None, wq, clean)
    x[5] = NAN
    layer.forward_mxfp8(x, wts["W_router"], None, wq, out)
    assert layer.status() == (0, 0)
    keep = [t for t in range(T) if t != 5]
    assert torch.equal(out[keep], clean[keep])
    assert bool(torch.isnan(out[5]).all())
    layer.close()


@pytest.mark.parametrize("Ds", [0, 64])
def test_int4_forward(Ds):
    from mixture_experts_layer_block_b200.native import MoELayer
    H, D, E, k, T = 256, 128, 8, 2, 11
    g = torch.Generator(device="cuda").manual_seed(Ds)

    def r(*shape, s=0.05):
        return (torch.randn(shape, generator=g, device="cuda") * s).to(torch.bfloat16)

    wts = {"W_up": r(E, D, H), "W_gate": r(E, D, H), "W_down": r(E, H, D)}
    if Ds:
        wts.update(Ws_up=r(Ds, H), Ws_gate=r(Ds, H), Ws_down=r(H, Ds))
    layer = MoELayer(H, D, E, k, 16, T, inter_shared=Ds)
    wq = layer.quantize_experts_int4(wts, 64)
    wr, x = r(E, H), r(T, H, s=1.0)
    clean, out = (torch.empty(T, H, device="cuda") for _ in range(2))
    layer.forward_int4(x, wr, None, wq, clean)
    x[5], x[9, 1] = NAN, NAN
    layer.forward_int4(x, wr, None, wq, out)
    keep = [t for t in range(T) if t not in (5, 9)]
    assert torch.equal(out[keep], clean[keep])
    assert bool(torch.isnan(out[[5, 9]]).all())
    layer.close()
