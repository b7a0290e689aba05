"""4-bit weights on the GPU: the quantiser and the layout bit for bit, and the products (one matrix,
the routed experts, the whole layer for a decode batch) against fp64 of the same quantised values.

Bounds are derived: a rounding to bf16 is off by at most 2^-8 of the value; an fp32 sum of K
products by at most K 2^-23 of the sum of their magnitudes (twice the bound of rounding to nearest,
for additions that truncate; the group scales' multiplications, one per 32 columns or more, are
within it too); the activation by 2^-18 |g| (1 + |u|), as for the bf16 block. Codes less their zero points
are exact in bf16, so nothing else is rounded.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

R16 = 2.0 ** -8
R32 = 2.0 ** -23
ACT = 2.0 ** -18


def _layer(H=256, D=128, E=8, k=2, T=16, **kw):
    from mixture_experts_layer_block_b200.native import MoELayer
    return MoELayer(H, D, E, k, 16, T, **kw)


def _checkpoint(R, K, group, zeros, seed):
    """Codes two to a byte, bf16 scales and zero points, with every code and extreme among them."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 16, (R, K), generator=g, dtype=torch.uint8)
    G = -(-K // group)
    s = (torch.rand(R, G, generator=g) * 0.9 + 0.1).mul(2.0 / K ** 0.5).to(torch.bfloat16)
    s[R // 2] *= -1  # a negative scale is a scale
    z = torch.randint(0, 16, (R, G), generator=g, dtype=torch.uint8) if zeros else None
    return q, s, z


def _values(q, s, z, group):
    at = torch.arange(q.shape[1]) // group
    return (q.double() - (8.0 if z is None else z.double()[:, at])) * s.double()[:, at]


def _pack(layer, q, s, z, group):
    p = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
    return layer.pack_int4(p.cuda(), s.cuda(), None if z is None else z.cuda(), group)


def _unpack(m):
    """(codes [R, K], scales [R, G] as bf16 bits, zeros [R, G] or None) by the header's layout."""
    R, K, G = m.rows, m.cols, -(-m.cols // m.group)
    nb = 2 * -(-K // 128)
    w = m.codes.cpu().numpy().view(np.uint32).reshape(-1, nb, 8, 4, 2, 2)  # tile, half block, i, j, h, m
    code = np.zeros((w.shape[0], 16, nb, 64), dtype=np.uint8)
    where = [(0, 0), (8, 0), (0, 2), (8, 2), (0, 1), (8, 1), (0, 3), (8, 3)]
    for i in range(8):
        for j in range(4):
            for h in range(2):
                for mm in range(2):
                    for n, (dr, dk) in enumerate(where):
                        code[:, i + dr, :, 32 * h + 8 * j + 4 * mm + dk] = w[:, :, i, j, h, mm] >> (4 * n) & 15
    code = code.reshape(-1, nb * 64)
    N = 128 // m.group
    e = m.scales.cpu().numpy().view(np.uint32 if m.zeros else np.uint16).reshape(-1, 16 * N * (nb // 2))
    r, g = np.arange(16)[:, None], np.arange(G)[None, :]
    rows = e[:, 16 * N * (g // N) + 2 * N * (r % 8) + 2 * (g % N) + r // 8].reshape(-1, G)
    zero = None
    if m.zeros:
        zero = torch.from_numpy((rows >> 16).astype(np.uint16).view(np.int16)).view(torch.bfloat16).float().numpy() - 128
    return code, (rows & 0xffff).astype(np.uint16), zero


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("R,K", [(1, 8), (16, 64), (33, 328), (130, 2056)])
def test_pack_layout(R, K, group, zeros):
    layer = _layer()
    q, s, z = _checkpoint(R, K, group, zeros, seed=R + K)
    code, sb, zero = _unpack(_pack(layer, q, s, z, group))
    np.testing.assert_array_equal(code[:R, :K], q.numpy())
    assert not code[R:].any() and not code[:, K:].any()
    np.testing.assert_array_equal(sb[:R], s.view(torch.int16).numpy().view(np.uint16))
    if zeros:
        np.testing.assert_array_equal(zero[:R], z.numpy())
    layer.close()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("R,K", [(3, 8), (48, 1024), (50, 2088)])
def test_quantize_bit_for_bit(R, K, group, zeros):
    layer = _layer()
    g = torch.Generator().manual_seed(R * K + group)
    G = -(-K // group)
    v = torch.randn(R, K, generator=g) * torch.exp2(torch.randint(-60, 60, (R, 1), generator=g).float())
    v[0, :] = 0.0                  # a row of zeros
    v[1, : min(K, 40)] = 1e-39     # scales that underflow or nearly do
    v[2] = v[2].abs()              # one sign
    v = v.to(torch.bfloat16)
    m = layer.quantize_int4(v.cuda(), group, zeros)
    code, sb, zero = _unpack(m)
    f = torch.zeros(R, G * group)
    f[:, :K] = v.float()
    f = f.view(R, G, group)
    mn, mx = f.amin(2).clamp(max=0), f.amax(2).clamp(min=0)
    s = ((mx - mn) / 15 if zeros else f.abs().amax(2) / 7).to(torch.bfloat16)
    sf = s.float()
    ok = sf > 0
    z = torch.where(ok, torch.round(-mn / sf).clamp(0, 15), torch.tensor(8.0)) if zeros else torch.full_like(sf, 8.0)
    q = torch.where(ok[..., None], (torch.round(f / sf[..., None]) + z[..., None]).clamp(0, 15), torch.tensor(8.0))
    np.testing.assert_array_equal(sb[:R], s.view(torch.int16).numpy().view(np.uint16))
    np.testing.assert_array_equal(code[:R, :K], q.view(R, -1)[:, :K].numpy())
    if zeros:
        np.testing.assert_array_equal(zero[:R], z.numpy())
    layer.close()


def _close(got, ref, err, name=""):
    err = err + (R16 * (ref.abs() + err) if got.dtype == torch.bfloat16 else 0) + 1e-30
    bad = ~((got.double() - ref).abs() <= err)
    assert not bool(bad.any()), (name, int(bad.sum()), float(((got.double() - ref).abs() / err).max()))


@pytest.mark.parametrize("T", [1, 2, 8, 9, 16, 37])
@pytest.mark.parametrize("R,K,group,zeros", [(1, 8, 32, False), (40, 72, 64, True), (257, 2056, 128, False),
                                             (512, 1024, 32, True), (2048, 328, 128, True), (4800, 520, 64, False),
                                             (17, 7168, 32, False)])
def test_matvec(T, R, K, group, zeros):
    layer = _layer()
    q, s, z = _checkpoint(R, K, group, zeros, seed=R)
    m = _pack(layer, q, s, z, group)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).cuda()
    w = _values(q, s, z, group).cuda()
    ref = x.double() @ w.T
    err = (K + 8) * R32 * (x.double().abs() @ w.abs().T)
    for dtype in (torch.float32, torch.bfloat16):
        buf = torch.full((T + 2, R), 7.0, dtype=dtype, device="cuda")
        layer.matvec_int4(x, m, buf[1:T + 1])
        _close(buf[1:T + 1], ref, err)
        assert bool((buf[0] == 7).all()) and bool((buf[T + 1] == 7).all())
    layer.close()


def _experts(H, D, E, Ds, group, zeros, seed, layer):
    shapes = {"W_up": (E * D, H), "W_gate": (E * D, H), "W_down": (E * H, D)}
    if Ds:
        shapes.update(Ws_up=(Ds, H), Ws_gate=(Ds, H), Ws_down=(H, Ds))
    val, packed = {}, {}
    for i, (n, (R, K)) in enumerate(shapes.items()):
        q, s, z = _checkpoint(R, K, group, zeros, seed + i)
        packed[n] = _pack(layer, q, s, z, group)
        val[n] = _values(q, s, z, group).cuda()
    return val, packed


def _block(x, up, gate, down):
    """(W_down SwiGLU(W_up x, W_gate x), its error bound) of one token in fp64."""
    H, D = up.shape[1], up.shape[0]
    u, g = up @ x, gate @ x
    eu, eg = H * R32 * (up.abs() @ x.abs()), H * R32 * (gate.abs() @ x.abs())
    s = torch.sigmoid(u)
    h = u * s * g
    eh = 1.1 * g.abs() * eu + (u * s).abs() * eg + eu * eg + ACT * g.abs() * (1 + u.abs())
    eh = eh + R16 * (h.abs() + eh)
    return down @ h, down.abs() @ eh + (D + 8) * R32 * (down.abs() @ h.abs())


def _reference(x, ids, w, val, H, D, E, Ds):
    T, k = ids.shape
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    err, size = torch.zeros_like(out), torch.zeros_like(out)
    for t in range(T):
        terms = [(int(e), float(p)) for e, p in zip(ids[t].tolist(), w[t].tolist()) if 0 <= e < E]
        for e, p in terms:
            y, ey = _block(x[t].double(), val["W_up"][e * D:(e + 1) * D], val["W_gate"][e * D:(e + 1) * D],
                           val["W_down"][e * H:(e + 1) * H])
            out[t] += p * y
            err[t] += abs(p) * ey
            size[t] += abs(p) * y.abs()
        if Ds:
            y, ey = _block(x[t].double(), val["Ws_up"], val["Ws_gate"], val["Ws_down"])
            out[t] += y
            err[t] += ey
            size[t] += y.abs()
    return out, err + (k + 16) * R32 * size


CASES = [(1, 256, 128, 8, 2, 0, 128, False), (16, 256, 128, 8, 2, 64, 32, True), (7, 272, 48, 5, 3, 0, 64, False),
         (16, 528, 272, 300, 8, 144, 128, True), (9, 1024, 512, 32, 32, 0, 32, False), (8, 64, 1040, 3, 1, 0, 64, True),
         # long sums of few output tiles; more tiles than SMs, unevenly; every expert with more than 8 tokens
         (16, 272, 1040, 8, 8, 0, 64, False), (16, 2560, 512, 24, 8, 272, 128, True), (7, 4816, 528, 16, 16, 0, 32, False),
         # the smallest sizes
         (1, 16, 16, 1, 1, 0, 32, True), (16, 16, 32, 2, 2, 16, 128, False),
         # the most slots and experts
         (16, 64, 32, 1024, 32, 16, 64, False), (8, 64, 32, 1024, 32, 0, 32, True)]


@pytest.mark.parametrize("T,H,D,E,k,Ds,group,zeros", CASES)
def test_experts(T, H, D, E, k, Ds, group, zeros):
    layer = _layer(H, D, E, k, inter_shared=Ds)
    val, packed = _experts(H, D, E, Ds, group, zeros, H + D, layer)
    g = torch.Generator().manual_seed(T * E)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).cuda()
    w = torch.softmax(torch.randn(T, k, generator=g), 1).cuda()
    ref, err = _reference(x, ids, w, val, H, D, E, Ds)
    for dtype in (torch.float32, torch.bfloat16):
        buf = torch.full((T + 2, H), 7.0, dtype=dtype, device="cuda")
        layer.experts_int4(x, ids, w, packed, buf[1:T + 1])
        _close(buf[1:T + 1], ref, err)
        assert bool((buf[0] == 7).all()) and bool((buf[T + 1] == 7).all())
        again = torch.empty(T, H, dtype=dtype, device="cuda")
        layer.experts_int4(x, ids, w, packed, again)
        assert torch.equal(again, buf[1:T + 1])
    layer.close()


@pytest.mark.parametrize("Ds", [0, 64])
def test_experts_with_dropped_and_repeated_slots(Ds):
    """Ids outside [0, E) contribute nothing (a token may have none left), an expert named twice by a
    token counts twice, and one expert may take every token."""
    T, H, D, E, k = 12, 256, 128, 8, 4
    layer = _layer(H, D, E, k, inter_shared=Ds)
    val, packed = _experts(H, D, E, Ds, 64, True, 5, layer)
    g = torch.Generator().manual_seed(9)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    w = torch.rand(T, k, generator=g).cuda()
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    ids[0] = -1
    ids[1] = torch.tensor([3, 3, 3, 3])
    ids[2] = torch.tensor([E, 2, -5, 2 ** 30])
    ids[3:, 0] = 6
    ids = ids.cuda()
    out = torch.full((T, H), float("nan"), device="cuda")
    layer.experts_int4(x, ids, w, packed, out)
    ref, err = _reference(x, ids, w, val, H, D, E, Ds)
    _close(out, ref, err)
    if not Ds:
        assert bool((out[0] == 0).all())
    ids.fill_(-1)  # nobody hits anything
    layer.experts_int4(x, ids, w, packed, out)
    ref, err = _reference(x, ids, w, val, H, D, E, Ds)
    _close(out, ref, err)
    layer.close()


def test_bad_values_stay_with_their_token_and_expert():
    """A NaN token spoils its own row; an expert whose scales are infinite spoils only the tokens that
    it serves."""
    T, H, D, E, k = 10, 256, 128, 6, 2
    layer = _layer(H, D, E, k)
    val, packed = _experts(H, D, E, 0, 32, False, 50, layer)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    ids = torch.stack([torch.randperm(E - 1, generator=g)[:k] for _ in range(T)]).to(torch.int32).cuda()
    ids[4, 1] = E - 1
    w = torch.rand(T, k, generator=g).cuda()
    clean = torch.empty(T, H, device="cuda")
    layer.experts_int4(x, ids, w, packed, clean)
    x2 = x.clone()
    x2[7, 3] = float("nan")
    q, s, z = _checkpoint(E * D, H, 32, False, 50)
    s[(E - 1) * D:] = float("inf")
    bad = dict(packed, W_up=_pack(layer, q, s, z, 32))
    out = torch.empty(T, H, device="cuda")
    layer.experts_int4(x2, ids, w, bad, out)
    keep = [t for t in range(T) if t not in (4, 7)]
    assert torch.equal(out[keep], clean[keep])
    assert bool(torch.isnan(out[7]).any()) and not bool(torch.isfinite(out[4]).all())
    layer.close()


@pytest.mark.parametrize("flags,bias,cf", [(0, True, 0.0), (32, False, 0.0), (0, True, 1.0)])
@pytest.mark.parametrize("T", [1, 11, 16])
def test_forward_int4(T, flags, bias, cf):
    """The layer: routing as moe_router_logits and moe_gate_topk give it, then the experts; with a
    capacity, an expert takes its lowest tokens only."""
    H, D, E, k, Ds = 256, 128, 8, 2, 64
    layer = _layer(H, D, E, k, inter_shared=Ds, flags=flags, capacity_factor=cf)
    val, packed = _experts(H, D, E, Ds, 128, False, 70, layer)
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    wr = (torch.randn(E, H, generator=g) * 0.1).to(torch.bfloat16).cuda()
    b = torch.randn(E, generator=g).cuda() if bias else None
    out = torch.empty(T, H, dtype=getattr(torch, layer.out_dtype), device="cuda")
    layer.forward_int4(x, wr, b, packed, out)
    logits = torch.empty(T, E, device="cuda")
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    layer.router_logits(x, wr, b, logits)
    layer.gate_topk(logits, k, ids, w)
    if cf:
        cap = -(-T * k // E)
        kept = ids.cpu().clone()
        for e in range(E):
            hit = [(t, j) for t in range(T) for j in range(k) if int(ids[t, j]) == e]
            for t, j in hit[cap:]:
                kept[t, j] = -1
        ids = kept.cuda()
    ref, err = _reference(x, ids, w, val, H, D, E, Ds)
    # the K-split router of the forward and the stage call's differ in the logits' last bits:
    # an fp32 dot product's bound (H 2^-23 of its terms' magnitudes, both sides) moves a softmax
    # weight by at most twice that of itself
    el = 4 * H * R32 * float((x.double().abs() @ wr.double().abs().T).max())
    err = err + 2 * el * sum(v.abs() for v in [ref]) + 2 * el * _reference(x, ids, w.abs(), val, H, D, E, 0)[0].abs()
    _close(out, ref, err)
    assert layer.status() == (0, 0)
    layer.close()


def test_forward_int4_close_to_the_bf16_layer():
    """Quantise the layer's experts and run both: the 4-bit layer is the bf16 layer on rounded
    weights, so it equals a bf16 forward of the dequantised weights (exact in bf16 here: power-of-two
    scales) up to the bf16 path's own roundings."""
    H, D, E, k, T = 256, 128, 8, 2, 16
    layer = _layer(H, D, E, k, flags=1024)
    g = torch.Generator().manual_seed(4)
    wts, packed = {}, {}
    for n, (R, K, s3) in {"W_up": (E * D, H, (E, D, H)), "W_gate": (E * D, H, (E, D, H)), "W_down": (E * H, D, (E, H, D))}.items():
        q = torch.randint(0, 16, (R, K), generator=g, dtype=torch.uint8)
        s = torch.full((R, -(-K // 64)), 2.0 ** -6).to(torch.bfloat16)
        packed[n] = _pack(layer, q, s, None, 64)
        wts[n] = _values(q, s, None, 64).to(torch.bfloat16).cuda().view(s3)
    wts["W_router"] = (torch.randn(E, H, generator=g) * 0.1).to(torch.bfloat16).cuda()
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    a, b = torch.empty(T, H, device="cuda"), torch.empty(T, H, device="cuda")
    layer.forward(x, wts, a)
    layer.forward_int4(x, wts["W_router"], None, packed, b)
    d = layer.router_logits(x, wts["W_router"], None, torch.empty(T, E, device="cuda"))
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    layer.gate_topk(d, k, ids, w)
    val = {n: wts[n].double().view(-1, wts[n].shape[-1]) for n in ("W_up", "W_gate", "W_down")}
    ref, err = _reference(x, ids, w, val, H, D, E, 0)
    size = _reference(x, ids, w.abs(), val, H, D, E, 0)[1]
    el = 4 * H * R32 * float((x.double().abs() @ wts["W_router"].double().abs().T).max())
    slack = 2 * el * (ref.abs() + size) + 1e-6
    assert bool(((b.double() - ref).abs() <= err + slack).all())
    assert bool(((a.double() - ref).abs() <= err + slack + 2 * R16 * (ref.abs() + err) + R16 * size).all())
    layer.close()


def test_captured_and_replayed_on_another_stream():
    T, H, D, E, k = 6, 256, 128, 16, 4
    layer = _layer(H, D, E, k)
    _, packed = _experts(H, D, E, 0, 128, False, 7, layer)
    wr = torch.randn(E, H).mul(0.1).to(torch.bfloat16).cuda()
    x = torch.randn(T, H).to(torch.bfloat16).cuda()
    out, one, ref, ref1 = (torch.empty(T, H, device="cuda") for _ in range(4))
    one = torch.empty(T, E * D, device="cuda")
    ref1 = torch.empty_like(one)
    layer.forward_int4(x, wr, None, packed, out)
    layer.matvec_int4(x, packed["W_up"], one)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward_int4(x, wr, None, packed, out)
        layer.matvec_int4(x, packed["W_up"], one)
    for seed in (1, 2):
        x.copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        layer.forward_int4(x, wr, None, packed, ref, stream=s)
        layer.matvec_int4(x, packed["W_up"], ref1, stream=s)
        s.synchronize()
        assert torch.equal(out, ref) and torch.equal(one, ref1)
    layer.close()


def test_weights_packed_right_before_they_are_read():
    """Laying out, quantising and reading follow one another on a stream: no product sees the buffers
    of the matrix before."""
    layer = _layer()
    R, K, T = 2048, 512, 4
    x = torch.randn(T, K).to(torch.bfloat16).cuda()
    out = torch.empty(T, R, device="cuda")
    got, refs = [], []
    mats = [torch.randn(R, K, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda() for i in range(4)]
    for m in mats:
        got.append(layer.matvec_int4(x, layer.quantize_int4(m, 64), torch.empty_like(out)))
    torch.cuda.synchronize()
    for m in mats:
        w = layer.quantize_int4(m, 64)
        torch.cuda.synchronize()
        refs.append(layer.matvec_int4(x, w, torch.empty_like(out)))
    for a, b in zip(got, refs):
        assert torch.equal(a, b)
    layer.close()


def test_no_tokens():
    layer = _layer()
    _, packed = _experts(256, 128, 8, 0, 64, False, 3, layer)
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(0, 256, device="cuda")
    layer.matvec_int4(x, packed["W_up"], torch.empty(0, 8 * 128, device="cuda"))
    layer.experts_int4(x, torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda"), packed, out)
    layer.forward_int4(x, torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda"), None, packed, out)
    layer.close()


def test_layer_forwards_beside_4_bit_calls():
    """The bf16 forwards (fused and separate kernels) give the same bits before and after 4-bit calls of
    the same handle, and the intermediates that those overwrite are not offered."""
    from mixture_experts_layer_block_b200 import native
    H, D, E, k, Ds = 256, 128, 8, 2, 64
    g = torch.Generator().manual_seed(8)

    def r(*shape, s=0.05):
        return (torch.randn(shape, generator=g) * s).to(torch.bfloat16).cuda()

    wts = {"W_router": r(E, H), "W_up": r(E, D, H), "W_gate": r(E, D, H), "W_down": r(E, H, D), "Ws_up": r(Ds, H),
           "Ws_gate": r(Ds, H), "Ws_down": r(H, Ds)}
    for flags in (0, native.MOE_FLAG_UNFUSED_SMALL):
        layer = native.MoELayer(H, D, E, k, 16, 64, inter_shared=Ds, flags=flags)
        wq = layer.quantize_experts_int4(wts, 32, True)
        for T in (5, 16, 50):
            x = r(T, H, s=1.0)
            a, b, c = (torch.empty(T, H, device="cuda") for _ in range(3))
            layer.forward(x, wts, a)
            layer.debug_outputs(T, k, "cuda")
            few = min(T, 16)
            layer.forward_int4(x[:few].contiguous(), wts["W_router"], None, wq, c[:few])
            with pytest.raises(native.MoEError) as err:
                layer.debug_outputs(T, k, "cuda")
            assert err.value.code == native.MOE_ERR_NOT_READY
            layer.forward(x, wts, b)
            assert torch.equal(a, b)
            # 4-bit weights are near the bf16 ones: half a step of each (a 30th of a group's spread) leaves
            # the layer's output well inside its own size
            assert float((c[:few] - a[:few]).norm()) < 0.5 * float(a[:few].norm())
        with pytest.raises(native.MoEError) as err:
            layer.forward_int4(r(17, H), wts["W_router"], None, wq, torch.empty(17, H, device="cuda"))
        assert err.value.code == native.MOE_ERR_UNSUPPORTED
        assert layer.status() == (0, 0)
        layer.close()


def test_offsets_past_32_bits():
    """Experts and rows whose codes lie more than 2^32 bytes into their buffers."""
    H, D, E, k, T = 7168, 2048, 640, 2, 3  # 4.7 GB of codes a matrix
    layer = _layer(H, D, E, k)
    g = torch.Generator(device="cuda").manual_seed(1)
    packed, kept = {}, {}
    some = [0, 300, 584, 638, 639]
    for n, (R, K) in {"W_up": (E * D, H), "W_gate": (E * D, H), "W_down": (E * H, D)}.items():
        q = torch.randint(0, 256, (R, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s = (torch.rand(R, K // 128, generator=g, device="cuda") + 0.5).mul(0.3 / K ** 0.5).to(torch.bfloat16)
        packed[n] = layer.pack_int4(q, s, None, 128)
        rows = R // E
        kept[n] = {e: _values(torch.stack((q[e * rows:(e + 1) * rows] & 15, q[e * rows:(e + 1) * rows] >> 4), 2).flatten(1).cpu(),
                              s[e * rows:(e + 1) * rows].cpu(), None, 128).cuda() for e in some}
        del q, s
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.tensor([[0, 639], [638, 300], [584, 639]], dtype=torch.int32, device="cuda")
    w = torch.rand(T, k, generator=g, device="cuda")
    out = torch.empty(T, H, device="cuda")
    layer.experts_int4(x, ids, w, packed, out)
    for t in range(T):
        ref, err = 0, 0
        for j in range(k):
            e, p = int(ids[t, j]), float(w[t, j])
            y, ey = _block(x[t].double(), kept["W_up"][e], kept["W_gate"][e], kept["W_down"][e])
            ref, err = ref + p * y, err + p * ey + 18 * R32 * p * y.abs()
        _close(out[t], ref, err)
    one = torch.empty(T, E * D, device="cuda")
    layer.matvec_int4(x, packed["W_up"], one)
    for e in some:
        ref = x.double() @ kept["W_up"][e].T
        _close(one[:, e * D:(e + 1) * D], ref, (H + 8) * R32 * (x.double().abs() @ kept["W_up"][e].abs().T))
    layer.close()


def test_overlapping_results_are_refused():
    from mixture_experts_layer_block_b200 import native
    H, D, E, k, T = 64, 32, 4, 2, 8
    layer = _layer(H, D, E, k)
    _, packed = _experts(H, D, E, 0, 64, True, 5, layer)
    buf = torch.randn(2 * T, H, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    x, ids = buf[:T], torch.tensor([[0, 1]] * T, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 0.5, device="cuda")
    router = torch.zeros(E, H, dtype=torch.bfloat16, device="cuda")
    for out in (x, buf[1:T + 1], buf[T - 1:2 * T - 1]):
        with pytest.raises(native.MoEError) as err:
            layer.experts_int4(x, ids, w, packed, out)
        assert err.value.code == native.MOE_ERR_INVALID_ARG
    with pytest.raises(native.MoEError) as err:
        layer.forward_int4(x, router, None, packed, buf.view(torch.float32).view(T, H))
    assert err.value.code == native.MOE_ERR_INVALID_ARG
    ref, out = torch.empty_like(x), buf[T:]
    layer.experts_int4(x, ids, w, packed, ref)
    layer.experts_int4(x, ids, w, packed, out)  # side by side is not overlapping
    assert torch.equal(out, ref)
    square = layer.quantize_int4(torch.randn(H, H, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda(), 64)
    with pytest.raises(native.MoEError) as err:
        layer.matvec_int4(x, square, x)
    assert err.value.code == native.MOE_ERR_INVALID_ARG
    layer.matvec_int4(x, square, out)
    layer.matvec_int4(x, square, ref)
    assert torch.equal(out, ref)
    layer.close()


@pytest.mark.parametrize("first", [False, True])
def test_forward_after_a_wait_that_ran_out(first):
    """A wait of a bf16 forward runs out (stalled on the host's request). Once the status has said so, a
    4-bit forward of the handle is the one that any other handle computes, whether its long router sum (4096 blocks of
    64, which outlasts the first looks at its barriers) is the first that the handle computes or not."""
    from mixture_experts_layer_block_b200.native import MOE_ERR_DEVICE_TIMEOUT
    H, D, E, k, T = 1 << 18, 16, 4, 1, 16
    g = torch.Generator(device="cuda").manual_seed(21)

    def r(*shape, s=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * s).to(torch.bfloat16)

    wts = {"W_router": r(E, H, s=H ** -0.5), "W_up": r(E, D, H, s=H ** -0.5), "W_gate": r(E, D, H, s=H ** -0.5),
           "W_down": r(E, H, D, s=0.25)}
    layer, other = (_layer(H, D, E, k, T=40, timeout_ns=limit) for limit in (50_000_000, 0))
    packed = other.quantize_experts_int4(wts, 64)
    x, before = r(T, H), r(40, H)
    ref, out = (torch.empty(T, H, device="cuda") for _ in range(2))
    other.forward_int4(x, wts["W_router"], None, packed, ref)
    assert other.status() == (0, 0)
    if not first:
        layer.forward_int4(x.neg(), wts["W_router"], None, packed, out)
    layer.inject_stall(1)
    layer.forward(before, wts, torch.empty(40, H, device="cuda"))
    rc, st = layer.status()
    assert rc == MOE_ERR_DEVICE_TIMEOUT and st & (1 << 30)
    for _ in range(2):
        out.fill_(float("nan"))
        layer.forward_int4(x, wts["W_router"], None, packed, out)
        assert layer.status() == (0, 0)
        assert torch.equal(out, ref)
    layer.close()
    other.close()


def test_forward_whose_own_wait_runs_out():
    """A limit that the router's sum cannot keep: each 4-bit forward ends, and each is reported."""
    from mixture_experts_layer_block_b200.native import MOE_ERR_DEVICE_TIMEOUT
    H, D, E, k, T = 1 << 18, 16, 4, 1, 16
    layer = _layer(H, D, E, k, timeout_ns=1_000)
    _, packed = _experts(H, D, E, 0, 128, False, 90, layer)
    x = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    wr = torch.ones(E, H, dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        layer.forward_int4(x, wr, None, packed, torch.empty(T, H, device="cuda"))
        rc, st = layer.status()
        assert rc == MOE_ERR_DEVICE_TIMEOUT and st & (1 << 30)
        assert layer.status() == (0, 0)
    layer.close()


@pytest.mark.parametrize("Ds", [0, 32])
def test_results_inside_the_weights_are_refused(Ds):
    """A result that lies inside any matrix of the experts, or begins or ends in the router's weights or the bias,
    is refused before anything is written."""
    from mixture_experts_layer_block_b200 import native
    H, D, E, k, T = 64, 32, 4, 2, 2
    layer = _layer(H, D, E, k, inter_shared=Ds)
    _, packed = _experts(H, D, E, Ds, 64, True, 15, layer)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    ids, w = torch.tensor([[0, 1]] * T, dtype=torch.int32, device="cuda"), torch.full((T, k), 0.5, device="cuda")
    big = torch.randn(64 * E * H, generator=g).cuda()
    router, bias = big[:E * H // 2].view(torch.bfloat16).view(E, H), big[E * H:E * H + E]
    kept = {n: (m.codes.clone(), m.scales.clone()) for n, m in packed.items()}
    before = big.clone()

    def refused(call):
        with pytest.raises(native.MoEError) as err:
            call()
        assert err.value.code == native.MOE_ERR_INVALID_ARG

    for m in packed.values():
        for buf in (m.codes, m.scales):
            out = buf[:2 * T * H].view(torch.bfloat16).view(T, H)
            refused(lambda: layer.experts_int4(x, ids, w, packed, out))
            if buf.numel() >= 4 * T * H:
                out = buf[-4 * T * H:].view(torch.float32).view(T, H)
                refused(lambda: layer.experts_int4(x, ids, w, packed, out))
                refused(lambda: layer.forward_int4(x, router, None, packed, out))
    for at in (0, E * H // 2 - 16, E * H + E - 4, E * H - T * H + 4):  # in the router's weights, at their end, in the bias
        out = big[at:at + T * H].view(T, H)
        refused(lambda: layer.forward_int4(x, router, bias, packed, out))
    torch.cuda.synchronize()
    assert torch.equal(big, before)
    for n, m in packed.items():
        assert torch.equal(m.codes, kept[n][0]) and torch.equal(m.scales, kept[n][1])
    # right behind the router's weights, and in front of the bias: nothing overlaps
    out, ref = big[E * H // 2:E * H // 2 + T * H].view(T, H), torch.empty(T, H, device="cuda")
    layer.forward_int4(x, router, bias, packed, ref)
    layer.forward_int4(x, router, bias, packed, out)
    assert torch.equal(out, ref)
    layer.close()


@pytest.mark.parametrize("R,K,group,zeros", [(5, 1 << 24, 128, False), (37, 1 << 22, 32, True), ((1 << 24) + 5, 8, 32, True),
                                             (1 << 22, 40, 64, False)])
def test_matvec_largest_extents(R, K, group, zeros):
    """The longest rows and many rows. A long row's x is zero but at random places (additions of zeros are
    exact, so that the bound counts the others)."""
    layer = _layer()
    g = torch.Generator(device="cuda").manual_seed(R + K)
    G = -(-K // group)
    q = torch.randint(0, 256, (R, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(R, G, generator=g, device="cuda") + 0.1).to(torch.bfloat16)
    z = torch.randint(0, 16, (R, G), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    m = layer.pack_int4(q, s, z, group)
    T = 3
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(K, device="cuda") if K < 2048 else torch.cat((torch.randint(0, K, (2000,), generator=g, device="cuda"),
                                                                  torch.tensor([0, K - 1], device="cuda"))).unique()
    x[:, at] = torch.randn(T, at.numel(), generator=g, device="cuda").to(torch.bfloat16)
    code = torch.where(at % 2 == 0, q[:, at // 2] & 15, q[:, at // 2] >> 4).double()
    w = (code - (8.0 if z is None else z[:, at // group].double())) * s[:, at // group].double()
    xs = x[:, at].double()
    ref, err = xs @ w.T, (2 * at.numel() + 8) * R32 * (xs.abs() @ w.abs().T)
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((T, R), float("nan"), dtype=dtype, device="cuda")
        layer.matvec_int4(x, m, out)
        _close(out, ref, err)
    layer.close()
