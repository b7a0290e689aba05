"""The feed-forward block's and the 4-bit products' host checks, without a GPU: the C entry points check
sizes, pointers and alignment before they look at the handle (NULL here), and the binding checks each
tensor before it passes an address."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def native():
    from mixture_experts_layer_block_b200 import build
    build.build()
    from mixture_experts_layer_block_b200 import native
    return native


P = 1 << 20  # an address that nothing reads: the handle is refused first


def _weights(native, up=P, gate=P, down=P):
    return native.moe_shared_w(up, gate, down)


def _ffn_forward(native, T=4, H=64, D=32, w=None, x=P, out=P, u=None, g=None, ws=P, nbytes=1 << 40):
    return native.lib.moe_ffn_forward(None, x, T, H, D, w or _weights(native), out, 1, u, g, ws, nbytes, None)


def _ffn_backward(native, T=4, H=64, D=32, w=None, dout=P, x=P, u=P, g=P, dx=P, grads=None, flags=0, ws=P, nbytes=1 << 40):
    return native.lib.moe_ffn_backward(None, dout, x, u, g, T, H, D, w or _weights(native), dx,
                                       grads or native.moe_ffn_grads(P, P, P), flags, ws, nbytes, None)


def test_workspace_bytes(native):
    f = native.lib.moe_ffn_workspace_bytes
    assert f(0, 64, 32, 0) == 0 and f(0, 64, 32, 1) == 0
    # at least the bf16 h of the forward, and du, dg and h of the backward
    for T, H, D in ((1, 8, 8), (16, 2048, 512), (17, 264, 136), (4096, 7168, 2048), (1 << 24, 64, 64)):
        assert f(T, H, D, 0) >= 2 * T * D
        assert f(T, H, D, 1) >= 6 * T * D
    for T, H, D in ((-1, 64, 32), (4, 0, 32), (4, 60, 32), (4, 64, 4), (4, 64, 36), (1 << 25, 64, 32), (4, 1 << 21, 32),
                    (4, 64, 1 << 21)):
        assert f(T, H, D, 0) == -1 and f(T, H, D, 1) == -1


def test_workspace_of_partial_sums_stays_small(native):
    """K is split only where tiles are few: the fp32 partials never pass 16 times one 256-row result."""
    f = native.lib.moe_ffn_workspace_bytes
    for T in (17, 100, 333, 515, 1000, 4096):
        for H, D in ((2048, 512), (2048, 2048), (7168, 2048), (264, 4096)):
            rows = -(-T // 256) * 256
            assert f(T, H, D, 0) <= 2 * T * D + 1024 + 16 * 4 * rows * (2 * (D + 64) + H)


@pytest.mark.parametrize("call", [_ffn_forward, _ffn_backward])
def test_ffn_refusals(native, call):
    bad, small, off = native.MOE_ERR_INVALID_ARG, native.MOE_ERR_UNSUPPORTED, native.MOE_ERR_MISALIGNED
    assert call(native) == bad  # nothing wrong but the handle
    for kw in (dict(T=-1), dict(H=0), dict(H=60), dict(D=36), dict(D=0), dict(ws=None), dict(x=None), dict(nbytes=0),
               dict(w=_weights(native, up=None)), dict(w=_weights(native, gate=None)), dict(w=_weights(native, down=None))):
        assert call(native, **kw) == bad, kw
    for kw in (dict(T=1 << 25), dict(H=1 << 21), dict(D=1 << 21)):
        assert call(native, **kw) == small, kw
    for kw in (dict(x=P + 8), dict(ws=P + 4), dict(u=P + 2, g=P), dict(u=P, g=P + 8), dict(w=_weights(native, up=P + 2)),
               dict(w=_weights(native, down=P + 8))):
        assert call(native, **kw) == off, kw


def test_ffn_forward_refusals(native):
    bad, off = native.MOE_ERR_INVALID_ARG, native.MOE_ERR_MISALIGNED
    for kw in (dict(out=None), dict(u=P), dict(g=P)):
        assert _ffn_forward(native, **kw) == bad, kw
    assert _ffn_forward(native, out=P + 8) == off
    # one byte less than the workspace's size
    n = native.lib.moe_ffn_workspace_bytes(4, 64, 32, 0)
    assert _ffn_forward(native, nbytes=n - 1) == bad
    # the handle is refused for an empty batch too, whose pointers may be null
    assert _ffn_forward(native, T=0, x=None, out=None, ws=None, nbytes=0) == bad


def test_ffn_backward_refusals(native):
    bad, off = native.MOE_ERR_INVALID_ARG, native.MOE_ERR_MISALIGNED
    for kw in (dict(dout=None), dict(u=None), dict(g=None), dict(flags=4), dict(flags=native.MOE_FFN_GRAD_ADD)):
        assert _ffn_backward(native, **kw) == bad, kw
    for kw in (dict(dx=P + 2), dict(grads=native.moe_ffn_grads(P, P + 8, P)), dict(dout=P + 1)):
        assert _ffn_backward(native, **kw) == off, kw


def test_int4_sizes(native):
    codes, scales = native.lib.moe_int4_code_bytes, native.lib.moe_int4_scale_bytes
    assert codes(1, 8) == 1024 and codes(16, 128) == 1024 and codes(17, 136) == 4 * 1024
    assert scales(1, 8, 128, 0) == 32 and scales(1, 8, 32, 1) == 4 * 64 and scales(33, 304, 64, 0) == 3 * 3 * 2 * 32
    for rows, cols, group in ((0, 64, 32), (16, 0, 32), (16, 60, 32), (16, 64, 16), (16, 64, 256), (-1, 64, 64),
                              (16, 1 << 25, 64), (1 << 42, 64, 64)):
        assert scales(rows, cols, group, 0) == -1, (rows, cols, group)
    assert codes(16, 60) == -1 and codes(0, 8) == -1


def test_int4_refusals(native):
    L, bad, small, off = native.lib, native.MOE_ERR_INVALID_ARG, native.MOE_ERR_UNSUPPORTED, native.MOE_ERR_MISALIGNED
    m = native.moe_int4_mat(P, P)

    def quant(src=P, rows=16, cols=64, group=32, codes=P, scales=P):
        return L.moe_quantize_int4(None, src, rows, cols, group, 0, codes, scales, None)

    def pack(q=P, s=P, z=None, rows=16, cols=64, group=32, codes=P, scales=P):
        return L.moe_pack_int4(None, q, s, z, rows, cols, group, codes, scales, None)

    def matvec(x=P, T=1, w=m, rows=16, cols=64, group=32, out=P, bf16=0):
        return L.moe_matvec_int4(None, x, T, w, rows, cols, group, 0, out, bf16, None)

    for f in (quant, pack, matvec):
        assert f() == bad
        for kw in (dict(rows=0), dict(cols=12), dict(group=48)):
            assert f(**kw) == bad, kw
        assert f(cols=1 << 25) == small
    for f, names in ((quant, ("src", "codes", "scales")), (pack, ("q", "s", "codes", "scales"))):
        for n in names:
            assert f(**{n: None}) == bad, n
            assert f(**{n: P + 8}) == off, n
    assert pack(z=P + 4) == off
    assert matvec(w=None) == bad and matvec(w=native.moe_int4_mat(P, None)) == bad and matvec(T=-1) == bad
    assert matvec(x=None) == bad and matvec(out=None) == bad
    assert matvec(rows=1 << 31) == small and matvec(T=1 << 25) == small
    assert matvec(x=P + 2) == off and matvec(w=native.moe_int4_mat(P + 4, P)) == off
    assert matvec(out=P + 2) == off and matvec(out=P + 2, bf16=1) == bad  # bf16 results need no more than their own boundary
    e = native.moe_int4_experts()
    assert L.moe_experts_int4(None, P, 1, P, P, 1, e, P, 0, None) == bad
    assert L.moe_forward_int4(None, P, 1, P, None, e, 1, P, None) == bad


def test_matvec_rows_that_do_not_round_up_within_31_bits(native):
    """The kernel's count of 16-row tiles is an int: the last sizes below 2^31 are refused, the first that fits
    is not (the handle is, here)."""
    def matvec(rows):
        return native.lib.moe_matvec_int4(None, P, 1, native.moe_int4_mat(P << 20, P << 21), rows, 8, 32, 0, P << 30, 0, None)

    for rows in ((1 << 31) - 15, (1 << 31) - 1, 1 << 31):
        assert matvec(rows) == native.MOE_ERR_UNSUPPORTED, rows
    assert matvec((1 << 31) - 16) == native.MOE_ERR_INVALID_ARG


# ---- the binding -------------------------------------------------------------------------------------
def _layer(native, H=64, D=32, E=4, k=2, Ds=0):
    layer = native.MoELayer.__new__(native.MoELayer)  # no handle: every call below is refused before the C call
    layer.h, layer.device, layer._torch_device, layer.out_dtype = None, 0, torch.device("cuda", 0), "float32"
    layer.cfg = native.moe_config(H, D, Ds, E, k, 16, 0.0, 16, 0, -1, 0, 0)
    return layer


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_checks_ffn_tensors(native):
    layer = _layer(native)
    w = {"Ws_up": _bf16(32, 64), "Ws_gate": _bf16(32, 64), "Ws_down": _bf16(64, 32)}
    x, out = _bf16(4, 64), _bf16(4, 64)
    with pytest.raises(ValueError, match="cuda:0"):  # right but for the device
        layer.ffn_forward(x, w, out)
    with pytest.raises(TypeError, match="bfloat16"):
        layer.ffn_forward(x.float(), w, out)
    with pytest.raises(ValueError, match="Ws_gate"):
        layer.ffn_forward(x, dict(w, Ws_gate=None), out)
    with pytest.raises(TypeError, match="torch tensor"):
        native._is_tensor([0.0], "x", (1,), native._BF16, 0)
    for bad in (_bf16(64), _bf16(2, 2, 64)):
        with pytest.raises(ValueError):
            layer.ffn_forward(bad, w, out)
    with pytest.raises(ValueError, match="contiguous"):
        native._is_tensor(_bf16(64, 4).T, "x", (4, 64), native._BF16, 0)
    with pytest.raises(ValueError, match="shape"):
        native._is_tensor(_bf16(4, 32), "x", (4, 64), native._BF16, 0)
    with pytest.raises(ValueError, match="multiples of 8"):
        layer.ffn_workspace_bytes(4, 60, 32)
    assert layer.ffn_workspace_bytes(4, 64, 32, True) > 0


def test_binding_checks_int4_arguments(native):
    layer = _layer(native)
    with pytest.raises(TypeError, match="Int4Matrix"):
        layer.matvec_int4(_bf16(1, 64), _bf16(16, 64), _bf16(1, 16))
    with pytest.raises(TypeError, match="Int4Matrix"):
        layer.experts_int4(_bf16(1, 64), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 2), {}, _bf16(1, 64))
    with pytest.raises(ValueError, match="groups of 32, 64 or 128"):
        native.Int4Matrix(16, 64, 48, False, "cpu")
    with pytest.raises(ValueError):
        layer.pack_int4(torch.zeros(16, dtype=torch.uint8), _bf16(16, 1))
    with pytest.raises(ValueError, match="contiguous"):
        layer.quantize_int4(_bf16(64, 16).T)
    for bad in (_bf16(64), 1.0):
        with pytest.raises(ValueError, match="matrix"):
            layer.quantize_int4(bad)
    m = native.Int4Matrix(4 * 32, 64, 32, False, "cpu")  # the buffers' sizes need no GPU
    assert m.codes.numel() == 8 * 1024 and m.scales.numel() == 8 * 4 * 32 and m.device == -1
    with pytest.raises(ValueError, match="cuda:0"):
        layer.matvec_int4(_bf16(1, 64), m, _bf16(1, 128))
    down = native.Int4Matrix(4 * 64, 32, 32, False, "cpu")
    wq = {"W_up": m, "W_gate": m, "W_down": down}
    with pytest.raises(ValueError, match="cuda:0"):
        layer._int4_experts(wq)
    layer.device = -1  # past the device check: the others
    assert layer._int4_experts(wq).group == 32
    with pytest.raises(ValueError, match="W_down"):
        layer._int4_experts(dict(wq, W_down=m))
    with pytest.raises(ValueError, match="group size"):
        layer._int4_experts(dict(wq, W_gate=native.Int4Matrix(4 * 32, 64, 64, False, "cpu")))
    with pytest.raises(ValueError, match="zero points"):
        layer._int4_experts(dict(wq, W_down=native.Int4Matrix(4 * 64, 32, 32, True, "cpu")))
    with pytest.raises(TypeError, match="Ws_up"):
        shared = _layer(native, Ds=32)
        shared.device = -1
        shared._int4_experts(wq)
