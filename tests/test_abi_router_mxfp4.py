"""Host-side argument checks of the router's training calls and of the MXFP4
calls: every case is rejected (or answered) before the library looks for a
device, so the codes are the same with or without a GPU and no pointer is
dereferenced."""
import pytest

from mxfp8_grouped_gemm_x32_b200 import lib

P, M, ODD = 1 << 20, (1 << 20) + 8, (1 << 20) + 1
INVALID, UNSUPPORTED, WORKSPACE, NO_DEVICE = 1, 2, 3, 7
BIG = 1 << 40


def _args(defaults, over):
    d = dict(defaults)
    assert set(over) <= set(d), over
    d.update(over)
    return tuple(d.values())


def _losses(**kw):
    return lib._lib.moe_router_losses(*_args(dict(
        logits=P, dt=0, T=8, E=16, k=2, mask=None, idx=P, prob=P, lse=P, counts=P, sums=P, tokens=P, losses=P, ws=P,
        wsb=BIG, st=None), kw))


def _bwd(**kw):
    return lib._lib.moe_router_bwd(*_args(dict(
        logits=P, dt=0, T=8, E=16, k=2, mask=None, idx=P, prob=P, lse=P, counts=P, tokens=P, dprob=None, dlosses=None,
        dlogits=P, st=None), kw))


def _quant(**kw):
    return lib._lib.moe_mlp_quantize_mxfp4(*_args(dict(src=P, dt=1, groups=1, rows=4, cols=64, q=P, ldq=max(0, kw.get("cols", 64) // 2), sf=P,
                                                       st=None), kw))


def _dequant(**kw):
    return lib._lib.moe_mlp_dequantize_mxfp4(*_args(dict(
        q=P, ldq=max(0, kw.get("cols", 64) // 2), sf=P, groups=1, rows=4, cols=64, dt=1, dst=P, st=None), kw))


def _fwd(**kw):
    T, k, E = kw.get("T", 64), kw.get("k", 2), kw.get("E", 4)
    return lib._lib.moe_grouped_mlp_fwd_mxfp4(*_args(dict(
        w1q=P, ld1=2048, w1sf=P, w2q=P, ld2=256, w2sf=P, T=64, H=256, I=512, E=4, k=2, cap=lib.moe_padded_rows(T, k, E), split=P, offs=P,
        s2r=P, prob=P, x=P, out=P, ws=P, wsb=BIG, st=None), kw))


@pytest.mark.parametrize("call", [_losses, _bwd])
@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), INVALID), (dict(idx=None), INVALID), (dict(prob=None), INVALID), (dict(lse=None), INVALID),
    (dict(counts=None), INVALID), (dict(tokens=None), INVALID), (dict(dt=2), INVALID), (dict(T=-1), INVALID),
    (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=17), INVALID), (dict(logits=ODD), INVALID),
    (dict(dt=1, logits=ODD), INVALID), (dict(lse=ODD), INVALID), (dict(counts=ODD), INVALID),
    (dict(E=257), UNSUPPORTED), (dict(E=64, k=33), UNSUPPORTED), (dict(T=1 << 29, k=2), UNSUPPORTED),
])
def test_router_calls(call, kw, code):
    assert call(**kw) == code


def test_router_calls_apart():
    assert _losses(sums=None) == INVALID and _losses(losses=None) == INVALID and _losses(losses=ODD) == INVALID
    assert _losses(ws=None) == WORKSPACE and _losses(ws=M) == WORKSPACE
    assert _losses(wsb=lib.moe_workspace_size(lib.MOE_OP_ROUTER_LOSSES, 8, 2, 16, 0, 0) - 1) == WORKSPACE
    assert _bwd(dlogits=None) == INVALID and _bwd(dprob=ODD) == INVALID and _bwd(dlosses=ODD) == INVALID
    assert _bwd(dlogits=ODD) == INVALID
    assert lib.moe_workspace_size(lib.MOE_OP_ROUTER_LOSSES, 0, 2, 16, 0, 0) > 0
    assert lib.moe_workspace_size(lib.MOE_OP_ROUTER_LOSSES, -1, 2, 16, 0, 0) == -1


@pytest.mark.parametrize("call,out", [(_quant, "q"), (_dequant, "dst")])
def test_codec_calls(call, out):
    assert call(groups=-1) == INVALID and call(rows=-1) == INVALID and call(cols=-32) == INVALID
    assert call(dt=2) == INVALID
    assert call(cols=48) == UNSUPPORTED
    for name in ("q", "sf", out):
        assert call(**{name: None}) == INVALID and call(**{name: M}) == INVALID
    assert call(ldq=16) == INVALID and call(ldq=40) == INVALID and call(ldq=-32) == INVALID
    # sizes past 32-bit unit numbers, also those whose product would wrap
    assert call(rows=1 << 31, cols=64) == UNSUPPORTED
    assert call(groups=1 << 30, rows=1 << 30, cols=1 << 20) == UNSUPPORTED
    assert call(rows=1 << 28, cols=64) == UNSUPPORTED
    # nothing to do: no pointer is needed
    assert call(rows=0, sf=None, **{out: None}) == 0 and call(cols=0) == 0 and call(groups=0) == 0


def test_forward_call():
    for name in ("w1q", "w1sf", "w2q", "w2sf", "split", "offs", "prob", "s2r", "x", "out"):
        assert _fwd(**{name: None}) == INVALID, name
    for name in ("w1q", "w1sf", "w2q", "w2sf", "x", "out"):
        assert _fwd(**{name: M}) == INVALID, name
    for kw in (dict(H=48), dict(I=96), dict(E=257, k=2), dict(k=5), dict(T=1 << 29), dict(T=-1),
               dict(T=1 << 25, k=1, H=4096)):
        assert _fwd(**kw) in (UNSUPPORTED, INVALID), kw
    assert _fwd(T=1 << 25, k=1, H=4096) == UNSUPPORTED
    assert _fwd(cap=lib.moe_padded_rows(64, 2, 4) - 128) == INVALID
    for kw in (dict(ld1=112), dict(ld1=136), dict(ld2=240), dict(ld2=264), dict(ld1=0)):
        assert _fwd(**kw) == INVALID, kw
    assert _fwd(cap=lib.moe_padded_rows(64, 2, 4) + 64) == INVALID
    need = lib.moe_workspace_size(lib.MOE_OP_FWD_MXFP4, 64, 2, 4, 256, 512)
    assert need > 0 and _fwd(wsb=need - 1) == WORKSPACE and _fwd(ws=None) == WORKSPACE and _fwd(ws=M) == WORKSPACE
    assert lib.moe_workspace_size(lib.MOE_OP_FWD_MXFP4, 64, 2, 4, 0, 512) == -1


@pytest.mark.parametrize("g,r,k", [(1, 1, 32), (3, 128, 128), (2, 129, 2880), (0, 5, 64), (7, 0, 96)])
def test_scale_bytes_of_the_python_layer(g, r, k):
    from mxfp8_grouped_gemm_x32_b200 import mxfp4
    assert mxfp4._scale_bytes(g, r, k) == lib.moe_mx_scale_bytes(g, r, k)


def test_tile_scales_call():
    f = lib._lib.moe_mxfp4_tile_scales
    assert f(P, 4, 64, 64, 2, 1, None, None) == INVALID and f(None, 4, 64, 64, 2, 0, P, None) == INVALID
    assert f(P, 4, 64, 64, 1, 1, P, None) == INVALID and f(P, 4, 64, 48, 2, 1, P, None) == INVALID
    assert f(P, 4, 64, 64, 2, 2, P, None) == INVALID and f(P, -1, 64, 64, 2, 1, P, None) == INVALID
    assert f(P, 4, 64, 64, 2, 1, M, None) == INVALID
    assert f(None, 0, 64, 64, 2, 1, None, None) == 0
    size = lib.moe_mxfp4_tiled_scale_bytes
    assert size(2, 97, 257 * 32, 1) == 2 * 2 * 33 * 1536 and size(3, 192, 256, 0) == 3 * 1536
    assert size(3, 193, 288, 0) == 3 * 2 * 2 * 1536 and size(1, 64, 33, 0) == -1 and size(1, 64, 32, 5) == -1


def test_half_the_bytes_of_the_mxfp8_recipe():
    """Codes of 4 bits: a layer's MXFP4 weights take half of its MXFP8 ones."""
    E, H, I = 8, 4096, 14336
    q8, sf = 3 * E * H * I, lib.moe_mx_scale_bytes(2 * E, I, H) + lib.moe_mx_scale_bytes(E, H, I)
    sf4 = lib.moe_mxfp4_tiled_scale_bytes(E, I, H, 1) + lib.moe_mxfp4_tiled_scale_bytes(E, H, I, 0)
    assert (q8 // 2 + sf4) / (q8 + sf) < 0.52


def test_python_layer_refuses_before_any_call():
    import torch
    from mxfp8_grouped_gemm_x32_b200 import mxfp4
    for bad, exc in (([1.0], TypeError), (torch.zeros(2, 32, dtype=torch.float16), TypeError),
                     (torch.zeros(2, 32), ValueError)):
        with pytest.raises(exc):
            mxfp4.quantize(bad)
    with pytest.raises(TypeError):
        mxfp4.dequantize(torch.zeros(2, 16, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), torch.float16)
    with pytest.raises(ValueError):
        mxfp4.dequantize(torch.zeros(2, 16, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8))
    with pytest.raises(TypeError):
        mxfp4.dequantize(None, None)
