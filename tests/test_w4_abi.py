"""Host side of the few-token operators (no GPU): sizes and refusals before any launch."""
import ctypes

import pytest

import prefill_moe_route_b200 as moe


def _linear(**kw):
    d = dict(M=4, N=256, K=512, out_type=moe.MOE_OUT_BF16, ldx=512, ldo=256)
    d.update(kw)
    return moe.MoeLinearShape(**d)


@pytest.mark.parametrize("N,K,blocks", [(1, 32, 1), (128, 128, 1), (129, 128, 2), (128, 160, 2), (6144, 6144, 48 * 48),
                                        (2**31 - 1, 32, 2**24), (1, 2**31 - 32, 2**24)])   # no 32-bit sums
def test_packed_size_counts_blocks_of_128_by_128(N, K, blocks):
    assert moe.moe_w4_packed_size(N, K) == blocks * (8192 + 512)


@pytest.mark.parametrize("N,K", [(0, 128), (128, 0), (128, 48), (-1, 128)])
def test_packed_size_refuses(N, K):
    n = ctypes.c_size_t(0)
    assert moe.load().moe_w4_packed_size(N, K, ctypes.byref(n)) == moe.MOE_ERR_INVALID_ARG
    assert moe.load().moe_w4_packed_size(128, 128, None) == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(M=0), dict(N=0), dict(K=0), dict(K=48), dict(ldx=504), dict(ldx=516), dict(ldo=255),
                                 dict(out_type=2), dict(out_type=-1), dict(M=-3)])
def test_linear_refuses_shapes(bad):
    sh = _linear(**bad)
    n = ctypes.c_size_t(0)
    assert moe.load().moe_linear_w4_workspace_size(ctypes.byref(sh), ctypes.byref(n)) == moe.MOE_ERR_INVALID_ARG


def test_linear_refuses_shapes_past_its_limits():
    n = ctypes.c_size_t(0)
    for bad in (dict(M=(1 << 19) + 1), dict(N=(1 << 24) + 1, ldo=1 << 25), dict(N=1 << 24, ldo=1 << 24, K=1 << 20, ldx=1 << 20)):
        sh = _linear(**bad)
        assert moe.load().moe_linear_w4_workspace_size(ctypes.byref(sh), ctypes.byref(n)) == moe.MOE_ERR_UNSUPPORTED


def test_linear_refuses_pointers_before_any_launch():
    sh = _linear()
    ok = dict(x=4096, w=8192, bias=None, out=16384, ws=32768)

    def call(**kw):
        a = dict(ok, **kw)
        return moe.moe_linear_w4(sh, a["x"], a["w"], a["bias"], a["out"], a["ws"], 1 << 30, stream=0, check=False)

    for kw in (dict(x=None), dict(w=None), dict(out=None), dict(ws=None), dict(x=4104), dict(w=8208), dict(ws=32784),
               dict(bias=4098), dict(out=16385), dict(out=4096), dict(out=32768)):
        assert call(**kw) == moe.MOE_ERR_INVALID_ARG, kw
    sh.out_type = moe.MOE_OUT_F32
    assert call(out=16386) == moe.MOE_ERR_INVALID_ARG
    assert moe.load().moe_linear_w4(None, 4096, 8192, None, 16384, 32768, 1 << 30, None) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_pack_w4(None, None, 128, 128, None, stream=0, check=False) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_pack_w4(4104, 4096, 128, 128, 8192, stream=0, check=False) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_pack_w4(4096, 4096, 128, 128, 8208, stream=0, check=False) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_pack_w4(4096, 4096, 128, 100, 8192, stream=0, check=False) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_pack_w4(4096, 1 << 20, 128, 128, 8192, stream=0, check=False) == moe.MOE_ERR_INVALID_ARG   # q overlaps
    assert moe.moe_pack_w4(1 << 20, 8448, 128, 128, 8192, stream=0, check=False) == moe.MOE_ERR_INVALID_ARG   # scales do
    assert moe.moe_last_error()


def test_workspace_parts_come_first_and_grow_with_the_token_tile():
    sizes = [moe.moe_linear_w4_workspace_size(_linear(M=m)) for m in (1, 8, 9, 16, 17, 32, 33, 64, 65)]
    assert sizes == sorted(sizes) and sizes[0] == sizes[1] and sizes[2] == sizes[3]


def _layer(**kw):
    d = dict(M=4, H=512, I=256, E=8, topk=2, shared_I=128, add_residual=1, routed_scale=1.0, norm_eps=1e-5, ldx=512, ldo=512)
    d.update(kw)
    return moe.MoeLayerShape(**d)


@pytest.mark.parametrize("bad,code", [
    (dict(M=0), moe.MOE_ERR_INVALID_ARG), (dict(E=0), moe.MOE_ERR_INVALID_ARG), (dict(topk=0), moe.MOE_ERR_INVALID_ARG),
    (dict(shared_I=-128), moe.MOE_ERR_INVALID_ARG), (dict(ldx=504), moe.MOE_ERR_INVALID_ARG),
    (dict(ldx=516), moe.MOE_ERR_INVALID_ARG), (dict(ldo=511), moe.MOE_ERR_INVALID_ARG),
    (dict(routed_scale=float("inf")), moe.MOE_ERR_INVALID_ARG), (dict(norm_eps=float("nan")), moe.MOE_ERR_INVALID_ARG),
    (dict(norm_eps=-1.0), moe.MOE_ERR_INVALID_ARG), (dict(M=17), moe.MOE_ERR_UNSUPPORTED),
    (dict(E=513), moe.MOE_ERR_UNSUPPORTED), (dict(topk=9), moe.MOE_ERR_UNSUPPORTED),
    (dict(E=64, topk=17), moe.MOE_ERR_UNSUPPORTED), (dict(H=576, ldx=576, ldo=576), moe.MOE_ERR_UNSUPPORTED),
    (dict(I=192), moe.MOE_ERR_UNSUPPORTED), (dict(shared_I=64), moe.MOE_ERR_UNSUPPORTED)])
def test_layer_refuses_shapes(bad, code):
    n = ctypes.c_size_t(0)
    assert moe.load().moe_layer_w4_workspace_size(ctypes.byref(_layer(**bad)), ctypes.byref(n)) == code


def test_layer_workspace_does_not_depend_on_the_token_count():
    assert len({moe.moe_layer_w4_workspace_size(_layer(M=m)) for m in (1, 8, 9, 16)}) == 1


def test_layer_refuses_pointers_before_any_launch():
    names = ["norm_w", "router_w", "bias", "w13", "w13_scales", "w2", "w2_scales", "shared_w13", "shared_w13_scales",
             "shared_w2", "shared_w2_scales"]
    good = {n: 4096 * (i + 1) for i, n in enumerate(names)}

    def call(shape=None, x=1 << 20, out=1 << 21, ws=1 << 22, ids=None, wts=None, **kw):
        w = moe.MoeLayerWeights.of(**dict(good, **kw))
        return moe.moe_layer_w4(shape or _layer(), w, x, out, ids, wts, ws, 1 << 30, stream=0, check=False)

    for kw in (dict(x=None), dict(out=None), dict(ws=None), dict(router_w=None), dict(w13=None), dict(w13_scales=None),
               dict(w2=None), dict(w2_scales=None), dict(shared_w13=None), dict(shared_w2_scales=None), dict(w13=4112),
               dict(shared_w2=4112), dict(norm_w=4104), dict(router_w=4104), dict(w2_scales=4104), dict(bias=4098),
               dict(x=(1 << 20) + 8), dict(ws=(1 << 22) + 128), dict(out=1 << 20), dict(out=1 << 22), dict(out=(1 << 21) + 1),
               dict(ids=4098), dict(wts=4098)):
        assert call(**kw) == moe.MOE_ERR_INVALID_ARG, kw
    assert moe.load().moe_layer_w4(None, None, None, None, None, None, None, 0, None) == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [b"\0" * 16, ctypes.c_void_p(4096), "4096", 4096.0], ids=["bytes", "c_void_p", "str", "float"])
def test_a_buffer_is_a_tensor_or_an_address(bad):
    """Python objects that ctypes would pass on as host memory are refused by name."""
    with pytest.raises(AttributeError):
        moe.moe_linear_w4(_linear(), bad, 8192, None, 16384, 32768, 1 << 30, stream=0)
    with pytest.raises(AttributeError):
        moe.moe_round_bf16(bad, 8192, 8, stream=0)
    with pytest.raises(AttributeError):
        moe.MoeLayerWeights.of(router_w=bad, w13=1, w13_scales=1, w2=1, w2_scales=1)
