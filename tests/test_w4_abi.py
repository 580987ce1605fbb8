"""Host side of the few-token operators (no GPU): sizes and refusals before any launch."""
import ctypes

import pytest

import prefill_moe_route_b200 as moe


def _linear(**kw):
    d = dict(M=4, N=256, K=512, out_type=moe.MOE_OUT_BF16, ldx=512, ldo=256)
    d.update(kw)
    return moe.MoeLinearShape(**d)


@pytest.mark.parametrize("N,K,blocks", [(1, 32, 1), (128, 128, 1), (129, 128, 2), (128, 160, 2), (6144, 6144, 48 * 48)])
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
    for bad in (dict(M=(1 << 20) + 1), dict(N=(1 << 24) + 1, ldo=1 << 25), dict(N=1 << 24, ldo=1 << 24, K=1 << 20, ldx=1 << 20)):
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
    assert moe.moe_last_error()


def test_workspace_parts_come_first_and_grow_with_the_token_tile():
    sizes = [moe.moe_linear_w4_workspace_size(_linear(M=m)) for m in (1, 8, 9, 16, 17, 32, 33, 64, 65)]
    assert sizes == sorted(sizes) and sizes[0] == sizes[1] and sizes[2] == sizes[3]
