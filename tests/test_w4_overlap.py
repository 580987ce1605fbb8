"""Buffers of the few-token operators that overlap are refused before any launch (no GPU)."""
import pytest

import prefill_moe_route_b200 as moe

BASE = 1 << 32


def _linear(M=4, N=256, K=512, ldx=512, ldo=256, out_type=moe.MOE_OUT_BF16, **at):
    """Refused for an overlap?  Addresses far apart unless given; w 69632 bytes, out 2048."""
    a = dict(dict(x=BASE, w=BASE + (1 << 24), bias=BASE + (2 << 24), out=BASE + (3 << 24), ws=BASE + (4 << 24)), **at)
    sh = moe.MoeLinearShape(M, N, K, out_type, ldx, ldo)
    rc = moe.moe_linear_w4(sh, a["x"], a["w"], a["bias"], a["out"], a["ws"], 1 << 30, stream=0, check=False)
    assert rc != moe.MOE_OK   # the addresses are made up
    hit = "overlap" in moe.moe_last_error()
    assert not hit or rc == moe.MOE_ERR_INVALID_ARG
    return hit


X, W, B, O, S = (BASE + (i << 24) for i in range(5))
WS = moe.moe_linear_w4_workspace_size(moe.MoeLinearShape.of(4, 256, 512))


@pytest.mark.parametrize("at,hit", [
    (dict(), False),
    (dict(out=X + 4094), True), (dict(out=X + 4096), False),            # x: 4 rows of 1024 bytes
    (dict(out=X - 2048 + 2), True), (dict(out=X - 2048), False),        # out: 4 rows of 512 bytes
    (dict(out=W + 69632 - 2), True), (dict(out=W + 69632), False),
    (dict(out=B + 1022), True), (dict(out=B + 1024), False), (dict(bias=O + 2044), True), (dict(bias=O + 2048), False),
    (dict(out=S + WS - 2), True), (dict(out=S + WS), False), (dict(ws=O), True),
    (dict(x=S + 256), True), (dict(w=S + 256), True), (dict(bias=S + 4), True), (dict(ws=X + 3840), True), (dict(ws=X + 4096), False),
    (dict(x=W), False),                                                  # two inputs may share bytes
    (dict(out_type=moe.MOE_OUT_F32, out=X - 4096 + 4), True), (dict(out_type=moe.MOE_OUT_F32, out=X - 4096), False),
])
def test_linear(at, hit):
    assert _linear(**at) is hit


@pytest.mark.parametrize("at,hit", [
    (dict(out=X + 1024), False),                       # columns 512 .. 767 of the rows that hold x in 0 .. 511
    (dict(out=X + 1022), True),                        # one column of x
    (dict(out=X + 2048 - 512), False), (dict(out=X + 2048 - 510), True),   # up to the next row's x, and into it
    (dict(out=X - 512), False), (dict(out=X - 510), True),
    (dict(out=X + 3 * 2048 + 1024), False), (dict(out=X + 3 * 2048 + 1022), True),
    (dict(out=X + 2048 + 1024, ldo=3 * 1024), False),  # every third row's gap
    (dict(out=X + 1024, ldo=1024 + 256), True),        # other pitches meet sooner or later
    (dict(out=X + 1024, ldo=1024 + 256, M=2), False),  # rows at 1024 and 3584, x at 0 and 2048: too few rows to meet
    (dict(out=X + 1024, ldo=512, M=2), True),          # rows at 1024 and 2048
])
def test_linear_rows_between_rows(at, hit):
    assert _linear(**dict(dict(ldx=1024, ldo=1024), **at)) is hit


NAMES = ["norm_w", "router_w", "bias", "w13", "w13_scales", "w2", "w2_scales", "shared_w13", "shared_w13_scales",
         "shared_w2", "shared_w2_scales"]
H, I, E, TOPK, SI = 512, 256, 8, 2, 128
BYTES = dict(norm_w=H * 2, router_w=E * H * 2, bias=E * 4, w13=E * I * H, w13_scales=E * I * H // 16, w2=E * I * H // 2,
             w2_scales=E * I * H // 32, shared_w13=SI * H, shared_w13_scales=SI * H // 16, shared_w2=SI * H // 2,
             shared_w2_scales=SI * H // 32)


def _layer(M=4, ldx=H, ldo=H, shared=SI, **at):
    a = dict({n: BASE + (i << 24) for i, n in enumerate(NAMES)}, x=BASE + (20 << 24), out=BASE + (21 << 24), ids=BASE + (22 << 24),
             wts=BASE + (23 << 24), ws=BASE + (24 << 24))
    a.update(at)
    sh = moe.MoeLayerShape.of(M, H, I, E, TOPK, 1.0, shared_I=shared, add_residual=True, ldx=ldx, ldo=ldo)
    w = moe.MoeLayerWeights.of(**{n: a[n] for n in NAMES})
    rc = moe.moe_layer_w4(sh, w, a["x"], a["out"], a["ids"], a["wts"], a["ws"], 1 << 30, stream=0, check=False)
    assert rc != moe.MOE_OK
    hit = "overlap" in moe.moe_last_error()
    assert not hit or rc == moe.MOE_ERR_INVALID_ARG
    return hit


@pytest.mark.parametrize("name", NAMES)
def test_layer_weights_stay_apart_from_what_is_written(name):
    end = BASE + (NAMES.index(name) << 24) + BYTES[name]
    assert not _layer(out=end) and _layer(out=end - 2)
    assert not _layer(ids=end) and _layer(ids=end - 4)
    assert not _layer(wts=end) and _layer(wts=end - 4)
    assert _layer(ws=BASE + (NAMES.index(name) << 24))
    if name.startswith("shared"):
        assert not _layer(out=end - 2, shared=0)   # not read then


@pytest.mark.parametrize("at,hit", [
    (dict(), False), (dict(ids=BASE + (23 << 24)), True), (dict(ids=None, wts=None), False),
    (dict(ids=BASE + (23 << 24) - 32), False), (dict(ids=BASE + (23 << 24) - 28), True),   # 4 x 2 of 4 bytes
    (dict(ids=BASE + (21 << 24) + 4092), True), (dict(wts=BASE + (21 << 24) + 4096), False),
    (dict(ids=BASE + (20 << 24)), True), (dict(wts=BASE + (24 << 24)), True),
    (dict(out=BASE + (20 << 24) + 1024, ldx=2 * H, ldo=2 * H), False),
    (dict(out=BASE + (20 << 24) + 1022, ldx=2 * H, ldo=2 * H), True),
    (dict(x=BASE + (24 << 24) + 4096), True),
])
def test_layer_tokens_and_outputs(at, hit):
    assert _layer(**at) is hit
