"""The few-token operators' layouts, and what they keep of values far below their block's largest."""
import pytest
import torch

import prefill_moe_route_b200 as moe
from test_gpu_layer_w4 import Layer
from w4_ref import layer_ref, rand_mx, swiglu_ref, value64

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _pack_expected(codes, scales):
    """The packed matrix byte by byte: absent rows and columns have zero codes and scale 127."""
    N, K = codes.shape[0], codes.shape[1] * 2
    RT, KC = -(-N // 128), -(-K // 128)
    c = torch.zeros(RT * 128, KC * 64, dtype=torch.uint8)
    c[:N, :K // 2] = codes
    s = torch.full((RT * 128, KC * 4), 127, dtype=torch.uint8)
    s[:N, :K // 32] = scales
    c = c.view(RT, 128, KC, 64).permute(0, 2, 1, 3)                       # [row tile][chunk][row][byte]
    s = s.view(RT, 4, 32, KC, 4).permute(0, 3, 2, 1, 4)                   # [row tile][chunk][r % 32][r / 32][group]
    return torch.cat([c.reshape(-1), s.reshape(-1)])


@pytest.mark.parametrize("N,K", [(1, 32), (128, 128), (130, 160), (127, 96), (257, 352), (300, 1024)])
def test_the_packed_layout_is_whole(N, K):
    g = torch.Generator(device=DEV)
    g.manual_seed(N + K)
    codes, scales = rand_mx(g, N, K, lo=0, hi=255)
    n = moe.moe_w4_packed_size(N, K)
    packed = torch.full((n,), 0xEE, device=DEV, dtype=torch.uint8)
    moe.moe_pack_w4(codes, scales, N, K, packed)
    assert torch.equal(packed.cpu(), _pack_expected(codes.cpu(), scales.cpu()))


def _wide(M, H, seed):
    """Blocks of 32 whose values lie up to 2^24 apart (bf16)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(M, H, generator=g, device=DEV)
    return (x * torch.exp2(-torch.randint(0, 25, (M, H), generator=g, device=DEV).float())).bfloat16()


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("M", [1, 4, 8, 16])
def test_layer_with_blocks_over_many_binades(M, norm):
    """What two columns keep of h: 2^-9 of each value (and an fp32 value passes through
    11 bits, 2^-12), but no less than 2^-21 of the block's largest, without a norm that
    alone: a block's scale leaves its largest between 2^7 and 2^8, lo's finest half step is
    2^-9 / 32 for values below 2^-6 and 2^-9 of the value above."""
    L = Layer(512, 16, 4, 256, 128, norm=norm)
    x = _wide(M, 512, seed=M)
    ws = L.workspace()
    out, ids, wts = L.run(x, ws)
    assert moe.moe_get_status(ws[0]) == (moe.MOE_OK, 0)
    experts = lambda e: (value64(L.w13[e], L.s13[e]), value64(L.w2[e], L.s2[e]))
    shared = (value64(L.sh[0][0], L.sh[1][0]), value64(L.sh[2][0], L.sh[3][0]))
    y, _, _, w, _ = layer_ref(x, L.norm_w, L.eps, L.router_w, L.bias, L.topk, L.scale, experts, shared, L.residual, ids=ids)
    x0 = x.double()
    h = x0
    if norm:
        h = x0 / torch.sqrt((x0 * x0).mean(-1, keepdim=True) + L.eps) * L.norm_w.double()
    blk = h.abs().reshape(M, -1, 32).amax(-1).repeat_interleave(32, -1)
    herr = 2.0 ** -21 * blk + ((2.0 ** -20 + 2.0 ** -12) * h.abs() if norm else 0.0)   # swiglu_ref adds 2^-9 of h
    tol = torch.zeros_like(y)
    for e in sorted(set(ids.flatten().tolist())):
        t, j = (ids == e).nonzero(as_tuple=True)
        ye, ee = swiglu_ref(h[t], herr[t], *experts(e))
        tol[t] += w[t, j, None] * (ee + 2.0 ** -16 * ye.abs())
    tol += swiglu_ref(h, herr, *shared)[1] + 2.0 ** -20 * y.abs() + 2.0 ** -8 * y.abs()
    assert bool(((wts.double() - w).abs() <= 1e-5 * w.abs() + 1e-7).all())
    assert bool(((out.double() - y).abs() <= tol).all())
    assert float((out.double() - y).norm()) <= 2.0 ** -8 * float(y.norm())
