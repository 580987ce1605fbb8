"""The few-token operators' layouts, ranges within a block, and the kernel that 5 to 8 tokens
take on large weights."""
import pytest
import torch

import prefill_moe_route_b200 as moe
from test_gpu_layer_w4 import Layer
from test_gpu_linear_w4 import Matrix, _check, _run_raw, _workspace, _x
from test_gpu_w4_timing import _child
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


# More than 8 units of 128 x 256 a CTA: there 5 to 8 tokens have their split made by a kernel before.
LARGE = [(152001, 96), (3200, 12320)]


@pytest.fixture(scope="module", params=LARGE, ids=["152001x96", "3200x12320"])
def large(request):
    return Matrix(*request.param, seed=11)


@pytest.mark.parametrize("M", [5, 8])
def test_large_weights_a_token_that_is_not_finite_is_nan_alone(M, large):
    clean = _x(M, large.K, seed=8)
    want = _run_raw(clean, large)
    _check(want, clean, large)
    for v in (float("inf"), float("-inf"), float("nan")):
        x = clean.clone()
        x[M // 2, 50] = v
        got = _run_raw(x, large)
        assert bool(got[M // 2].isnan().all())
        keep = torch.arange(M, device=DEV) != M // 2
        assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("M", [5, 8])
def test_large_weights_rows_inside_larger_buffers(M, large):
    N, K = large.N, large.K
    xb = torch.full((M + 2, K + 40), float("nan"), device=DEV, dtype=torch.bfloat16)
    x = xb[1:M + 1, 8:K + 8]
    x.copy_(_x(M, K))
    for dt, ot in ((torch.float32, moe.MOE_OUT_F32), (torch.bfloat16, moe.MOE_OUT_BF16)):
        ob = torch.full((M + 2, N + 3), 77.0, device=DEV, dtype=dt)
        out = ob[1:M + 1, 1:N + 1]
        sh = moe.MoeLinearShape.of(M, N, K, ldx=xb.stride(0), ldo=ob.stride(0), out_type=ot)
        ws, n = _workspace(sh)
        moe.moe_linear_w4(sh, x, large.packed, None, out, ws, n)
        _check(out, x, large)
        ob[1:M + 1, 1:N + 1] = 77.0
        assert bool((ob == 77.0).all())


@pytest.mark.parametrize("M", [5, 8])
def test_large_weights_captured_and_replayed_beside_other_counts(M, large):
    """One workspace for 4, M and 16 tokens in one graph: the operand blocks lie behind the
    parts, which every count leaves empty."""
    N, K = large.N, large.K
    counts = (4, M, 16)
    shs = [moe.MoeLinearShape.of(m, N, K, out_type=moe.MOE_OUT_F32) for m in counts]
    ws, n = _workspace(*shs)
    xs = [_x(m, K) for m in counts]
    outs = [torch.empty(m, N, device=DEV) for m in counts]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(2):
                for sh, x, out in zip(shs, xs, outs):
                    moe.moe_linear_w4(sh, x, large.packed, None, out, ws, n)
        for seed in range(3):
            for m, x, out in zip(counts, xs, outs):
                x.copy_(_x(m, K, seed=20 + seed + m))
                out.zero_()
            g.replay()
            st.synchronize()
            for x, out in zip(xs, outs):
                _check(out, x, large)
    assert moe.moe_get_status(ws) == (moe.MOE_OK, 0)


WITHHELD = """
import torch
import test_gpu_linear_w4 as t
import prefill_moe_route_b200 as moe
M, N, K = (int(a) for a in sys.argv[1:])
mat = t.Matrix(N, K)
sh = moe.MoeLinearShape.of(M, N, K, out_type=moe.MOE_OUT_F32)
ws, n = t._workspace(sh)
out = torch.empty(M, N, device='cuda')
moe.moe_linear_w4(sh, t._x(M, K), mat.packed, None, out, ws, n)
rc, st = moe.moe_get_status(ws)
assert rc == moe.MOE_ERR_DEVICE_TIMEOUT and st == 1, (rc, st)
moe.moe_workspace_init(ws, n)
t._run(M, N, K, moe.MOE_OUT_F32, mat=mat, ws=(ws, n))
print('child ok')
"""


@pytest.mark.parametrize("M", [5, 8])
def test_large_weights_a_part_that_never_comes_ends_in_a_status(M):
    _child(WITHHELD, M, 3200, 12320, MOE_TEST_WITHHOLD_FLAG="1", MOE_WAIT_TIMEOUT_MS="20")


@pytest.mark.parametrize("M", [1, 4, 8, 16])
@pytest.mark.parametrize("norm,S", [(False, 0), (False, 128), (True, 0)])
def test_layer_forms_a_token_that_is_not_finite_is_nan_alone(M, norm, S):
    """Without a norm an infinity gives sigmoids of 0 and 1, so weights of 0 among the chosen;
    without a shared expert nothing else makes the token NaN."""
    L = Layer(512, 16, 4, 256, S, norm=norm, residual=False)
    ws = L.workspace()
    x = L.x(M)
    want = L.run(x, ws)
    bad = M // 2
    keep = torch.arange(M, device=DEV) != bad
    for v in (float("nan"), float("inf"), float("-inf")):
        for sign in (1.0, -1.0):
            L.router_w[:, 100] = L.router_w[:, 100].abs() * sign   # every logit the same way
            base = L.run(x, ws)
            y = x.clone()
            y[bad, 100] = v
            out, ids, wts = L.run(y, ws)
            assert moe.moe_get_status(ws[0]) == (moe.MOE_OK, 0)
            assert bool(out[bad].isnan().all()) and int(ids.min()) >= 0 and int(ids.max()) < 16
            assert torch.equal(out[keep], base[0][keep]) and torch.equal(ids[keep], base[1][keep])
    assert bool(want[0].isfinite().all())


@pytest.mark.parametrize("M", [1, 4, 8, 16])
def test_layer_experts_masked_by_the_bias(M):
    """A bias of -inf or of fp32's lowest value keeps an expert out while others are left; with
    fewer left than top-k the masked ones follow, the lower expert first."""
    L = Layer(512, 16, 4, 256, 128)
    for low in (float("-inf"), torch.finfo(torch.float32).min):
        L.bias[:] = 0.1
        L.bias[3:13] = low
        ws = L.workspace()
        x = L.x(M)
        got = L.run(x, ws)
        assert moe.moe_get_status(ws[0]) == (moe.MOE_OK, 0)
        assert not (set(got[1].flatten().tolist()) & set(range(3, 13)))
        L.check(x, got)
        L.bias[:] = low
        L.bias[[5, 9]] = 0.1
        out, ids, wts = L.run(x, ws)
        for row in ids.tolist():
            assert set(row[:2]) == {5, 9} and row[2:] == [0, 1]
        assert bool(out.isfinite().all())
