"""moe_linear_w4 (MXFP4 weights, bf16 activations) against a 64-bit product."""
import os
import subprocess
import sys

import pytest
import torch

import prefill_moe_route_b200 as moe
from conftest import ROOT
from w4_ref import linear_ref, rand_mx, value64

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


class Matrix:
    def __init__(self, N, K, seed=0, lo=117, hi=123):
        self.N, self.K = N, K
        self.codes, self.scales = rand_mx(_gen(seed), N, K, lo=lo, hi=hi)
        self.repack()

    def repack(self):
        self.w = value64(self.codes, self.scales)
        self.packed = torch.empty(moe.moe_w4_packed_size(self.N, self.K), device=DEV, dtype=torch.uint8)
        moe.moe_pack_w4(self.codes, self.scales, self.N, self.K, self.packed)


def _workspace(*shapes):
    n = max(moe.moe_linear_w4_workspace_size(s) for s in shapes)
    ws = torch.empty(n, device=DEV, dtype=torch.uint8)
    moe.moe_workspace_init(ws, n)
    return ws, n


def _x(M, K, seed=1, loud=True):
    g = _gen(seed)
    x = torch.randn(M, K, generator=g, device=DEV)
    if loud:   # a few channels far above the rest
        x = x * (1 + 200 * (torch.rand(K, generator=g, device=DEV) < 0.02))
    return x.bfloat16()


def _check(got, x, mat, bias=None):
    y, tol = linear_ref(x, mat.w, bias)
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * y.abs()
    d = (got.double() - y).abs()
    bad = ~(d <= tol)
    assert not bad.any(), f"{int(bad.sum())} outputs off, worst {float((d - tol).max()):.3g} past the bound"
    if got.dtype == torch.float32:
        # roundings of either sign: K + 8 of them add like their root (rms of partial sums <= rms of |x||w|)
        rel = float(d.norm() / y.norm()) if float(y.norm()) else 0.0
        big = float((x.double().square() @ mat.w.square().T).sqrt().norm() / y.norm()) if float(y.norm()) else 0.0
        assert rel <= 2.0 ** -23 * (x.shape[1] + 8) ** 0.5 * max(1.0, big) + 2.0 ** -20, rel


def _run(M, N, K, out_type, bias=None, mat=None, x=None, ws=None):
    mat = mat or Matrix(N, K, seed=N + K)
    x = _x(M, K, seed=M) if x is None else x
    sh = moe.MoeLinearShape.of(M, N, K, out_type=out_type)
    ws, n = ws or _workspace(sh)
    out = torch.empty(M, N, device=DEV, dtype=torch.float32 if out_type == moe.MOE_OUT_F32 else torch.bfloat16)
    moe.moe_linear_w4(sh, x, mat.packed, bias, out, ws, n)
    assert moe.moe_get_status(ws) == (moe.MOE_OK, 0)
    _check(out, x, mat, bias)
    return out


SIZES = [(1, 1, 32), (1, 128, 128), (3, 127, 96), (1, 129, 160), (2, 300, 288), (8, 512, 512), (9, 256, 384),
         (16, 1000, 2912), (17, 64, 32), (31, 130, 416), (32, 512, 1024), (33, 129, 320), (64, 384, 512), (65, 257, 512),
         (128, 128, 256), (200, 100, 2080), (1000, 300, 96), (3, 60, 40000), (40, 130, 32800), (2, 100003, 64), (1, 6144, 6144), (5, 4099, 2912), (40, 2000, 4096), (1, 20011, 512), (5, 152001, 96),
         (8, 3200, 12320)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("out_type", [moe.MOE_OUT_F32, moe.MOE_OUT_BF16])
def test_against_64_bits(M, N, K, out_type):
    bias = torch.randn(N, device=DEV) if (M + N) % 2 else None
    _run(M, N, K, out_type, bias)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 15, 16, 20, 24, 48, 63])
def test_every_token_count(M):
    _run(M, 1536, 1536, moe.MOE_OUT_F32, mat=_shared_matrix())


_cache = {}


def _shared_matrix():
    if "m" not in _cache:
        _cache["m"] = Matrix(1536, 1536, seed=5)
    return _cache["m"]


@pytest.mark.parametrize("M", [1, 7, 16, 20, 70])
def test_rows_inside_larger_buffers(M):
    """ldx, ldo: NaN beside the rows is not read, the neighbours of out stay as they were."""
    N, K = 259, 480
    mat = Matrix(N, K, seed=3)
    xb = torch.full((M + 2, K + 40), float("nan"), device=DEV, dtype=torch.bfloat16)
    x = xb[1:M + 1, 8:K + 8]
    x.copy_(_x(M, K))
    for dt, ot in ((torch.float32, moe.MOE_OUT_F32), (torch.bfloat16, moe.MOE_OUT_BF16)):
        ob = torch.full((M + 2, N + 3), 77.0, device=DEV, dtype=dt)
        out = ob[1:M + 1, 1:N + 1]
        sh = moe.MoeLinearShape.of(M, N, K, ldx=xb.stride(0), ldo=ob.stride(0), out_type=ot)
        ws, n = _workspace(sh)
        moe.moe_linear_w4(sh, x, mat.packed, None, out, ws, n)
        _check(out, x, mat)
        ob[1:M + 1, 1:N + 1] = 77.0
        assert bool((ob == 77.0).all())


def test_ranges_of_values():
    """Zero rows, subnormal and huge activations, blocks over many binades, extreme weight scales."""
    N, K = 256, 512
    mat = Matrix(N, K, seed=9)
    x = _x(12, K).float()
    x[0] = 0.0
    x[1] *= 1e-30
    x[2] = torch.randn(K, device=DEV) * 1e-38          # subnormal bf16 among them
    x[3] *= 1e30
    x[4] *= torch.exp2(-torch.arange(K, device=DEV) % 32.0)
    x[5, 1:] = 0.0
    x[6] = 3.0e38 * torch.sign(torch.randn(K, device=DEV)) * (torch.arange(K, device=DEV) % 32 == 0)
    x[7, ::2] = -0.0
    x = x.bfloat16()
    x[8] = torch.tensor([0x0001, 0x8001, 0x0080, 0x7F7F], dtype=torch.int32).to(torch.int16).view(torch.bfloat16).to(DEV).repeat(K // 4)
    x[8, K // 2:] = 0
    lo = x.clone()
    lo[3] = 0
    lo[6] = 0
    lo[8] = 0
    _run(12, N, K, moe.MOE_OUT_F32, mat=mat, x=lo)
    got = _run_raw(x, mat)
    y = x.double() @ mat.w.T
    fits = x.double().abs() @ mat.w.abs().T < 3.3e38   # else an fp32 partial sum may overflow where the sum does not
    assert bool(fits[3].all()) and bool(fits[6].any())
    _, tol = linear_ref(x, mat.w)
    assert bool(((got.double() - y).abs()[fits] <= tol[fits]).all())
    tiny = Matrix(128, 128, seed=2, lo=0, hi=3)        # scales 2^-127 ..
    _run(3, 128, 128, moe.MOE_OUT_F32, mat=tiny, x=(_x(3, 128).float() * 1e30).bfloat16())
    large = Matrix(128, 128, seed=2, lo=250, hi=255)   # .. 2^127
    _run(3, 128, 128, moe.MOE_OUT_F32, mat=large, x=(_x(3, 128).float() * 1e-8).bfloat16())


def _run_raw(x, mat, out_type=moe.MOE_OUT_F32):
    M = x.shape[0]
    sh = moe.MoeLinearShape.of(M, mat.N, mat.K, out_type=out_type)
    ws, n = _workspace(sh)
    out = torch.empty(M, mat.N, device=DEV)
    moe.moe_linear_w4(sh, x, mat.packed, None, out, ws, n)
    assert moe.moe_get_status(ws) == (moe.MOE_OK, 0)
    return out


@pytest.mark.parametrize("M", [4, 16, 40])
def test_a_token_that_is_not_finite_is_nan_alone(M):
    mat = Matrix(640, 768, seed=4)
    clean = _x(M, 768, seed=8)
    want = _run_raw(clean, mat)
    for v in (float("inf"), float("-inf"), float("nan")):
        x = clean.clone()
        x[M // 2, 500] = v
        got = _run_raw(x, mat)
        assert bool(got[M // 2].isnan().all())
        keep = torch.arange(M, device=DEV) != M // 2
        assert torch.equal(got[keep], want[keep])


def test_a_tensor_that_covers_all_codes_is_packed_in_place():
    """The packed layout, byte by byte, padding included."""
    N, K = 130, 160
    mat = Matrix(N, K, seed=6)
    got = mat.packed.cpu()
    RT, KC = 2, 2
    codes = got[:RT * KC * 8192].reshape(RT, KC, 128, 64)
    sf = got[RT * KC * 8192:].reshape(RT, KC, 512)
    c, s = mat.codes.cpu(), mat.scales.cpu()
    for n in (0, 1, 31, 32, 127, 128, 129):
        for k in (0, 32, 96, 128):
            want = c[n, k // 2:k // 2 + 16]
            at = (k % 128) // 2
            assert torch.equal(codes[n // 128, k // 128, n % 128, at:at + 16], want)
            r = n % 128
            assert sf[n // 128, k // 128, 16 * (r % 32) + 4 * (r // 32) + (k % 128) // 32] == s[n, k // 32]
    assert int(codes[1, :, 2:].sum()) == 0 and int(codes[:, 1, :, 16:].sum()) == 0


def test_same_bits_every_time_and_one_workspace_for_many_shapes():
    shapes = [(1, 6144, 2048), (20, 1000, 2048), (64, 130, 512), (8, 12000, 512), (16, 2048, 2048), (130, 256, 96)]
    mats = [Matrix(N, K, seed=i) for i, (_, N, K) in enumerate(shapes)]
    shs = [moe.MoeLinearShape.of(*s, out_type=moe.MOE_OUT_F32) for s in shapes]
    ws = _workspace(*shs)
    first = {}
    for turn in range(4):
        for i, (M, N, K) in enumerate(shapes):
            out = _run(M, N, K, moe.MOE_OUT_F32, mat=mats[i], ws=ws)
            if turn:
                assert torch.equal(out, first[i])
            first[i] = out


@pytest.mark.parametrize("M", [3, 24])
def test_captured_and_replayed_with_new_inputs(M):
    N, K = 2000, 1024
    mat = Matrix(N, K, seed=7)
    sh = moe.MoeLinearShape.of(M, N, K, out_type=moe.MOE_OUT_F32)
    ws, n = _workspace(sh)
    x = _x(M, K)
    out = torch.empty(M, N, device=DEV)
    torch.cuda.synchronize()   # the inputs were made on another stream
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        moe.moe_linear_w4(sh, x, mat.packed, None, out, ws, n)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(3):
                moe.moe_linear_w4(sh, x, mat.packed, None, out, ws, n)
        for seed in range(5):
            x.copy_(_x(M, K, seed=20 + seed))
            out.zero_()
            g.replay()
            st.synchronize()
            _check(out, x, mat)


def test_the_first_call_of_a_process_is_captured():
    code = """
import sys; sys.path.insert(0, 'tests')
import torch
import test_gpu_linear_w4 as t
import prefill_moe_route_b200 as moe
for M in (2, 40):
    mat = t.Matrix(500, 640)
    sh = moe.MoeLinearShape.of(M, 500, 640, out_type=moe.MOE_OUT_F32)
    ws, n = t._workspace(sh)
    x, out = t._x(M, 640), torch.empty(M, 500, device='cuda')
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_linear_w4(sh, x, mat.packed, None, out, ws, n)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    t._check(out, x, mat)
print('child ok')
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "child ok" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]


def test_a_chain_rewrites_its_own_input():
    """x is overwritten between the calls by kernels of the same stream, the library's and others."""
    N = K = 1024
    mat = Matrix(N, K, seed=3, lo=113, hi=116)
    sh = moe.MoeLinearShape.of(6, N, K)
    ws, n = _workspace(sh)
    a, b = _x(6, K), torch.empty(6, N, device=DEV, dtype=torch.bfloat16)
    want = a.clone()
    for i in range(30):
        moe.moe_linear_w4(sh, a, mat.packed, None, b, ws, n)
        moe.moe_linear_w4(sh, b, mat.packed, None, a, ws, n)
        if i % 3 == 0:
            a.mul_(0.5)
    got = a.clone()
    x = want
    for i in range(30):
        for _ in range(2):
            y = torch.empty_like(x)
            torch.cuda.synchronize()
            moe.moe_linear_w4(sh, x, mat.packed, None, y, ws, n)
            torch.cuda.synchronize()
            x = y
        if i % 3 == 0:
            x = x * 0.5
    assert torch.equal(got, x)


def test_two_calls_at_once():
    """Two streams, a workspace each, enough calls that they overlap; and a chain
    whose input is the call before's output."""
    N = K = 2048
    mats = [Matrix(N, K, seed=i, lo=113, hi=116) for i in range(2)]
    sh = moe.MoeLinearShape.of(4, N, K)
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    bufs = []
    for i in range(2):
        ws, n = _workspace(sh)
        bufs.append(([_x(4, K, seed=i)] + [torch.empty(4, N, device=DEV, dtype=torch.bfloat16) for _ in range(20)], ws, n))
    torch.cuda.synchronize()
    for j in range(20):
        for i in range(2):
            b, ws, n = bufs[i]
            moe.moe_linear_w4(sh, b[j], mats[i].packed, None, b[j + 1], ws, n, stream=st[i])
    torch.cuda.synchronize()
    for i in range(2):
        b, ws, _ = bufs[i]
        assert moe.moe_get_status(ws) == (moe.MOE_OK, 0)
        for j in range(20):
            _check(b[j + 1], b[j], mats[i])


def test_refusals_on_the_device():
    mat = Matrix(128, 128)
    x, out = _x(2, 128), torch.empty(2, 128, device=DEV, dtype=torch.bfloat16)
    sh = moe.MoeLinearShape.of(2, 128, 128)
    ws, n = _workspace(sh)
    assert moe.moe_linear_w4(sh, x, mat.packed, None, out, ws, n - 1, check=False) == moe.MOE_ERR_WORKSPACE
    host = torch.empty(4096, dtype=torch.uint8).data_ptr() // 256 * 256 + 256
    assert moe.moe_linear_w4(sh, x, mat.packed, None, out, host, n, check=False) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_linear_w4(sh, x.data_ptr() + 2, mat.packed, None, out, ws, n, check=False) == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("M", [2, 8, 16, 32, 70])
def test_a_part_that_never_comes_ends_in_a_status(M):
    """A withheld part of a sum: the waits on it run out, the call ends, the
    status says so; after a zero-fill the workspace serves again."""
    code = """
import sys; sys.path.insert(0, 'tests')
import torch
import test_gpu_linear_w4 as t
import prefill_moe_route_b200 as moe
mat = t.Matrix(1024, 4096)
M = int(sys.argv[1])
sh = moe.MoeLinearShape.of(M, 1024, 4096, out_type=moe.MOE_OUT_F32)
ws, n = t._workspace(sh)
out = torch.empty(M, 1024, device='cuda')
moe.moe_linear_w4(sh, t._x(M, 4096), mat.packed, None, out, ws, n)
rc, st = moe.moe_get_status(ws)
assert rc == moe.MOE_ERR_DEVICE_TIMEOUT and st == 1, (rc, st)
moe.moe_workspace_init(ws, n)
t._run(M, 1024, 4096, moe.MOE_OUT_F32, mat=mat, ws=(ws, n))
print('child ok')
"""
    env = dict(os.environ, MOE_TEST_WITHHOLD_FLAG="1", MOE_WAIT_TIMEOUT_MS="20")
    r = subprocess.run([sys.executable, "-c", code, str(M)], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "child ok" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]


@pytest.mark.parametrize("M", [1, 7, 16, 20, 70])
def test_x_and_out_as_columns_of_one_buffer(M):
    N, K = 259, 480
    mat = Matrix(N, K, seed=3)
    buf = torch.full((M, 768), 77.0, device=DEV, dtype=torch.bfloat16)
    x, out = buf[:, :K], buf[:, 488:488 + N]
    x.copy_(_x(M, K))
    sh = moe.MoeLinearShape.of(M, N, K, ldx=768, ldo=768)
    ws, n = _workspace(sh)
    moe.moe_linear_w4(sh, x, mat.packed, None, out, ws, n)
    _check(out, x, mat)
    assert bool((buf[:, K:488] == 77.0).all()) and bool((buf[:, 488 + N:] == 77.0).all())
    over = moe.moe_linear_w4(sh, x, mat.packed, None, buf[:, K - 2:], ws, n, check=False)
    assert over == moe.MOE_ERR_INVALID_ARG
