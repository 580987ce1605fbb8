"""The few-token operators when the GPU's timing is not the usual one: CTAs that come
late, streams beside the call's own."""
import hashlib
import os
import subprocess
import sys

import pytest
import torch

import prefill_moe_route_b200 as moe
from conftest import ROOT
from test_gpu_layer_w4 import Layer

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _child(code, *args, **env):
    r = subprocess.run([sys.executable, "-c", "import sys; sys.path.insert(0, 'tests')\n" + code, *map(str, args)], cwd=ROOT,
                       env=dict(os.environ, **env), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "child ok" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
    return r.stdout


def digest(tensors):
    h = hashlib.sha256()
    for t in tensors:
        h.update(t.contiguous().view(torch.uint8).cpu().numpy().tobytes())
    return h.hexdigest()


LATE = """
import test_gpu_layer_w4 as t
import test_gpu_w4_timing as tt
import prefill_moe_route_b200 as moe
L = t.Layer(*eval(sys.argv[2]))
ws = L.workspace()
for turn in range(3):
    x = L.x(int(sys.argv[1]), seed=turn)
    got = L.run(x, ws)
    assert moe.moe_get_status(ws[0]) == (moe.MOE_OK, 0), turn
    L.check(x, got)
    print('bits', tt.digest(got))
print('child ok')
"""


@pytest.mark.parametrize("M", [1, 4, 8, 16])
@pytest.mark.parametrize("shape", [(512, 8, 2, 256), (2048, 64, 8, 256, 256)])
def test_a_block_that_routes_late_finds_its_sigmoids(M, shape):
    """One CTA looks for the sigmoids long after the others have routed and, in the
    small layer (fewer shares than CTAs), have drawn all there is to do."""
    out = _child(LATE, M, shape, MOE_TEST_HOLD_ROUTING_US="100", MOE_WAIT_TIMEOUT_MS="50")
    L = Layer(*shape)
    ws = L.workspace()
    want = [digest(L.run(L.x(M, seed=turn), ws)) for turn in range(3)]
    assert [line.split()[1] for line in out.splitlines() if line.startswith("bits")] == want


@pytest.mark.parametrize("M", [1, 4, 8, 16])
@pytest.mark.parametrize("shape", [(512, 8, 2, 256), (2048, 64, 8, 256, 256)])
def test_beside_a_stream_that_fills_the_gpu(M, shape):
    """Another stream's products hold SMs, so that CTAs of the layer start at all times."""
    L = Layer(*shape)
    ws = L.workspace()
    xs = [L.x(M, seed=j) for j in range(4)]
    want = [L.run(x, ws) for x in xs]
    a = torch.randn(3000, 3000, device=DEV, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for turn in range(25):
        with torch.cuda.stream(other):
            for _ in range(8):
                a = (a @ a) * 1e-2
        for x, w in zip(xs, want):
            got = L.run(x, ws)
            assert moe.moe_get_status(ws[0]) == (moe.MOE_OK, 0)
            assert all(torch.equal(p, q) for p, q in zip(got, w))
    torch.cuda.synchronize()


SLOW_PREDECESSOR = """
import torch
import test_gpu_linear_w4 as tl
import test_gpu_layer_w4 as ty
import prefill_moe_route_b200 as moe
# holds its stream 50 ms and lets its successors start at once
spin = torch.cuda._compile_kernel('''
extern "C" __global__ void spin(long long ns) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  long long t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  for (int i = 0; i < 100000000; ++i) {
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    if (t - t0 > ns) break;
  }
}''', 'spin')
M = int(sys.argv[1])
mat = tl.Matrix(1000, 1024)
sh = moe.MoeLinearShape.of(M, 1000, 1024, out_type=moe.MOE_OUT_F32)
ws, n = tl._workspace(sh)
x, out = tl._x(M, 1024), torch.empty(M, 1000, device='cuda')
L = ty.Layer(512, 8, 2, 256)
lws = L.workspace()
for turn in range(2):
    torch.cuda.synchronize()
    spin((1, 1, 1), (32, 1, 1), (50000000,))
    moe.moe_linear_w4(sh, x, mat.packed, None, out, ws, n)
    assert moe.moe_get_status(ws) == (moe.MOE_OK, 0), turn
    tl._check(out, x, mat)
    if M <= 16:
        y = L.x(M, seed=turn)
        torch.cuda.synchronize()
        spin((1, 1, 1), (32, 1, 1), (50000000,))
        got = L.run(y, lws)
        assert moe.moe_get_status(lws[0]) == (moe.MOE_OK, 0), turn
        L.check(y, got)
print('child ok')
"""


@pytest.mark.parametrize("M", [2, 8, 16, 32, 70])
def test_a_slow_kernel_before_the_call_is_not_a_wait_of_the_call(M):
    """The kernel before takes ten times a wait's limit and lets the call's kernels start beside it."""
    _child(SLOW_PREDECESSOR, M, MOE_WAIT_TIMEOUT_MS="5")


LONG_LINEAR = """
import torch
import test_gpu_linear_w4 as tl
import prefill_moe_route_b200 as moe
M, N, K = 131072, 6144, 6144
mat = tl.Matrix(N, K)
x = torch.cat([tl._x(4096, K, seed=i) for i in range(32)])
sh = moe.MoeLinearShape.of(M, N, K)
ws, n = tl._workspace(sh)
out = torch.empty(M, N, device='cuda', dtype=torch.bfloat16)
for turn in range(2):
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    moe.moe_linear_w4(sh, x, mat.packed, None, out, ws, n)
    b.record()
    assert moe.moe_get_status(ws) == (moe.MOE_OK, 0), turn
    assert a.elapsed_time(b) > 3.0, a.elapsed_time(b)   # several times the limit of a wait
rows = torch.arange(5, M, 997, device='cuda')
tl._check(out[rows], x[rows], mat)
print('child ok')
"""

LONG_LAYER = """
import torch
import test_gpu_layer_w4 as ty
import prefill_moe_route_b200 as moe
L = ty.Layer(16384, 64, 16, 8192)
ws = L.workspace()
x = L.x(int(sys.argv[1]))
for turn in range(2):
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    got = L.run(x, ws)
    b.record()
    assert moe.moe_get_status(ws[0]) == (moe.MOE_OK, 0), turn
    assert a.elapsed_time(b) > 1.2, a.elapsed_time(b)   # past the limit of a wait
L.check(x, got)
print('child ok')
"""


def test_a_product_may_take_longer_than_a_wait():
    _child(LONG_LINEAR, MOE_WAIT_TIMEOUT_MS="1")


@pytest.mark.parametrize("M", [4, 8])
def test_a_layer_may_take_longer_than_a_wait(M):
    _child(LONG_LAYER, M, MOE_WAIT_TIMEOUT_MS="1")


@pytest.mark.parametrize("M", [1, 4, 8, 16])
@pytest.mark.parametrize("shape", [(512, 8, 2, 256), (2048, 64, 8, 256, 256)])
def test_a_call_leaves_what_the_next_one_starts_from(M, shape):
    """The task counter and the count of routed CTAs are zero when a call has ended: the
    next call's kernels read them before any kernel of that call has ended."""
    L = Layer(*shape)
    ws = L.workspace()
    for turn in range(5):
        L.run(L.x(M, seed=turn), ws)
        words = ws[0][:256].view(torch.int32).tolist()
        assert words[16] == 0 and words[18] == 0 and words[:3] == [0, 0, 0], turn
    assert moe.moe_get_status(ws[0]) == (moe.MOE_OK, 0)


USED_UP = """
import torch
import test_gpu_linear_w4 as tl
import test_gpu_layer_w4 as ty
import prefill_moe_route_b200 as moe
op, M = sys.argv[1], int(sys.argv[2])
if op == 'linear':
    mat = tl.Matrix(1024, 4096)
    sh = moe.MoeLinearShape.of(M, 1024, 4096, out_type=moe.MOE_OUT_F32)
    ws, n = tl._workspace(sh)
    x, out = tl._x(M, 4096), torch.empty(M, 1024, device='cuda')
    call = lambda: moe.moe_linear_w4(sh, x, mat.packed, None, out, ws, n)
    check = lambda: tl._check(out, x, mat)
else:
    L = ty.Layer(1024, 16, 4, 256, 128)
    ws, n = L.workspace()
    x = L.x(M)
    got = []
    call = lambda: got.append(L.run(x, (ws, n)))
    check = lambda: L.check(x, got[-1])
call()   # one hand-over of this call is withheld
assert moe.moe_get_status(ws) == (moe.MOE_ERR_DEVICE_TIMEOUT, 1)
for turn in range(3):   # the workspace is not what a call starts from: each says so
    call()
    assert moe.moe_get_status(ws) == (moe.MOE_ERR_DEVICE_TIMEOUT, 1), turn
moe.moe_workspace_init(ws, n)
for turn in range(2):
    call()
    assert moe.moe_get_status(ws) == (moe.MOE_OK, 0)
    check()
print('child ok')
"""


@pytest.mark.parametrize("op,M", [("linear", 2), ("linear", 16), ("linear", 70), ("layer", 1), ("layer", 4), ("layer", 8), ("layer", 16)])
def test_a_workspace_that_was_given_up_on_says_so_until_it_is_zero_filled(op, M):
    _child(USED_UP, op, M, MOE_TEST_WITHHOLD_FLAG="1", MOE_WAIT_TIMEOUT_MS="20")


@pytest.mark.parametrize("M", [1, 4, 8, 16])
def test_captured_behind_copies_fills_and_joined_streams(M):
    """The node before a call in a graph is a copy, a fill, or kernels of two streams that
    meet there; two calls of one graph run side by side."""
    from test_gpu_linear_w4 import Matrix, _check, _workspace, _x
    L = Layer(512, 8, 2, 256)
    mats = [Matrix(512, 512, seed=i, lo=113, hi=116) for i in range(2)]
    sh = moe.MoeLinearShape.of(M, 512, 512)
    spaces = [_workspace(sh) for _ in range(2)]
    lws = L.workspace()
    src, x, h = (_x(M, 512, seed=i, loud=False) for i in range(3))
    a, b, y = (torch.empty_like(x) for _ in range(3))
    ids, wts = torch.empty(M, 2, device=DEV, dtype=torch.int32), torch.empty(M, 2, device=DEV)
    noise = torch.randn(2048, 2048, device=DEV)
    lsh = L.shape(M)

    def step(main, side):
        x.copy_(src)                                                    # a copy node
        moe.moe_linear_w4(sh, x, mats[0].packed, None, a, *spaces[0])
        side.wait_stream(main)
        with torch.cuda.stream(side):                                   # a branch that ends later
            noise @ noise
            b.zero_()
            moe.moe_linear_w4(sh, a, mats[1].packed, None, b, *spaces[1])
        moe.moe_linear_w4(sh, src, mats[1].packed, None, h, *spaces[0])
        main.wait_stream(side)
        moe.moe_layer_w4(lsh, L.weights, b, y, ids, wts, *lws)          # behind both branches
        a.zero_()                                                       # a fill node
        moe.moe_linear_w4(sh, y, mats[0].packed, None, a, *spaces[1])

    torch.cuda.synchronize()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(main):
        step(main, side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=main):
            step(main, side)
        for turn in range(6):
            src.copy_(_x(M, 512, seed=50 + turn, loud=False))
            for t in (x, a, b, y, h):
                t.fill_(7.0)
            g.replay()
            main.synchronize()
            want = torch.empty_like(x)
            moe.moe_linear_w4(sh, src, mats[0].packed, None, want, *spaces[0])
            main.synchronize()
            _check(b, want, mats[1])
            _check(h, src, mats[1])
            L.check(b, (y, ids, wts))
            _check(a, y, mats[0])
    for ws in (spaces[0][0], spaces[1][0], lws[0]):
        assert moe.moe_get_status(ws) == (moe.MOE_OK, 0)
