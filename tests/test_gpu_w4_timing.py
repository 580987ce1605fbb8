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
