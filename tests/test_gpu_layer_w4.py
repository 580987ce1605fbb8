"""moe_layer_w4 (a whole MoE layer for a few tokens) against its definition in 64 bits."""
import os
import subprocess
import sys

import pytest
import torch

import prefill_moe_route_b200 as moe
from conftest import ROOT
from w4_ref import layer_ref, linear_ref, rand_mx, value64

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _packed(scales, rows, K):
    p = torch.empty_like(scales)
    moe.moe_pack_mxfp4_scales(scales, scales.shape[0], rows, K, p)
    return p


class Layer:
    """Weights of one layer on the GPU; run() calls the library, check() compares."""

    def __init__(self, H, E, topk, I, S=0, norm=True, bias=True, residual=True, scale=2.5, seed=0, eps=1e-5):
        self.H, self.E, self.topk, self.I, self.S = H, E, topk, I, S
        self.scale, self.residual, self.eps = scale, residual, eps
        g = _gen(seed)
        self.w13, self.s13 = rand_mx(g, E, 2 * I, H, lo=118, hi=121)
        self.w2, self.s2 = rand_mx(g, E, H, I, lo=118, hi=121)
        self.router_w = (torch.randn(E, H, generator=g, device=DEV) * 2.0 / H ** 0.5).bfloat16()
        self.norm_w = (1 + 0.2 * torch.randn(H, generator=g, device=DEV)).bfloat16() if norm else None
        self.bias = 0.1 * torch.randn(E, generator=g, device=DEV) if bias else None
        self.sh = None
        if S:
            self.sh = (*rand_mx(g, 1, 2 * S, H, lo=118, hi=121), *rand_mx(g, 1, H, S, lo=118, hi=121))
        self.bind()

    def bind(self):
        sh = self.sh
        self.sf13, self.sf2 = _packed(self.s13, 2 * self.I, self.H), _packed(self.s2, self.H, self.I)
        self.weights = moe.MoeLayerWeights.of(
            router_w=self.router_w, norm_w=self.norm_w, bias=self.bias, w13=self.w13, w13_scales=self.sf13, w2=self.w2,
            w2_scales=self.sf2, shared_w13=sh and sh[0], shared_w13_scales=sh and _packed(sh[1], 2 * self.S, self.H),
            shared_w2=sh and sh[2], shared_w2_scales=sh and _packed(sh[3], self.H, self.S))

    def shape(self, M, ldx=None, ldo=None):
        return moe.MoeLayerShape.of(M, self.H, self.I, self.E, self.topk, self.scale, shared_I=self.S, norm_eps=self.eps,
                                    add_residual=self.residual, ldx=ldx, ldo=ldo)

    def workspace(self):
        n = moe.moe_layer_w4_workspace_size(self.shape(1))
        ws = torch.empty(n, device=DEV, dtype=torch.uint8)
        moe.moe_workspace_init(ws, n)
        return ws, n

    def x(self, M, seed=1):
        return torch.randn(M, self.H, generator=_gen(seed), device=DEV).bfloat16()

    def run(self, x, ws, stream=None, out=None):
        M = x.shape[0]
        out = torch.empty(M, self.H, device=DEV, dtype=torch.bfloat16) if out is None else out
        ids = torch.empty(M, self.topk, device=DEV, dtype=torch.int32)
        wts = torch.empty(M, self.topk, device=DEV)
        moe.moe_layer_w4(self.shape(M, x.stride(0), out.stride(0)), self.weights, x, out, ids, wts, *ws, stream)
        return out, ids, wts

    def check(self, x, got):
        out, ids, wts = got
        e13 = lambda e: (value64(self.w13[e], self.s13[e]), value64(self.w2[e], self.s2[e]))
        sh = (value64(self.sh[0][0], self.sh[1][0]), value64(self.sh[2][0], self.sh[3][0])) if self.sh else None
        assert int(ids.min()) >= 0 and int(ids.max()) < self.E
        assert all(len(set(r)) == self.topk for r in ids.tolist())
        args = (x, self.norm_w, self.eps, self.router_w, self.bias, self.topk, self.scale, e13, sh, self.residual)
        y, tol, ids64, _, margin = layer_ref(*args)
        # an fp32 logit is off by less than 1e-5 here and a sigmoid moves by a quarter of it at most
        sure = margin > 1e-5
        assert int(sure.sum()) * 2 >= len(x)
        assert torch.equal(ids[sure].long(), ids64[sure])
        y, tol, _, w, _ = layer_ref(*args, ids=ids)
        assert bool(((wts.double() - w).abs() <= 1e-5 * w.abs() + 1e-7).all())
        d = (out.double() - y).abs()
        assert bool((d <= tol + 2.0 ** -8 * y.abs()).all()), f"worst {float((d - tol - 2.0 ** -8 * y.abs()).max()):.3g}"
        # over all outputs: bf16 (2^-8 / sqrt 3), h and mid to 2^-9 each, signs at random: well under 2^-8
        assert float(d.norm()) <= 2.0 ** -8 * float(y.norm())


CASES = [
    # M, H, E, topk, I, S, norm, bias, residual
    (1, 128, 1, 1, 128, 0, False, False, False),
    (1, 128, 4, 1, 128, 0, True, True, True),
    (16, 128, 4, 4, 128, 128, True, True, False),
    (2, 256, 8, 2, 256, 0, False, True, True),
    (3, 384, 13, 5, 128, 256, True, False, True),
    (4, 512, 8, 2, 256, 0, False, True, False),
    (5, 2176, 40, 3, 384, 128, True, False, True),
    (7, 1024, 33, 8, 640, 0, True, True, True),
    (8, 640, 300, 8, 128, 384, True, True, True),
    (9, 768, 512, 16, 128, 128, True, True, True),
    (11, 1280, 96, 6, 256, 512, False, False, False),
    (13, 896, 64, 12, 256, 128, True, True, False),
    (15, 256, 257, 9, 128, 0, True, True, True),
    (16, 2048, 128, 8, 384, 256, True, True, True),
    (16, 512, 512, 16, 128, 0, False, True, False),
    (1, 6144, 64, 8, 256, 256, True, False, True),
    (2, 8192, 12, 3, 1024, 0, True, True, False),
    (10, 3328, 20, 2, 1152, 640, False, True, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "M%d_H%d_E%d_k%d_I%d_S%d" % c[:6])
def test_against_64_bits(case):
    M, H, E, topk, I, S, norm, bias, residual = case
    L = Layer(H, E, topk, I, S, norm, bias, residual, seed=M + H)
    ws = L.workspace()
    for seed in (1, 2):
        x = L.x(M, seed)
        got = L.run(x, ws)
        assert moe.moe_get_status(ws[0]) == (moe.MOE_OK, 0)
        L.check(x, got)


def test_every_token_count_on_one_workspace():
    L = Layer(512, 32, 4, 256, 128)
    ws = L.workspace()
    for M in list(range(1, 17)) + [3, 16, 1, 9, 8]:
        x = L.x(M, seed=M)
        L.check(x, L.run(x, ws))
    assert moe.moe_get_status(ws[0]) == (moe.MOE_OK, 0)


def test_other_shapes_on_one_workspace_and_the_same_bits_every_time():
    Ls = [Layer(512, 32, 4, 256, 128), Layer(2048, 8, 2, 128, 512), Layer(1152, 200, 7, 384, 0, norm=False)]
    n = max(moe.moe_layer_w4_workspace_size(L.shape(1)) for L in Ls)
    ws = torch.empty(n, device=DEV, dtype=torch.uint8)
    moe.moe_workspace_init(ws, n)
    first = {}
    for turn in range(4):
        for i, L in enumerate(Ls):
            for M in (1, 6, 16):
                x = L.x(M, seed=M)
                got = L.run(x, (ws, n))
                if turn == 0:
                    L.check(x, got)
                    first[i, M] = got
                assert all(torch.equal(a, b) for a, b in zip(got, first[i, M]))


@pytest.mark.parametrize("M", [1, 6, 12])
def test_rows_inside_larger_buffers(M):
    L = Layer(384, 16, 3, 128, 128)
    xb = torch.full((M + 2, 384 + 24), float("nan"), device=DEV, dtype=torch.bfloat16)
    ob = torch.full((M + 2, 384 + 5), 77.0, device=DEV, dtype=torch.bfloat16)
    x, out = xb[1:M + 1, 8:392], ob[1:M + 1, 3:387]
    x.copy_(L.x(M))
    L.check(x, L.run(x, L.workspace(), out=out))
    out.fill_(77.0)
    assert bool((ob == 77.0).all())


def test_ties_go_to_the_lower_expert():
    L = Layer(256, 24, 5, 128, bias=False)
    L.router_w[:] = L.router_w[0].clone()
    L.router_w[7] = 0   # sigmoid 1/2, above or below the tied rest
    x = L.x(6)
    out, ids, _ = L.run(x, L.workspace())
    h = x.double() / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + L.eps) * L.norm_w.double()
    rest = [e for e in range(24) if e != 7]
    for t, logit in enumerate((h @ L.router_w[0].double()).tolist()):
        want = rest[:5] if logit > 0 else [7] + rest[:4]
        assert ids[t].tolist() == want
    L2 = Layer(256, 24, 5, 128, norm=False, bias=False)
    L2.router_w.zero_()
    assert L2.run(x, L2.workspace())[1].tolist() == [[0, 1, 2, 3, 4]] * 6


def test_zero_tokens_and_wide_ranges():
    L = Layer(512, 16, 4, 128, 128)
    x = L.x(8).float()
    x[0] = 0.0
    x[1] *= 1e-6
    x[2] *= 1e6
    x[3, ::32] *= 4096.0
    x[4, 1:] = 0.0
    x = x.bfloat16()
    L.check(x, L.run(x, L.workspace()))


@pytest.mark.parametrize("M", [1, 2, 4, 8, 16])
def test_a_token_that_is_not_finite_is_nan_alone(M):
    L = Layer(512, 16, 4, 256, 128)
    ws = L.workspace()
    x = L.x(M)
    want = L.run(x, ws)
    bad = M // 2
    keep = torch.arange(M, device=DEV) != bad
    for v in (float("nan"), float("inf")):
        y = x.clone()
        y[bad, 100] = v
        out, ids, wts = L.run(y, ws)
        assert moe.moe_get_status(ws[0]) == (moe.MOE_OK, 0)
        assert bool(out[bad].isnan().all()) and int(ids.min()) >= 0 and int(ids.max()) < 16
        assert torch.equal(out[keep], want[0][keep]) and torch.equal(ids[keep], want[1][keep])


def test_optional_outputs_and_absent_parts():
    L = Layer(256, 8, 2, 128)
    x = L.x(3)
    ws = L.workspace()
    want = L.run(x, ws)
    out = torch.empty_like(want[0])
    moe.moe_layer_w4(L.shape(3), L.weights, x, out, None, None, *ws)
    assert torch.equal(out, want[0])


@pytest.mark.parametrize("M", [1, 4, 5, 16])
def test_captured_and_replayed_with_new_inputs(M):
    L = Layer(1024, 64, 6, 256, 256)
    ws = L.workspace()
    x, out = L.x(M), torch.empty(M, 1024, device=DEV, dtype=torch.bfloat16)
    ids, wts = torch.empty(M, 6, device=DEV, dtype=torch.int32), torch.empty(M, 6, device=DEV)
    sh = L.shape(M)
    torch.cuda.synchronize()   # the inputs were made on another stream
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        moe.moe_layer_w4(sh, L.weights, x, out, ids, wts, *ws)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(3):
                moe.moe_layer_w4(sh, L.weights, x, out, ids, wts, *ws)
        for seed in range(4):
            x.copy_(L.x(M, seed=30 + seed))
            out.zero_()
            g.replay()
            st.synchronize()
            L.check(x, (out, ids, wts))


def test_the_first_call_of_a_process_is_captured():
    code = """
import sys; sys.path.insert(0, 'tests')
import torch
import test_gpu_layer_w4 as t
import prefill_moe_route_b200 as moe
for M in (1, 2, 7, 12):
    L = t.Layer(512, 16, 4, 256, 128)
    ws = L.workspace()
    x, out = L.x(M), torch.empty(M, 512, device='cuda', dtype=torch.bfloat16)
    ids, wts = torch.empty(M, 4, device='cuda', dtype=torch.int32), torch.empty(M, 4, device='cuda')
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_layer_w4(L.shape(M), L.weights, x, out, ids, wts, *ws)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    L.check(x, (out, ids, wts))
print('child ok')
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "child ok" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]


def test_a_chain_of_layers_on_one_buffer_pair():
    """h goes back and forth through the layer; another stream's kernels run meanwhile."""
    L = Layer(1024, 32, 4, 256, 128)
    ws = L.workspace()
    a, b = L.x(5), torch.empty(5, 1024, device=DEV, dtype=torch.bfloat16)
    x = a.clone()
    torch.cuda.synchronize()
    other, busy = torch.cuda.Stream(), torch.randn(2048, 2048, device=DEV)
    for i in range(20):
        with torch.cuda.stream(other):
            busy = busy @ busy * 1e-3
        L.run(a, ws, out=b)
        L.run(b, ws, out=a)
    torch.cuda.synchronize()
    for i in range(40):
        x = L.run(x, ws)[0]
        torch.cuda.synchronize()
    assert torch.equal(a, x) and moe.moe_get_status(ws[0]) == (moe.MOE_OK, 0)


def test_two_calls_at_once():
    """Two streams with a workspace each: the kernels share the SMs and must not wait for each other."""
    Ls = [Layer(2048, 64, 8, 256, 256, seed=1), Layer(2048, 64, 8, 256, 256, seed=2)]
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [L.workspace() for L in Ls]
    xs = [[L.x(8, seed=j) for j in range(25)] for L in Ls]
    torch.cuda.synchronize()
    got = [[], []]
    for j in range(25):
        for i in range(2):
            with torch.cuda.stream(st[i]):
                got[i].append(Ls[i].run(xs[i][j], ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert moe.moe_get_status(ws[i][0]) == (moe.MOE_OK, 0)
        for j in range(0, 25, 6):
            Ls[i].check(xs[i][j], got[i][j])


def test_a_decode_step_of_projection_layer_and_logits():
    """The operators as a program chains them: projection, layer, vocabulary logits, each
    reading what the one before wrote, captured once and replayed."""
    M, H, K, V = 4, 1024, 768, 3001
    L = Layer(H, 32, 4, 256, 256)
    g = _gen(3)
    mats = []
    for N, k in ((H, K), (V, H)):
        c, s = rand_mx(g, N, k, lo=118, hi=121)
        p = torch.empty(moe.moe_w4_packed_size(N, k), device=DEV, dtype=torch.uint8)
        moe.moe_pack_w4(c, s, N, k, p)
        mats.append((p, value64(c, s)))
    sa, sb = moe.MoeLinearShape.of(M, H, K), moe.MoeLinearShape.of(M, V, H, out_type=moe.MOE_OUT_F32)
    n = moe.moe_linear_w4_workspace_size(sa)
    lw = torch.empty(n, device=DEV, dtype=torch.uint8)
    moe.moe_workspace_init(lw, n)
    ws = L.workspace()
    a = torch.randn(M, K, generator=g, device=DEV).bfloat16()
    h, y = torch.empty(M, H, device=DEV, dtype=torch.bfloat16), torch.empty(M, H, device=DEV, dtype=torch.bfloat16)
    ids, wts = torch.empty(M, 4, device=DEV, dtype=torch.int32), torch.empty(M, 4, device=DEV)
    logits = torch.empty(M, V, device=DEV)

    def step():
        moe.moe_linear_w4(sa, a, mats[0][0], None, h, lw, n)
        moe.moe_layer_w4(L.shape(M), L.weights, h, y, ids, wts, *ws)
        moe.moe_linear_w4(sb, y, mats[1][0], None, logits, lw, n)

    torch.cuda.synchronize()   # the inputs were made on another stream
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step()
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            step()
        for seed in range(3):
            a.copy_(torch.randn(M, K, generator=_gen(40 + seed), device=DEV).bfloat16())
            for t in (h, y, logits):
                t.zero_()
            graph.replay()
            st.synchronize()
            ref, tol = linear_ref(a, mats[0][1])
            assert bool(((h.double() - ref).abs() <= tol + 2.0 ** -8 * ref.abs()).all())
            L.check(h, (y, ids, wts))
            ref, tol = linear_ref(y, mats[1][1])
            assert bool(((logits.double() - ref).abs() <= tol).all())


def test_the_weights_of_moe_forward_serve_as_they_are():
    """One copy of an expert's weights: the layer and moe_forward_routed read the same
    buffers; moe_forward quantizes its activations, so its result is only near."""
    L = Layer(1024, 16, 4, 256, norm=False, residual=False)
    x = L.x(8)
    out, ids, wts = L.run(x, L.workspace())
    sh = dict(M=8, H=1024, I=256, E=16, topk=4, routed_scale=2.5, wfmt=moe.MOE_W_MXFP4)
    n = moe.moe_workspace_size(sh)
    ws = torch.empty(n, device=DEV, dtype=torch.uint8)
    moe.moe_workspace_init(ws, n)
    y = torch.empty_like(out)
    moe.moe_forward_routed(sh, x, ids, wts, L.w13, L.sf13, L.w2, L.sf2, y, ws, n)
    cos = torch.nn.functional.cosine_similarity(out.double(), y.double(), dim=-1)
    assert float(cos.min()) > 0.95   # E2M1 keeps two significant bits of x: a relative error of about 0.1


def test_refusals_on_the_device():
    L = Layer(256, 8, 2, 128)
    x, out = L.x(2), torch.empty(2, 256, device=DEV, dtype=torch.bfloat16)
    ws, n = L.workspace()
    sh = L.shape(2)

    def rc(shape=sh, w=L.weights, xx=x, o=out, nbytes=n):
        return moe.moe_layer_w4(shape, w, xx, o, None, None, ws, nbytes, check=False)

    assert rc(nbytes=n - 1) == moe.MOE_ERR_WORKSPACE
    assert rc(o=x) == moe.MOE_ERR_INVALID_ARG
    assert rc(xx=x.cpu()) == moe.MOE_ERR_INVALID_ARG
    bad = moe.MoeLayerWeights.of(**dict(L.weights.tensors, w2=L.w2.data_ptr() + 16))
    assert rc(w=bad) == moe.MOE_ERR_INVALID_ARG
    assert rc() == moe.MOE_OK


@pytest.mark.parametrize("M", [1, 4, 8, 16])
def test_a_flag_that_never_comes_ends_in_a_status(M):
    code = """
import sys; sys.path.insert(0, 'tests')
import test_gpu_layer_w4 as t
import prefill_moe_route_b200 as moe
L = t.Layer(1024, 16, 4, 256, 128)
ws = L.workspace()
x = L.x(int(sys.argv[1]))
L.run(x, ws)
rc, st = moe.moe_get_status(ws[0])
assert rc == moe.MOE_ERR_DEVICE_TIMEOUT and st == 1, (rc, st)
moe.moe_workspace_init(*ws)
L.check(x, L.run(x, ws))
assert moe.moe_get_status(ws[0]) == (moe.MOE_OK, 0)
print('child ok')
"""
    env = dict(os.environ, MOE_TEST_WITHHOLD_FLAG="1", MOE_WAIT_TIMEOUT_MS="20")
    r = subprocess.run([sys.executable, "-c", code, str(M)], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "child ok" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
