"""Cases of the few-token operators on MXFP4 weights with bf16 activations.

Two operators, each in a plain form (elementary torch operations in 32 bits, 64
where a border decides) and as the library's calls (``own``):

linear   y = x W^T (+ bias), W in MXFP4 (E2M1 codes, one E8M0 scale for 32
         values along K), x bf16 as it is.
layer    a whole mixture-of-experts layer: RMS norm, router product, sigmoid +
         bias top-k, SwiGLU experts with MXFP4 weights, an always-used shared
         expert, the residual.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases
def _linear(name, M, N, K, out="bf16", bias=False, padx=0, pado=0):
    return dict(name=name, op="linear", M=M, N=N, K=K, out=out, bias=bias, padx=padx, pado=pado)


def _layer(name, M, H, E, topk, I, shared=0, norm=True, residual=True, bias=True, scale=2.5):
    return dict(name=name, op="layer", M=M, H=H, E=E, topk=topk, I=I, shared=shared, norm=norm,
                residual=residual, bias=bias, scale=scale)


def listed():
    return [
        # one token through a small projection: nothing but latency
        _linear("linear 1x512x512", 1, 512, 512),
        # one token through a projection of the hidden state (attention output, hidden 6144)
        _linear("linear 1x6144x6144", 1, 6144, 6144),
        # one token against a slice of the vocabulary: the logits stay in 32 bits
        _linear("linear 1x40003x6144 f32", 1, 40003, 6144, out="f32"),
        # four rows of a speculative decode step through a dense gate + up projection
        _linear("linear 4x12288x6144", 4, 12288, 6144),
        # ragged: odd rows, K not a multiple of the tile, a bias, rows inside larger buffers
        _linear("linear 7x4099x2912 strided", 7, 4099, 2912, bias=True, padx=24, pado=5),
        # a batch of decoding sequences through the down projection of a dense layer
        _linear("linear 32x6144x12288", 32, 6144, 12288),
        # a short prompt in one piece
        _linear("linear 512x6144x2048", 512, 6144, 2048),
        # the small layer of the tests: routing only, no norm, no shared expert
        _layer("layer 4 tokens tiny", 4, 512, 8, 2, 256, norm=False, residual=False, scale=1.0),
        # one decoding sequence, a rank's slice of 256 experts (TP8)
        _layer("layer 1 token tp8", 1, 6144, 256, 8, 256, shared=256),
        # four rows of a speculative decode step, the same slice
        _layer("layer 4 tokens tp8", 4, 6144, 256, 8, 256, shared=256),
        # ragged: odd batch, hidden and expert counts off the powers of two
        _layer("layer 5 tokens ragged", 5, 2176, 40, 3, 384, shared=128, bias=False),
        # sixteen sequences, a rank's slice at TP4: about a hundred distinct experts
        _layer("layer 16 tokens tp4", 16, 6144, 256, 8, 512, shared=512),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        while True:
            M, N, K = _log_int(rng, 1, 512), _log_int(rng, 64, 40003), 32 * _log_int(rng, 4, 400)
            if N * K <= 32 << 20 and M * N * K <= 512 * 6144 * 2048:
                break
        c = _linear("", M, N, K, out=rng.choice(["bf16", "bf16", "f32"]), bias=rng.random() < 0.5,
                    padx=8 * rng.randrange(4), pado=rng.randrange(8))
    else:
        E = _log_int(rng, 4, 256)
        c = _layer("", _log_int(rng, 1, 16), 128 * _log_int(rng, 2, 48), E, rng.randint(1, min(E, 10)),
                   128 * rng.randint(1, 4), shared=128 * rng.randrange(5), norm=rng.random() < 0.7,
                   residual=rng.random() < 0.5, bias=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))
    del c["name"]
    return c


def _mx_bytes(rows, K):
    return rows * K // 2 + rows * K // 32


def work(case):
    c = case
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        nbytes = _mx_bytes(N, K) + 2 * M * K + M * N * (4 if c["out"] == "f32" else 2) + (4 * N if c["bias"] else 0)
        return {"bytes": nbytes, "flops": 2 * M * N * K}
    M, H, E, k, I, S = c["M"], c["H"], c["E"], c["topk"], c["I"], c["shared"]
    distinct = E * (1.0 - (1.0 - k / E) ** M)        # experts that M tokens name, independent choices
    one = _mx_bytes(2 * I, H) + _mx_bytes(H, I)
    nbytes = distinct * one + 2 * E * H + 4 * M * H + 8 * M * k + (2 * H if c["norm"] else 0)
    flops = 2 * M * E * H + M * k * 6 * H * I
    if S:
        nbytes += _mx_bytes(2 * S, H) + _mx_bytes(H, S)
        flops += M * 6 * H * S
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ the inputs
class State:
    pass


def _weights(g, *shape):
    """MXFP4 of normal weights of deviation about 0.02: the 16 codes come about equally often."""
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(119, 122, (*shape[:-1], shape[-1] // 32), generator=g, device=DEV, dtype=torch.uint8)
    return codes, scales


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV) * std


def _hidden(g, rows, width):
    """Hidden states: normal, with a few channels some times larger than the rest."""
    loud = 1.0 + 7.0 * (torch.rand(width, generator=g, device=DEV) < 0.01)
    return (_normal(g, rows, width) * loud).to(torch.bfloat16)


def prepare(case, seed):
    c, s = case, State()
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s.case = c
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        s.codes, s.scales = _weights(g, N, K)
        s.xbuf = _hidden(g, M, K + c["padx"])
        s.x = s.xbuf[:, :K]
        s.bias = _normal(g, N) if c["bias"] else None
        s.obuf = torch.zeros(M, N + c["pado"], device=DEV, dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16)
        s.out = s.obuf[:, :N]
        if own:
            import prefill_moe_route_b200 as moe
            s.shape = moe.MoeLinearShape.of(M, N, K, s.xbuf.stride(0), s.obuf.stride(0),
                                            moe.MOE_OUT_F32 if c["out"] == "f32" else moe.MOE_OUT_BF16)
            s.packed = torch.empty(moe.moe_w4_packed_size(N, K), device=DEV, dtype=torch.uint8)
            moe.moe_pack_w4(s.codes, s.scales, N, K, s.packed)
            s.ws_bytes = moe.moe_linear_w4_workspace_size(s.shape)
            s.ws = torch.empty(s.ws_bytes, device=DEV, dtype=torch.uint8)
            moe.moe_workspace_init(s.ws, s.ws_bytes)
        return s
    M, H, E, I, S = c["M"], c["H"], c["E"], c["I"], c["shared"]
    s.x = _hidden(g, M, H)
    s.norm_w = (1.0 + _normal(g, H, std=0.1)).to(torch.bfloat16) if c["norm"] else None
    s.router_w = _normal(g, E, H, std=0.02).to(torch.bfloat16)
    s.bias = _normal(g, E, std=0.1) if c["bias"] else None
    s.eps = 1e-5
    s.w13, s.s13 = _weights(g, E, 2 * I, H)
    s.w2, s.s2 = _weights(g, E, H, I)
    s.sw13 = s.ss13 = s.sw2 = s.ss2 = None
    if S:
        s.sw13, s.ss13 = _weights(g, 1, 2 * S, H)
        s.sw2, s.ss2 = _weights(g, 1, H, S)
    s.out = torch.zeros(M, H, device=DEV, dtype=torch.bfloat16)
    s.ids = torch.zeros(M, c["topk"], device=DEV, dtype=torch.int32)
    s.wts = torch.zeros(M, c["topk"], device=DEV)
    if own:
        import prefill_moe_route_b200 as moe

        def packed(scales, rows, K):
            if scales is None:
                return None
            p = torch.empty_like(scales)
            moe.moe_pack_mxfp4_scales(scales, scales.shape[0], rows, K, p)
            return p

        s.shape = moe.MoeLayerShape.of(M, H, I, E, c["topk"], c["scale"], shared_I=S, norm_eps=s.eps,
                                       add_residual=c["residual"])
        s.weights = moe.MoeLayerWeights.of(
            router_w=s.router_w, norm_w=s.norm_w, bias=s.bias, w13=s.w13, w13_scales=packed(s.s13, 2 * I, H),
            w2=s.w2, w2_scales=packed(s.s2, H, I), shared_w13=s.sw13, shared_w13_scales=packed(s.ss13, 2 * S, H),
            shared_w2=s.sw2, shared_w2_scales=packed(s.ss2, H, S))
        s.ws_bytes = moe.moe_layer_w4_workspace_size(s.shape)
        s.ws = torch.empty(s.ws_bytes, device=DEV, dtype=torch.uint8)
        moe.moe_workspace_init(s.ws, s.ws_bytes)
    return s


# ------------------------------------------------------------------ one pass
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
_table = None


def _dequant(codes, scales):
    """fp32 values of MXFP4: element 2i in the low half of byte i, one power-of-two scale for 32 values."""
    global _table
    if _table is None or _table.device != codes.device:
        _table = torch.tensor(_E2M1, device=codes.device)
    v = torch.stack((_table[(codes & 15).int()], _table[(codes >> 4).int()]), dim=-1)
    v = v.reshape(*scales.shape, 32) * torch.exp2(scales.float() - 127.0).unsqueeze(-1)
    return v.reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _plain_linear(s):
    y = s.x.float() @ _dequant(s.codes, s.scales).T
    if s.bias is not None:
        y = y + s.bias
    s.out.copy_(y)
    return s.out


def _experts(x, w13, s13, w2, s2):
    """[M, H] through each token's own experts (weights [M, n, ...]): [M, n, H]."""
    I = w13.shape[-2] // 2
    gu = (_dequant(w13, s13) @ x[:, None, :, None]).squeeze(-1)
    mid = _silu(gu[..., :I]) * gu[..., I:]
    return (_dequant(w2, s2) @ mid.unsqueeze(-1)).squeeze(-1)


def _plain_layer(s):
    c = s.case
    x = s.x.double()
    if c["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s.eps) * s.norm_w.double()
    score = torch.sigmoid(x @ s.router_w.double().T)        # 64 bits: the k-th place is a border
    pick = score if s.bias is None else score + s.bias.double()
    ids = torch.sort(pick, dim=-1, descending=True, stable=True).indices[:, :c["topk"]]
    w = torch.gather(score, 1, ids)
    w = w / w.sum(-1, keepdim=True) * c["scale"]
    x = x.float()
    y = (_experts(x, s.w13[ids], s.s13[ids], s.w2[ids], s.s2[ids]) * w.float().unsqueeze(-1)).sum(1)
    if c["shared"]:
        gu = x @ _dequant(s.sw13, s.ss13)[0].T
        mid = _silu(gu[:, :c["shared"]]) * gu[:, c["shared"]:]
        y = y + mid @ _dequant(s.sw2, s.ss2)[0].T
    if c["residual"]:
        y = y + s.x.float()
    s.out.copy_(y)
    s.ids.copy_(ids)
    s.wts.copy_(w)
    return s.out, s.ids, s.wts


def run(state):
    s = state
    if own:
        import prefill_moe_route_b200 as moe
        if s.case["op"] == "linear":
            moe.moe_linear_w4(s.shape, s.x, s.packed, s.bias, s.out, s.ws, s.ws_bytes)
            return s.out
        moe.moe_layer_w4(s.shape, s.weights, s.x, s.out, s.ids, s.wts, s.ws, s.ws_bytes)
        return s.out, s.ids, s.wts
    return _plain_linear(s) if s.case["op"] == "linear" else _plain_layer(s)


# ------------------------------------------------------------------ the definition in 64 bits
def _value64(codes, scales):
    """E2M1 from its fields: sign, two exponent bits, one fraction bit; times 2^(scale - 127)."""
    nib = torch.empty(*codes.shape, 2, dtype=torch.float64, device=codes.device)
    for half in range(2):
        n = (codes >> (4 * half)) & 15
        e, f = ((n >> 1) & 3).double(), (n & 1).double()
        mag = torch.where(e > 0, torch.exp2(e - 1.0) * (1.0 + 0.5 * f), 0.5 * f)
        nib[..., half] = torch.where(n > 7, -mag, mag)
    scale = torch.exp2(scales.double() - 127.0).repeat_interleave(32, dim=-1)
    return nib.flatten(-2) * scale


def _swiglu64(x, w13, s13, w2, s2):
    h = _value64(w13, s13) @ x
    gate, up = h.chunk(2)
    return _value64(w2, s2) @ (gate * torch.sigmoid(gate) * up)


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    if case["op"] == "linear":
        y = torch.cat([s.x.double() @ _value64(a, b).T for a, b in zip(s.codes.split(4096), s.scales.split(4096))], 1)
        return y if s.bias is None else y + s.bias.double()
    outs, ids, wts = [], [], []
    for t in range(case["M"]):
        x0 = s.x[t].double()
        x = x0
        if case["norm"]:
            x = x0 / torch.sqrt(x0.square().sum() / x0.numel() + s.eps) * s.norm_w.double()
        sig = 1.0 / (1.0 + torch.exp(-(s.router_w.double() @ x)))
        rank = sig if s.bias is None else sig + s.bias.double()
        rank = rank.tolist()
        sel = sorted(range(case["E"]), key=lambda e: (-rank[e], e))[:case["topk"]]
        w = sig[torch.tensor(sel, device=sig.device)]
        w = w / w.sum() * case["scale"]
        y = x0 if case["residual"] else torch.zeros_like(x0)
        for e, we in zip(sel, w):
            y = y + we * _swiglu64(x, s.w13[e], s.s13[e], s.w2[e], s.s2[e])
        if case["shared"]:
            y = y + _swiglu64(x, s.sw13[0], s.ss13[0], s.sw2[0], s.ss2[0])
        outs.append(y)
        ids.append(torch.tensor(sel, device=sig.device, dtype=torch.int32))
        wts.append(w)
    return torch.stack(outs), torch.stack(ids), torch.stack(wts)
