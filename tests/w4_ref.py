"""Plain 64-bit forms of the few-token operators, and the inputs of their tests."""
import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def value64(codes, scales):
    """fp64 values of MXFP4: element 2i in bits 3:0 of byte i; one E8M0 scale for 32."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=codes.device)
    idx = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).long()
    return table[idx] * torch.exp2(scales.double() - 127.0).repeat_interleave(32, dim=-1)


def rand_mx(gen, *shape, lo=117, hi=123):
    """Random codes (every code) and scales 2^(lo-127) .. 2^(hi-128)."""
    dev = gen.device
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=gen, device=dev, dtype=torch.uint8)
    scales = torch.randint(lo, hi, (*shape[:-1], shape[-1] // 32), generator=gen, device=dev, dtype=torch.uint8)
    return codes, scales


def split_error(x, w_abs):
    """Bound on what the two-column form of x may lose in x W^T: 2^-21 of its
    block's largest value for every element, times |w|.  The scale exponent s is at
    least -112 and values below 2^-14 2^s become zero, so where the block's largest
    value is itself tiny the loss is up to 2^-14 2^-112 = 2^-126: subnormal
    activations count as zero."""
    M, K = x.shape
    amax = x.double().abs().reshape(M, K // 32, 32).amax(-1).repeat_interleave(32, -1)
    return (amax * 2.0 ** -21 + 2.0 ** -126) @ w_abs.T


def linear_ref(x, w, bias=None):
    """(x W^T + bias in 64 bits, bound on an fp32 result's error): the split's loss,
    and K + 8 fp32 additions, each off by at most 2^-23 of sum |x w| (a full step:
    no rounding mode is assumed of the tensor cores), and the bias's addition."""
    x = x.double()
    y = x @ w.T
    tol = split_error(x, w.abs()) + (x.shape[1] + 8) * 2.0 ** -23 * (x.abs() @ w.abs().T)
    if bias is not None:
        y = y + bias.double()
        tol = tol + 2.0 ** -24 * y.abs()
    return y, tol


def swiglu_ref(x, xerr, w13, w2):
    """One expert in 64 bits on x [M][H] known to within xerr: (y, bound on an
    implementation that holds x and mid as two operand columns)."""
    I = w13.shape[0] // 2
    K1, K2 = w13.shape[1], I
    gu = x @ w13.T
    # x held to 2^-9 of each value (the columns' loss for an fp32 value), K1 + 8 fp32 additions of full steps
    e = (xerr + 2.0 ** -9 * x.abs()) @ w13.abs().T + (K1 + 8) * 2.0 ** -23 * (x.abs() @ w13.abs().T)
    g, u, eg, eu = gu[:, :I], gu[:, I:], e[:, :I], e[:, I:]
    silu = g * torch.sigmoid(g)
    mid = silu * u
    # |silu'| < 1.1; the products' and the exponential's own roundings: 2^-18 of mid
    em = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + 2.0 ** -18 * mid.abs()
    # mid is rounded to 11 bits (2^-12) and held to 2^-9; a block's small values to 2^-21 of its largest
    blk = (mid.abs() + em).reshape(mid.shape[0], I // 32, 32).amax(-1).repeat_interleave(32, -1)
    em = em + (2.0 ** -9 + 2.0 ** -12) * (mid.abs() + em) + 2.0 ** -21 * blk + 2.0 ** -126
    y = mid @ w2.T
    ey = em @ w2.abs().T + (K2 + 8) * 2.0 ** -23 * ((mid.abs() + em) @ w2.abs().T)
    return y, ey


def layer_ref(x, norm_w, eps, router_w, bias, topk, scale, experts, shared, residual, ids=None):
    """The whole layer in 64 bits.  experts(e) -> (w13, w2) values; shared the
    same or None.  ids: selection to use (else the 64-bit one).  Returns out,
    bound (without bf16's rounding), ids, weights, and each token's margin
    between the last chosen and the first not chosen score."""
    x0 = x.double()
    h = x0
    if norm_w is not None:
        h = x0 / torch.sqrt((x0 * x0).mean(-1, keepdim=True) + eps) * norm_w.double()
    # 1 / rms in fp32: the sum of squares, division, root and factor, each few roundings
    herr = 2.0 ** -20 * h.abs() if norm_w is not None else torch.zeros_like(h)
    s = torch.sigmoid(h @ router_w.double().T)
    score = s if bias is None else s + bias.double()
    order = torch.sort(score, dim=-1, descending=True, stable=True)
    E = s.shape[1]
    margin = order.values[:, topk - 1] - order.values[:, topk] if topk < E else torch.full((len(x),), 1.0, device=x.device)
    if topk > 1:   # the order within the selection is part of the result
        inner = (order.values[:, :topk - 1] - order.values[:, 1:topk]).amin(-1)
        margin = torch.minimum(margin, inner)
    if ids is None:
        ids = order.indices[:, :topk]
    w = torch.gather(s, 1, ids.long())
    w = w / w.sum(-1, keepdim=True) * scale
    out, err = torch.zeros_like(h), torch.zeros_like(h)
    for e in sorted(set(ids.flatten().tolist())):
        t, j = (ids == e).nonzero(as_tuple=True)
        y, ey = swiglu_ref(h[t], herr[t], *experts(e))
        out[t] += w[t, j, None] * y
        err[t] += w[t, j, None] * (ey + 2.0 ** -16 * y.abs())   # the weight itself: a handful of fp32 roundings
    if shared is not None:
        y, ey = swiglu_ref(h, herr, *shared)
        out, err = out + y, err + ey
    if residual:
        out = out + x0
    return out, err + 2.0 ** -20 * out.abs(), ids, w, margin
