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
