"""Plain 64-bit forms of the norm and of the products with an epilogue, for the tests."""
import math

import torch

BF16 = torch.bfloat16
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
# |act'| is at most this (the maxima are 1.1290 for both gelus and 1.0999 for silu)
LIPSCHITZ = 1.13
# the activations' own error, as include/nvfp4.h states it: times max(|v|, 1)
ACT_ERROR = 5e-7


def norm_rows(x, residual, weight, eps):
    """(h, n) as bf16: h = bf16(x + r), n = bf16(fp32(fp32(h * rstd) * w)), rstd the fp32
    rounding of the 64-bit 1 / sqrt(mean(h^2) + eps)."""
    h = x if residual is None else (x.float() + residual.float()).to(BF16)
    hd = h.double()
    rstd = (1.0 / torch.sqrt(hd.square().mean(-1, keepdim=True) + eps)).float()
    n = h.float() * rstd
    if weight is not None:
        n = n * weight.float()
    return h, n.to(BF16)


def norm_rows_64(h, weight, eps):
    hd = h.double()
    n = hd * torch.rsqrt(hd.square().mean(-1, keepdim=True) + eps)
    return n if weight is None else n * weight.double()


def act64(v, act):
    if act == "relu":
        return v.clamp(min=0.0)
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v * math.sqrt(0.5))
    if act == "gelu_tanh":
        return v * torch.sigmoid(math.sqrt(8.0 / math.pi) * (v + 0.044715 * v ** 3))
    if act == "silu":
        return v * torch.sigmoid(v)
    return v


def epilogue_64(v, dv, act, gated, residual):
    """(y, bound): the epilogue on the 64-bit v, and how far the kernel's bf16 may be from y
    when its fp32 v is within dv of it.

    An activation moves by at most LIPSCHITZ * dv and adds its own error; a product of a and
    b moves by |a| db + |b| da + da db and one rounding; the residual's addition is one
    rounding more (2^-24 relative each); the last one to bf16 is half a step, 2^-8 |y| (and
    half the smallest subnormal, 2^-134)."""
    if gated:
        g, u = v[:, 0::2], v[:, 1::2]
        dg, du = dv[:, 0::2], dv[:, 1::2]
    else:
        g, dg = v, dv
    a = act64(g, act)
    da = dg if act == "none" else LIPSCHITZ * dg + ACT_ERROR * g.abs().clamp(min=1.0)
    if gated:
        y = a * u
        d = a.abs() * du + u.abs() * da + da * du
        d = d + 2.0 ** -24 * (y.abs() + d)
    else:
        y, d = a, da
    if residual is not None:
        y = y + residual.double()
        d = d + 2.0 ** -24 * (y.abs() + d)
    return y, d + 2.0 ** -8 * (y.abs() + d) + 2.0 ** -134


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def dequant64(packed, sf, rows, K):
    """float64 E2M1 * E4M3 of a packed operand with 128x4 scales."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=packed.device)
    v = torch.stack((table[(packed & 15).long()], table[(packed >> 4).long()]), -1)
    rt, kc = -(-rows // 128), -(-K // 64)
    s = sf.view(torch.float8_e4m3fn).double().view(rt, kc, 32, 4, 4).permute(0, 3, 2, 1, 4)
    s = s.reshape(rt * 128, kc * 4)[:rows, :K // 16]
    return (v.view(rows, K // 16, 16) * s.unsqueeze(-1)).view(rows, K)


def fp4_product_64(a, sfa, b, sfb, alpha, bias, M, N, K):
    """(v, dv): alpha * A B^T + bias in 64 bits, and the fp32 kernel's distance from it.

    The products of dequantized values are exact; the tensor cores add the 64 of a K step
    into an fp32 accumulator, and the split-K builds at most 8 partial sums: K / 64 + 8
    additions, each off by at most 2^-23 (rounded or cut) of a partial sum, which is at most
    S = sum |a b|.  alpha and the bias add two roundings of 2^-24."""
    A, B = dequant64(a, sfa, M, K), dequant64(b, sfb, N, K)
    al = float(alpha)
    v = (A @ B.T) * al
    dv = (A.abs() @ B.abs().T) * abs(al) * ((K / 64 + 8) * 2.0 ** -23) + 2.0 ** -24 * v.abs()
    if bias is not None:
        v = v + bias.double()
        dv = dv + 2.0 ** -24 * (v.abs() + dv)
    return v, dv


def int8_product_64(a, sa, b, sb, bias):
    """(v, dv) of the int8 product: the integer sum is exact; its conversion to fp32, the two
    scales and the bias are four roundings of 2^-24."""
    v = (a.double() @ b.double().T) * sa.double().unsqueeze(-1) * sb.double()
    dv = 3 * 2.0 ** -24 * v.abs() * (1 + 2.0 ** -20)
    if bias is not None:
        v = v + bias.double()
        dv = dv + 2.0 ** -24 * (v.abs() + dv)
    return v, dv


def check(y, y64, bound, what):
    assert y.dtype == BF16 and y.shape == y64.shape, what
    assert torch.isfinite(y).all(), f"{what}: not finite"
    excess = (y.double() - y64).abs() - bound
    worst = float(excess.max())
    assert worst <= 0, f"{what}: {int((excess > 0).sum())} values, worst by {worst:.3e} over the bound"
