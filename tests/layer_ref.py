"""Plain fp64 references of the operators that run a calibrated layer, and their error bounds.

Independent of the CUDA path: E2M1 and E4M3 values are written out from their formats. Bounds are
worst-case ones: a term's products are exact, and a sum of depth d in fp32, each step of which may
truncate (2^-23), is off by at most d 2^-23 of the sum of magnitudes.
"""
import math

import numpy as np
import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def e4m3_table():
    """fp64 values of the E4M3 codes 0..127 (127 is NaN)."""
    v = [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)]
    v[127] = math.nan
    return torch.tensor(v, dtype=torch.float64)


def nibbles(packed):
    """[..., C/2] bytes -> [..., C] nibbles, the low one first."""
    p = packed.cpu()
    return torch.stack((p & 15, p >> 4), -1).flatten(-2).long()


def weight_values(packed, codes):
    """q * v_c of packed weights, exact in fp64, [..., C]."""
    n = nibbles(packed)
    q = torch.tensor(E2M1, dtype=torch.float64)[n & 7] * (1 - 2 * (n >> 3)).double()
    return q * e4m3_table()[codes.cpu().long()].repeat_interleave(16, -1)


def block_scale(codes, g):
    """s = fp32(v_c * g) as fp64, codes above 126 as 126."""
    v = e4m3_table()[codes.cpu().long().clamp(max=126)].numpy().astype(np.float32)
    g = g.cpu().numpy().astype(np.float32).reshape((-1,) + (1,) * (v.ndim - 1))
    return torch.from_numpy((v * g).astype(np.float64))


def pack(w, codes, g):
    """Nibbles of w [G, R, C]: sign and the E2M1 code of |w| / s, nearest, ties to the even code.
    The comparison |w| against midpoint * s is exact in fp64 (24 + 24 + 3 bits at most)."""
    a = w.cpu().double().abs()
    s = block_scale(codes, g).repeat_interleave(16, -1)
    j = torch.zeros(a.shape, dtype=torch.long)
    for k in range(1, 8):
        mid = 0.5 * (E2M1[k - 1] + E2M1[k]) * s
        j += ((a > mid) | ((a == mid) & (k % 2 == 0))).long() * (s > 0)
    return j | (torch.signbit(w.cpu()).long() << 3)


def x_values(x, x_scale=None, scale_block=0):
    x = x.cpu()
    if x_scale is None:
        return x.double()
    v = x.float().double()
    s = x_scale.cpu().double()
    return v * (s if scale_block == 0 else s.repeat_interleave(scale_block, 1)[:, :x.shape[1]])


def matvec(x, packed, codes, g, experts=None):
    """(y, bound of the fp32 sums) in fp64; x in fp64 [n, C]; rows of empty slots are NaN."""
    groups, rows, cin = packed.shape[0], packed.shape[1], 2 * packed.shape[2]
    n = x.shape[0]
    ids = [0] * n if experts is None else experts.cpu().tolist()
    y = torch.full((len(ids), rows), math.nan, dtype=torch.float64)
    tol = torch.zeros_like(y)
    depth = cin / 16 + 32  # products of one k-step and the chain over k-steps, splits joined
    blocks = torch.nn.functional.pad(x.abs(), (0, -cin % 128)).view(n, -1, 128)
    top = blocks.amax(-1).repeat_interleave(128, 1)[:, :cin]
    known = {}
    for i, e in enumerate(ids):
        if not 0 <= e < groups:
            continue
        if e not in known:
            known[e] = weight_values(packed[e], codes[e])
        w, row = known[e], x[i // (len(ids) // n)]
        ge = float(g[e])
        y[i] = (w @ row) * ge
        # fp32 sums, and activations rounded below 2^-39 of the largest of their 128 channels.
        tol[i] = abs(ge) * (depth * 2.0 ** -23 * (w.abs() @ row.abs()) + 2.0 ** -39 * (w.abs() @ top[i // (len(ids) // n)]))
    return y, tol


def check_matvec(y, ref, tol):
    used = ~torch.isnan(ref)
    d = (y.cpu().double() - ref).abs()
    lim = tol + HALF_STEP[y.dtype] * (ref.abs() + tol) + 1e-300
    bad = used & ~(d <= lim)
    assert not bad.any(), f"{int(bad.sum())} of {int(used.sum())} off, worst {float((d / lim)[used].max())} of the bound"


def rmsnorm(x, weight=None, eps=1e-6, residual=None):
    """(r rounded to x's type, v in fp64)."""
    r = x.cpu()
    if residual is not None:
        r = (r.float() + residual.cpu().float()).to(x.dtype)
    v = r.double()
    v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + float(np.float32(eps)))
    return r, v if weight is None else v * weight.cpu().double()


def rmsnorm_rel(cin):
    """Relative bound of v in fp32: half the sum of squares' (a thread's chain, two shuffle trees, the
    mean and eps), the root, the quotient and two products."""
    return (max(cin / 1024, 32) + 12) * 2.0 ** -25 + 4 * 2.0 ** -24


def scale_blocks(cin, scale_block):
    return 1 if scale_block == 0 else -(-cin // scale_block)


def check_y8(y8, scale, v, scale_block, rel):
    """E4M3 values and scales against v (fp64): each scale within rel of max|v| / 448, each value
    within half an E4M3 step of v over the stored scale."""
    n, cin = v.shape
    blk = cin if scale_block == 0 else scale_block
    nb = scale_blocks(cin, scale_block)
    q, s = y8.cpu().float().double(), scale.cpu().double().view(n, nb)
    want = torch.nn.functional.pad(v, (0, nb * blk - cin)).view(n, nb, blk).abs().amax(-1) / 448.0
    assert ((s - want).abs() <= (rel + 2.0 ** -23) * want + 2.0 ** -149).all()
    se = s.repeat_interleave(blk, 1)[:, :cin]
    u = torch.where(se > 0, v / se.clamp(min=1e-300), torch.zeros_like(v))
    e = torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6)))
    half = torch.exp2(e - 4)  # half a step of 3 mantissa bits, or of the subnormals
    assert ((q - u).abs() <= half + u.abs() * (rel + 2.0 ** -22)).all()
    assert (q[se == 0] == 0).all()


def e4m3_of_quotient(v, scale_block):
    """E4M3 of 448 v / max|v| per row or 128 channels: nearest, ties to even, in fp64."""
    n, cin = v.shape
    blk = cin if scale_block == 0 else scale_block
    nb = scale_blocks(cin, scale_block)
    u = torch.nn.functional.pad(v, (0, nb * blk - cin)).view(n, nb, blk)
    m = u.abs().amax(-1, keepdim=True)
    u = torch.where(m > 0, 448.0 * u / m.clamp(min=1e-300), torch.zeros_like(u)).view(n, -1)[:, :cin]
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(u / step) * step
