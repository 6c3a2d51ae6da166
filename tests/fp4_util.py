"""Microscaled 4-bit floating point in fp64, by comparison with every representable value, and the
layout of the scales. The values, scales and borders between roundings are all exact in fp64."""
import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E4M3 = torch.tensor([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119],
                    dtype=torch.float64)  # every one without a sign, up to 448


def nearest(v, table):
    """Index of the entry of `table` (ascending) nearest to v >= 0, of two as near the even one, of values beyond
    the last the last."""
    mid = (table[:-1] + table[1:]) / 2
    up = torch.bucketize(v, mid, right=True)   # entries whose middle is at most v
    low = torch.bucketize(v, mid, right=False)
    return torch.where(up == low, up, low + low % 2)


def tensor_scale64(x):
    """The smallest power of two with max |x| <= 2688 ts, over the finite x, not below 2^-90."""
    x = x.double()
    top = float(torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).max()) if x.numel() else 0.0
    ts = 2.0 ** -90
    while top > 2688.0 * ts:
        ts *= 2.0
    return ts


def quantize64(x, fmt, ts=None):
    """(codes, scales as bytes, values): codes 0..15 of x's shape, scale bytes a block, values in fp64."""
    x = x.double()
    n = 16 if fmt == "nvfp4" else 32
    v = x.reshape(*x.shape[:-1], -1, n)
    amax = v.abs().amax(-1)
    bad = ~torch.isfinite(v).all(-1)
    amax = torch.where(bad, torch.zeros_like(amax), amax)
    if fmt == "nvfp4":
        byte = nearest(amax / 6.0 / ts, E4M3)
        step = E4M3[byte] * ts
        byte = torch.where(bad, 0x7F, byte)
    else:
        e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)
        e = torch.where(amax == 0, -127, e)
        byte, step = e + 127, torch.exp2(e.double())
        byte = torch.where(bad, 0xFF, byte)
    d = step[..., None]
    q = torch.where(d > 0, v.abs() / torch.where(d > 0, d, torch.ones_like(d)), torch.zeros_like(v))
    code = nearest(torch.where(bad[..., None], torch.zeros_like(q), q), E2M1)
    values = torch.copysign(E2M1[code], v) * d
    values = torch.where(bad[..., None], torch.full_like(values, float("nan")), values)
    return code.reshape(x.shape), byte, values.reshape(x.shape)


def scale_bytes_of(q):
    """The scale bytes of an Fp4Tensor a block, [rows, blocks], and whether all the padding is zero."""
    K = q.shape[-1]
    rows, blocks = q.codes.numel() // (K // 2), K // (32 if q.format else 16)
    R, J = (rows + 127) // 128, (blocks + 3) // 4
    t = q.scales.cpu().view(R, J, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R * 128, J * 4)
    pad = t.clone()
    pad[:rows, :blocks] = 0
    return t[:rows, :blocks].long(), bool((pad == 0).all())


def codes_of(q):
    c = q.codes.cpu().long()
    return torch.stack((c & 15, c >> 4), -1).reshape(*q.shape)


def exact_operand(seed, rows, K, fmt):
    """bf16 values that 4 bits hold exactly: quarters of small whole numbers in each block, one of them the largest, so
    that the block's scale is a power of two, another one from block to block."""
    g = torch.Generator().manual_seed(seed)
    n = 16 if fmt == "nvfp4" else 32
    codes = E2M1[torch.randint(0, 8, (rows, K // n, n), generator=g)]
    codes = codes * (torch.randint(0, 2, codes.shape, generator=g) * 2 - 1)
    at = torch.randint(0, n, (rows, K // n, 1), generator=g)
    codes.scatter_(-1, at, torch.where(torch.rand(at.shape, generator=g) < 0.5, 6.0, -6.0).double())
    up = torch.exp2(torch.randint(0, 3, (rows, K // n, 1), generator=g).double())
    return (codes * up).reshape(rows, K).to(torch.bfloat16)
