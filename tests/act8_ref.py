"""The 8-bit activation format from its definition, in binary64."""
import torch

BLOCK = 32


def code_values():
    """What the 256 codes stand for."""
    v = []
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = float("nan") if c & 127 == 127 else (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
        v.append(-x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64)


def _blocks(x):
    n = (x.shape[1] + BLOCK - 1) // BLOCK
    full = x.new_zeros(x.shape[0], n * BLOCK)
    full[:, :x.shape[1]] = x
    return full.view(x.shape[0], n, BLOCK)


def scale_bytes(x):
    """The least e >= -127 with max |x| <= 448 * 2^e over each block's finite
    elements, + 127."""
    b = _blocks(x.double().cpu())
    top = torch.where(torch.isfinite(b), b.abs(), 0.0).amax(2)
    byte = torch.zeros(top.shape, dtype=torch.int64)
    for e in range(-127, 121):
        byte += (top > 448.0 * 2.0 ** e).long()
    return byte


def pack_values(x):
    """(scale bytes, the values that the codes stand for)."""
    byte = scale_bytes(x)
    b = _blocks(x.double().cpu())
    y = b * torch.exp2(127.0 - byte)[..., None]
    y = torch.where(torch.isfinite(y), y, float("nan"))
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    q = torch.round(y / step) * step
    return byte, (q * torch.exp2(byte - 127.0)[..., None]).flatten(1)[:, :x.shape[1]]


def unpack_values(codes, scales):
    v = _blocks(code_values()[codes.cpu().long()])
    s = scales.cpu().double()
    s = torch.where(s == 255, float("nan"), torch.exp2(s - 127.0))
    return (v * s[..., None]).flatten(1)[:, :codes.shape[1]]
