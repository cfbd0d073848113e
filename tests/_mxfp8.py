"""A plain 64-bit MXFP8 quantiser and decoder for the tests (CPU or GPU tensors): nearest of the E4M3
magnitudes by distance, ties to the even code, with the smallest power-of-two scale that fits the block."""
import torch

from tests._mxfp4 import power_of_two


def magnitudes(device):
    """The values of codes 0 .. 126 (127 is NaN): 2^-9 steps below 2^-6, then eight to an octave."""
    c = torch.arange(127, device=device)
    e, m = c // 8, (c % 8).double()
    return torch.where(e > 0, (8 + m) * power_of_two(e - 10), m * 2.0 ** -9)


def quantize(x):
    """x [..., K] -> (codes uint8 [..., K], scale bytes uint8 [..., K/32], values float64)."""
    grid = magnitudes(x.device)
    b = x.double().unflatten(-1, (-1, 32))
    bad = ~torch.isfinite(b).all(-1)
    amax = torch.where(bad, 0.0, b.abs().amax(-1))
    e = torch.full(amax.shape, -127, dtype=torch.int64, device=x.device)
    for _ in range(256):                       # the smallest exponent that fits
        e += (amax > 448 * power_of_two(e)).long()
    scale = power_of_two(e).unsqueeze(-1)
    v = torch.where(bad.unsqueeze(-1), 0.0, b) / scale
    up = torch.searchsorted(grid, v.abs().contiguous()).clamp(max=126)     # first magnitude >= |v|
    lo = (up - 1).clamp(min=0)
    dlo, dup = v.abs() - grid[lo], grid[up] - v.abs()
    code = torch.where((dlo < dup) | ((dlo == dup) & (lo % 2 == 0)), lo, up)
    codes = (code + 128 * torch.signbit(b).long()).to(torch.uint8)
    codes = torch.where(bad.unsqueeze(-1), torch.zeros_like(codes), codes)
    values = torch.where(torch.signbit(b), -grid[code], grid[code]) * scale
    values = torch.where(bad.unsqueeze(-1), float("nan"), values)
    return codes.flatten(-2), torch.where(bad, 255, e + 127).to(torch.uint8), values.flatten(-2)


def decode(codes, s):
    """codes [..., K] and scale bytes [..., K/32] -> float64 [..., K]."""
    grid = torch.cat((magnitudes(codes.device), torch.full((1,), float("nan"), dtype=torch.float64, device=codes.device)))
    c = codes.long()
    v = torch.where(c >= 128, -grid[c & 127], grid[c & 127]).unflatten(-1, (-1, 32))
    scale = torch.where(s == 255, float("nan"), power_of_two(s.int() - 127))
    return (v * scale.unsqueeze(-1)).flatten(-2)
