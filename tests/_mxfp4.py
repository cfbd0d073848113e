"""A plain 64-bit MXFP4 quantiser and decoder for the tests (CPU or GPU tensors), written from the OCP
definition: nearest of the eight E2M1 magnitudes by distance, ties to the even code."""
import torch

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def power_of_two(e):
    """2^e in float64, from its bits (torch.ldexp goes through an inexact pow on the GPU)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def quantize(x):
    """x [..., K] -> (codes uint8 [..., K], one per byte, scale bytes uint8 [..., K/32], values float64)."""
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)
    b = x.double().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    e = torch.frexp(torch.where(bad | (amax == 0), torch.full_like(amax, 2.0 ** -140), amax)).exponent - 1 - 2
    e = e.clamp(min=-127)
    scale = power_of_two(e).unsqueeze(-1)
    v = torch.where(bad.unsqueeze(-1), 0.0, b) / scale
    dist = (v.abs().clamp(max=6.0).unsqueeze(-1) - grid).abs()
    near = dist == dist.amin(-1, keepdim=True)
    odd = torch.arange(8, device=x.device) % 2
    code = (near.double() * (2 - odd)).argmax(-1)      # of two at the same distance, the even one
    codes = (code + 8 * torch.signbit(b).long()).to(torch.uint8)
    codes = torch.where(bad.unsqueeze(-1), torch.zeros_like(codes), codes)
    values = torch.where(torch.signbit(b), -grid[code], grid[code]) * scale
    values = torch.where(bad.unsqueeze(-1), float("nan"), values)
    s = torch.where(bad, 255, e + 127).to(torch.uint8)
    return codes.flatten(-2), s, values.flatten(-2)


def pack(codes):
    return codes[..., 0::2] + 16 * codes[..., 1::2]


def decode(packed, s):
    """Packed codes [..., K/2] and scale bytes [..., K/32] -> float64 [..., K]."""
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=packed.device)
    c = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).long()
    v = torch.where(c >= 8, -grid[c & 7], grid[c & 7]).unflatten(-1, (-1, 32))
    scale = torch.where(s == 255, float("nan"), power_of_two(s.int() - 127))
    return (v * scale.unsqueeze(-1)).flatten(-2)


def tile_scales(s):
    """[G, N, K/32] -> the weights' atoms [G, ceil(N/128), ceil(K/128), 512], element by element."""
    g, n, kb = s.shape
    nb, ka = -(-n // 128), -(-kb // 4)
    out = torch.zeros((g, nb, ka, 512), dtype=torch.uint8, device=s.device)
    col = torch.arange(n, device=s.device).unsqueeze(1)
    b = torch.arange(kb, device=s.device).unsqueeze(0)
    out[:, (col // 128).expand(n, kb), (b // 4).expand(n, kb), 16 * (col % 32) + 4 * (col // 32 % 4) + b % 4] = s
    return out
