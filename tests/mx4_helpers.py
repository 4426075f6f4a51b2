"""Microscaled 4-bit floats in plain torch, on any device: the tests' own reading of the formats."""
import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E4M3 = torch.float8_e4m3fn


def codes_of(q):
    """M x K codes of M x K / 2 bytes."""
    return torch.stack((q & 15, q >> 4), 2).flatten(1)


def tile_scales(b, fill=0):
    """M x G scale bytes in tiles of 128 rows x 4 blocks, `fill` where the matrix ends."""
    M, G = b.shape
    tiles = torch.full((-(-M // 128), -(-G // 4), 512), fill, dtype=torch.uint8, device=b.device)
    r, k = torch.arange(M, device=b.device)[:, None], torch.arange(G, device=b.device)[None, :]
    tiles[r // 128, k // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + k % 4] = b
    return tiles


def untile_scales(tiles, M, G):
    r, k = torch.arange(M, device=tiles.device)[:, None], torch.arange(G, device=tiles.device)[None, :]
    return tiles[r // 128, k // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + k % 4]


def scale64(b, block):
    if block == 16:
        return b.view(E4M3).double()
    return torch.where(b == 255, float("nan"), 2.0 ** (b.double() - 127))


def values64(q, b, block, ts=None):
    """What codes and (row by row) scale bytes stand for."""
    c = codes_of(q)
    v = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64, device=q.device)[c.long()]
    v = v * scale64(b, block).repeat_interleave(block, 1)
    return v if ts is None else v * ts.double()


def nearest_code(y):
    """e2m1 code of each y (no NaN): nearest, halves to the even code, the sign in bit 3."""
    a = y.abs().double().clamp(max=6.0)
    table = torch.tensor(E2M1, dtype=torch.float64, device=y.device)
    up = torch.searchsorted(table, a).clamp(max=7)            # first value >= a
    down = (up - 1).clamp(min=0)
    du, dd = table[up] - a, a - table[down]
    take_up = (du < dd) | ((du == dd) & (up % 2 == 0)) | (up == 0)
    return torch.where(take_up, up, down).to(torch.uint8) + 8 * torch.signbit(y).to(torch.uint8)


def quantise(x, block, ts=None):
    """(q, M x G scale bytes): the formulas of tile_mx4_quantize, step by step in fp32."""
    M, K = x.shape
    b = x.float().view(M, K // block, block)
    a = b.abs().amax(2)
    finite = b.isfinite().all(2)
    a = torch.where(finite, a, torch.zeros_like(a))
    if block == 16:
        t = torch.ones((), device=x.device) if ts is None else ts
        s = (a / (6 * t)).clamp(max=448).to(E4M3)
        d = s.float() * t
        byte = s.view(torch.uint8)
        nan = 0x7F
    else:
        e = torch.where(a > 0, torch.frexp(a).exponent - 1 - 2, -127).clamp(min=-127)
        byte = (e + 127).to(torch.uint8)
        d = (2.0 ** e.double()).float()
        nan = 0xFF
    some = (d > 0) & (a > 0) & finite
    y = torch.where(some[:, :, None], b / d[:, :, None], torch.zeros_like(b))
    c = torch.where(some[:, :, None], nearest_code(y), torch.zeros_like(y, dtype=torch.uint8)).view(M, K)
    return c[:, 0::2] | c[:, 1::2] << 4, torch.where(finite, byte, torch.full_like(byte, nan))
