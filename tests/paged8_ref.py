"""Plain forms of the 8-bit paged cache: e4m3 by its definition, rows with a
power-of-two scale, and ragged batches (paged_ref.Batch) in 8-bit pages."""
import math

import torch

import paged_ref

U_E4M3 = 2.0 ** -4                     # half a step, relative; 2^-10 at least (half the subnormal step)


def _two(e):
    """2^e in 64 bits, e an integer tensor within the normal range."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def round_e4m3(x):
    """The nearest number +-m 2^e with m < 16, e >= -9 (ties to an even m), of
    fp64 values up to 448."""
    x = x.double()
    e = (torch.frexp(x).exponent - 4).clamp(min=-9)
    return (x * _two(-e)).round() * _two(e)


def scale_byte(amax):
    """The smallest byte in 10 .. 246 with amax <= 448 * 2^(byte - 127)."""
    m, e = torch.frexp(amax.double())
    return torch.where(amax == 0, 10, (torch.where(m > 0.875, e, e - 1) - 8 + 127).clamp(10, 246))


def quantise(x):
    """fp64 rows [..., d] -> (values of the codes, scale bytes)."""
    byte = scale_byte(x.abs().amax(-1))
    y = (x * _two(127 - byte)[..., None]).clamp(-448, 448)
    return round_e4m3(y), byte


def codes_of(x):
    """e4m3 bytes of exact e4m3 numbers (by a table of all of them)."""
    table = decode(torch.arange(256, dtype=torch.uint8))
    keys = {float(v): i for i, v in enumerate(table.tolist()) if v == v and i != 128}
    flat = [keys[float(v)] for v in x.reshape(-1).tolist()]
    return torch.tensor(flat, dtype=torch.uint8).reshape(x.shape)


def decode(codes):
    """fp64 numbers of e4m3 bytes: sign, 4 bits of exponent (bias 7), 3 of mantissa."""
    c = codes.long()
    sign, e, m = torch.where(c >= 128, -1.0, 1.0).double(), (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * _two(e - 7), m / 8 * 2.0 ** -6)
    return torch.where((c & 127) == 127, math.nan, sign * v)


def values(codes, byte):
    """fp64 rows of codes (uint8 or float8) and scale bytes."""
    return decode(codes.cpu().view(torch.uint8)) * _two(byte.cpu().view(torch.uint8).long() - 127)[..., None]


class Batch8(paged_ref.Batch):
    """A Batch whose pages are 8-bit: k8, v8, ks, vs on the device; k and v hold
    the values they stand for.  Slots past a sequence's end and unused pages hold NaN
    codes under a scale of infinity."""

    def __init__(self, *a, spread=False, **kw):
        super().__init__(*a, **kw)
        for x in "kv":
            rows = getattr(self, x).cpu().double()
            unused = rows[..., 0].isnan()
            rows = torch.nan_to_num(rows)
            if spread:                   # rows of very different sizes, some of them all zeros
                size = torch.randint(-9, 10, rows.shape[:3], generator=self.g)
                rows = rows * _two(size if x == "v" else torch.clamp(size, -9, 1))[..., None]
                rows[size == 9] = 0
            code, byte = quantise(rows)
            c8 = code.float().to(torch.float8_e4m3fn).view(torch.uint8)
            c8[unused], byte[unused] = 0x7f, 255
            setattr(self, x + "8", c8.view(torch.float8_e4m3fn).to(self.device))
            setattr(self, x + "s", byte.to(torch.uint8).view(torch.float8_e8m0fnu).to(self.device))
            v = values(c8, byte.to(torch.uint8))
            setattr(self, x, torch.where(unused[..., None], math.nan, v).to(self.dtype).to(self.device))

    def cache8(self, vc, block_table=None):
        return vc.Paged8Cache(self.k8, self.v8, self.ks, self.vs, self.block_table if block_table is None else block_table,
                              self.dtype)
