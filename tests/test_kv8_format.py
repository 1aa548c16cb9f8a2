"""The float64 form of the 8-bit rows that the tests of the append stand on, pinned to the element format itself (no GPU)."""
import math

import torch

from kv8_util import E4M3, exponent8, grid8, held64, quantise64

# magnitudes of the codes 0 .. 126, from the format: 4 bits of exponent, bias 7, 3 stored bits; 127 is NaN
CODES = torch.tensor([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127],
                     dtype=torch.float64)


def _nearest(x):
    """By comparison with every code: the nearest value, of two as near the one whose code is even; 448 at most."""
    d = (x.abs()[:, None] - CODES).abs()
    best = d.amin(1, keepdim=True)
    two = (d == best).sum(1) == 2
    lower = (d == best).to(torch.int64).argmax(1)
    code = torch.where(two, lower + lower % 2, lower)
    return torch.where(x < 0, -CODES[code], CODES[code])


def test_the_grid_is_the_type_s_rounding_exactly():
    assert torch.equal(torch.arange(127, dtype=torch.uint8).view(E4M3).double(), CODES)
    middle = (CODES[1:] + CODES[:-1]) / 2
    x = torch.cat([CODES, middle, *(y * (1 + s * 2.0 ** -t) for y in (CODES, middle) for s in (-1, 1) for t in (50, 23, 10)),
                   torch.tensor([2.0 ** -10, 2.0 ** -11, 2.0 ** -40, 449.0, 464.0, 1e9], dtype=torch.float64)])
    x = torch.cat([x, -x])
    assert torch.equal(grid8(x), _nearest(x))
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(20_000, dtype=torch.float64, generator=g) * torch.exp2(torch.randint(-14, 9, (20_000,), generator=g).double()))
    assert torch.equal(grid8(x), _nearest(x))
    x = x.float().clamp(-448, 448)                                    # of float32 the type itself rounds so
    assert torch.equal(grid8(x.double()), x.to(E4M3).double())


def test_rows_have_the_least_scale_and_are_off_by_half_a_step_of_it():
    g = torch.Generator().manual_seed(2)
    for dt, low, high in ((torch.bfloat16, -64, 63), (torch.float16, -15, 7)):
        x = torch.randn((400, 64), dtype=torch.float64, generator=g) * torch.exp2(torch.arange(400).double() / 400 * 90 - 45)[:, None]
        if dt == torch.float16:
            x = x.clamp(-65504, 65504)
        k = exponent8(x.abs().amax(-1), dt)
        for row, e in zip(x.abs().amax(-1).tolist(), k.tolist()):
            assert e == min(high, max(low, math.ceil(math.log2(row / 448.0) - 1e-15)))
        code, scale = quantise64(x, dt)
        assert torch.equal(code, code.float().to(E4M3).double()) and torch.equal(scale.to(torch.int64) - 127, k)
        y, unit = held64(code, scale), torch.exp2(k.double())[:, None]
        whole = x.abs() <= 448 * unit
        assert bool(((y - x).abs() <= torch.maximum(x.abs() * 2.0 ** -4, unit * 2.0 ** -10))[whole].all())
        assert bool((y.abs() == 448 * unit)[~whole].all())
