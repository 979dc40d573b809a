"""The terms that decode attention over a 4-bit cache holds its weights in: four e5m2 numbers, the
first the nearest, the next two cut off what is left (as f16) in units of 2^-4, the last
the rest rounded in units of 2^-10.  The arithmetic is restated here with torch's conversions;
what is checked is the error that the other tests and the documents name.

w runs to 2^15: 2^11 times a weight of up to 8 (the lazy reference) times the mantissa, below 2,
of its V scale.  A weight as large as the reference is at least 2^11."""
import torch

TOP = 2.0 ** 15
REFERENCE = 2.0 ** 11


def e5m2(x):
    return x.clamp(-57344, 57344).to(torch.float8_e5m2).float()


def cut(x):
    """What the upper byte of an f16 number says."""
    return (x.view(torch.int16) & -256).view(torch.float16)


def held(w):
    first = e5m2(w)
    total = first.double()
    x = ((w - first) * 16).to(torch.float16)
    for _ in range(2):
        term = cut(x)
        total += term.double() / 16
        x = x - term
    x = x * 64
    assert bool((x.abs() <= 57344).all() | x.isnan().any())
    return total + e5m2(x.float()).double() / 1024


def near(k, g):
    """Numbers of [2^k, 2^(k + 1)]."""
    return torch.cat([torch.rand(50000, generator=g) + 1, torch.tensor([1.0, 2.0]),
                      1 + torch.arange(8192) / 8192.0]) * 2.0 ** k


def test_error_of_the_terms():
    g = torch.Generator().manual_seed(0)
    for k in range(-34, 15):
        w = near(k, g)
        err = (held(w) - w.double()).abs()
        assert (err <= torch.maximum(2.0 ** -12 * w.double(),
                                     torch.tensor(2.0 ** -34 * REFERENCE))).all(), k


def test_small_weights():
    g = torch.Generator().manual_seed(1)
    for k in range(-24, 0):          # an eighth, down to 2^-35 of the reference
        w = near(k, g)
        assert ((held(w) - w.double()).abs() <= 2.0 ** -2.8 * w.double()).all(), k
    # what a weight of 2^-28 of the reference loses is less than its rounding to bf16 would be
    w = near(-17, g)
    assert ((held(w) - w.double()).abs() <= 2.0 ** -6 * w.double()).all()
    w = near(-14, g)
    assert ((held(w) - w.double()).abs() <= 2.0 ** -9 * w.double()).all()


def test_no_side_is_favoured():
    g = torch.Generator().manual_seed(2)
    for k in (-10, 0, 14):
        w = near(k, g)
        off = (held(w) - w.double()) / w.double()
        assert abs(off.mean()) < 2.0 ** -15


def test_ends():
    for w in (0.0, 2.0 ** -60, TOP, TOP - 2.0 ** -9, 2.0 ** -24):
        assert abs(held(torch.tensor([w])).item() - w) <= max(2.0 ** -12 * w, 2.0 ** -23)
    assert held(torch.tensor([float("nan")])).isnan().all()
