"""The terms that decode attention over an 8-bit cache holds its weights in: four e4m3
numbers 1, 2^5, 2^10 and 2^25 apart, each the rest of those before rounded to
nearest (saturating).  The arithmetic is restated here with torch's conversions;
what is checked is the error that the other tests and the documents name.

w runs to 256: 16 times a weight of up to 8 (the lazy reference) times the mantissa,
below 2, of its V scale."""
import torch

RATIOS = (32.0, 32.0, 2.0 ** 15)


def held(w):
    a, unit, total = w.clone(), 1.0, torch.zeros_like(w, dtype=torch.float64)
    for ratio in RATIOS + (None,):
        c = a.clamp(-448, 448).to(torch.float8_e4m3fn).float()
        total += c.double() / unit
        if ratio:
            a = (a - c) * ratio
            unit *= ratio
    return total


def test_error_of_the_terms():
    g = torch.Generator().manual_seed(0)
    for k in range(-46, 8):
        w = torch.cat([torch.rand(20000, generator=g) + 1, torch.tensor([1.0, 2.0]),
                       1 + torch.arange(4096) / 4096.0]) * 2.0 ** k
        err = (held(w) - w.double()).abs()
        w = w.double()
        assert (err <= torch.maximum(2.0 ** -13 * w, torch.tensor(2.0 ** -25))).all(), k
        # small ones: a sixteenth of themselves, and nothing at all of what is below 2^-35
        assert (err <= torch.maximum(2.0 ** -4 * w, torch.tensor(2.0 ** -35))).all(), k
    # what a weight of 2^-20 and more loses is less than its rounding to bf16 would be
    w = (torch.rand(20000, generator=g) + 1) * 16 * 2.0 ** -20
    assert ((held(w) - w.double()).abs() <= 2.0 ** -9 * w.double()).all()


def test_sign_and_ends():
    for w in (0.0, 2.0 ** -60, 256.0, 255.99):
        assert abs(held(torch.tensor([w])).item() - w) <= max(2.0 ** -13 * w, 2.0 ** -35)
    assert held(torch.tensor([float("nan")])).isnan().all()
