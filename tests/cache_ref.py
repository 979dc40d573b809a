"""64-bit references of the operators that fill a KV cache and of decode
attention over a cache held in 8 bits, and the error bounds the tests hold
the kernels to.  Nothing here uses the package's arithmetic.

Bounds (each step's worst case, relative to the terms it acts on):

* bf16 output: half a step, 2^-8 of the value (eps / 2 with eps = 2^-7).
* norm in fp32: the sum of n squares errs by at most n 2^-24 of itself, the
  root, the reciprocal and the two products by a few 2^-24 more:
  (n / 2 + 8) 2^-24 relative.
* cos and sin: the phase's rounding moves the angle by at most 2^-25 pi <
  2^-23; the functions themselves are allowed 2^-21 absolute.  Each of the two
  products and their sum rounds once more: 3 * 2^-24.  In all 2^-20 of |a| +
  |b| times mscale, the norm's error apart.
* e4m3 code: half a step, 2^-4 of the value or 2^-10 below 2^-6, plus the
  fp32 error of what is rounded.
"""
import math

import torch

BF16_HALF = 2.0 ** -8
E4M3_MAX = 448.0


def turns_to_radians(turns):
    """Radians per position of turns int64 (a fraction of a turn in units of 2^-64)."""
    return [(int(t) % (1 << 64)) / 2.0 ** 64 * 2 * math.pi for t in turns.tolist()]


def angles64(turns, positions):
    """[rows, half] angles modulo a turn, exact integers first."""
    rows = []
    for p in positions.tolist():
        rows.append([((int(t) * int(p)) % (1 << 64)) / 2.0 ** 64 * 2 * math.pi
                     for t in turns.tolist()])
    return torch.tensor(rows, dtype=torch.float64).reshape(len(rows), -1)


def head_rows(x, turns, positions, *, norm=None, eps=1e-6, start=0, interleaved=False, mscale=1.0):
    """(exact, error bound of the fp32 result) of norm and rotation; x [rows, heads, dim] bf16 on
    the CPU, turns int64 or None."""
    y = x.double().clone()
    err = torch.zeros_like(y)
    if norm is not None:
        n = norm.numel()
        inv = 1.0 / torch.sqrt(y[..., :n].pow(2).mean(-1, keepdim=True) + eps)
        y[..., :n] = y[..., :n] * inv * norm.double()
        err[..., :n] = (n / 2 + 8) * 2.0 ** -24 * y[..., :n].abs()
    if turns is not None:
        half = turns.numel()
        i = torch.arange(half)
        a = start + (2 * i if interleaved else i)
        b = a + (1 if interleaved else half)
        phi = angles64(turns, positions)[:, None]
        c, s = phi.cos() * mscale, phi.sin() * mscale
        ya, yb, ea, eb = y[..., a], y[..., b], err[..., a], err[..., b]
        size = (ya.abs() + yb.abs()) * abs(mscale)
        y[..., a] = ya * c - yb * s
        y[..., b] = yb * c + ya * s
        e = (ea + eb) * abs(mscale) + size * 2.0 ** -20
        err[..., a] = e
        err[..., b] = e
    return y, err


def assert_bf16(got, exact, err, what):
    g = got.detach().cpu().double()
    bound = BF16_HALF * (exact.abs() + err) + err + 2.0 ** -134   # half the least bf16 number
    worst = ((g - exact).abs() - bound).max().item() if g.numel() else -1.0
    assert torch.isfinite(g).all() and worst <= 0, f"{what}: {worst:.3g} above the bound"


def scale_exponents(amax):
    """Least e with amax <= 448 * 2^e, clamped to [-60, 120]; -60 where amax is 0."""
    e = torch.ceil(torch.log2(amax.clamp_min(2.0 ** -400) / E4M3_MAX))
    e = torch.where(amax > E4M3_MAX * torch.exp2(e), e + 1, e)          # a log2 rounded down
    e = torch.where(amax <= E4M3_MAX * torch.exp2(e - 1), e - 1, e)     # or up
    return e.clamp(-60, 120)


def half_step(x):
    """Half the distance between e4m3 numbers around |x| <= 448."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -40))).clamp_min(-6)
    return torch.exp2(e - 4)


def decode_reference(q, k, v, kv_len, *, group, scale, offsets=None, causal=False, sink=None):
    """fp64 attention of q [rows, hq, d] on per-sequence lists k[b], v[b] of [L, hkv, d] fp64.
    Returns out, lse, the weighted spread sqrt(sum w (v - out)^2), sum w |v| and the largest
    sum_c |q_c k_c| * scale of a row's keys."""
    rows, hq, d = q.shape
    out = torch.zeros(rows, hq, d, dtype=torch.float64)
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64)
    mass, big = torch.zeros_like(out), torch.zeros(rows, hq, dtype=torch.float64)
    for b in range(len(kv_len)):
        r0, r1 = (b, b + 1) if offsets is None else (offsets[b], offsets[b + 1])
        L = kv_len[b]
        for r in range(r0, r1):
            lim = min(L, L - (r1 - r0) + (r - r0) + 1) if causal else L
            for h in range(hq):
                g = h // group
                K, V = k[b][:max(lim, 0), g], v[b][:max(lim, 0), g]
                t = -math.inf if sink is None else float(sink[h])
                x = q[r, h].double()
                s = (K @ x) * scale
                m = max(s.max().item() if len(s) else -math.inf, t)
                if m == -math.inf:
                    continue
                w = torch.exp(s - m)
                z = w.sum() + math.exp(t - m)
                out[r, h] = (w @ V) / z
                lse[r, h] = m + torch.log(z)
                mass[r, h] = (w @ V.abs()) / z
                if len(s):
                    big[r, h] = ((K.abs() @ x.abs()) * abs(scale)).max()
    return out, lse, mass, big
