"""References in 64 bits for the norm before the exchange and the experts' products, and the
bounds that their tests hold the kernels to.

Bounds.  eps32 = 2^-24 is half a step of float32.  A float32 sum of n products is off by at
most n * 2 * eps32 * sum |products| (one rounding an addition and one a product, whatever
the order; twice that where the matrix units may cut instead of round).  A rounding to the
output type adds half a step: 2^-8 of the value for bfloat16, 2^-24 for float32, 2^-4 for
e4m3 (or half of e4m3's smallest step, 2^-10 of the scale).

8-bit rows meet their weights in the matrix unit's 8-bit form, which adds eight neighbouring
products (elements 8i .. 8i + 7) at a time with the bits down to 2^-13 of the largest one's
power of two and cuts what is below; the sums of eight are then added in float32.  (Seen on
the GPU, products of powers of two: 2^16 - 2^16 + 2^(16-j) in one such eight is 2^(16-j) up to
j = 13 and 0 from j = 14 on; with the third product in another eight it is 2^(16-j) at every j
that e4m3 reaches, 24 and more.)  So each of the other seven products loses less than 2^-13 of
the largest: at most 7 * 2^-13 * max|x| * max|w| for every eight, summed over the row."""
import numpy as np
import torch

from moe_alltoallv_resident_amd import a2av

EPS32 = 2.0 ** -24
HALF_STEP = {a2av.F32: 2.0 ** -24, a2av.BF16: 2.0 ** -8, a2av.MX8: 2.0 ** -4}
TORCH = {a2av.F32: torch.float32, a2av.BF16: torch.bfloat16}
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64)


def scale_value(b):
    """E8M0 bytes in float64."""
    v = torch.exp2(b.to(torch.float64) - 127)
    return torch.where(b == 255, torch.full_like(v, float("nan")), v)


def mx8_values(rows, n):
    """8-bit rows -> (values, element values, scales) in float64 on the CPU."""
    rows = rows.cpu()
    q = E4M3[rows[..., :n].to(torch.int64)]
    s = scale_value(rows[..., n:n + n // 32])
    return q * s.repeat_interleave(32, dim=-1), q, s


def mx4_values(w, scales):
    w = w.cpu()
    v = torch.stack((E2M1[(w & 15).to(torch.int64)], E2M1[(w >> 4).to(torch.int64)]), dim=-1).flatten(-2)
    return v * scale_value(scales.cpu()).repeat_interleave(32, dim=-1)


def values(t, kind, n, scales=None):
    """A tensor of any element type in float64 on the CPU."""
    if kind == a2av.MX8 and scales is None:
        return mx8_values(t, n)[0]
    if kind == a2av.MX8:
        return E4M3[t.cpu().to(torch.int64)] * scale_value(scales.cpu()).repeat_interleave(32, dim=-1)
    if kind == a2av.MX4:
        return mx4_values(t, scales)
    return t.cpu().to(torch.float64)


def encode_mx8(v):
    """float32 [..., n] -> 8-bit rows (uint8), by the definition: the smallest power of two
    that keeps 32 elements within 448."""
    n = v.shape[-1]
    b = v.to(torch.float64).reshape(-1, n // 32, 32)
    a = b.abs().amax(dim=-1)
    e = torch.ceil(torch.log2(torch.where(a > 0, a, torch.ones_like(a)) / 448))
    e = torch.where(a / torch.exp2(e) > 448, e + 1, e)
    e = torch.where(a / torch.exp2(e - 1) <= 448, e - 1, e)
    e = torch.where(a > 0, e, torch.full_like(e, -127)).clamp(min=-127)
    q = (b / torch.exp2(e)[..., None]).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1, n)
    out = torch.zeros((q.shape[0], a2av.a2av_row_bytes(a2av.MX8, n)), dtype=torch.uint8)
    out[:, :n] = q
    out[:, n:n + n // 32] = (e + 127).to(torch.uint8)
    return out.reshape(v.shape[:-1] + (out.shape[-1],))


def assert_close(got, want, err, what):
    """got, want float64 [..]; err the largest difference allowed for each element.  NaN
    has to stand where the reference has it."""
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    bad = ((got - want).abs() > err) & ~nan & (got != want)
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}: got {got[at]!r}, "
                             f"want {want[at]!r} +- {err[at]!r}")


def assert_mx8_close(rows, want, err, what):
    """8-bit rows against values before their rounding (float64), which the float32 arithmetic
    may miss by err.  The scale is the definition's for a largest element within that error;
    the elements are within half a step at the scale that was taken."""
    n = want.shape[-1]
    got, q, s = mx8_values(rows, n)
    group = want.unflatten(-1, (-1, 32))
    finite = torch.isfinite(group).all(dim=-1)
    assert torch.equal(torch.isnan(s), ~finite), f"{what}: NaN scales in other places"
    a, d = group.abs().amax(dim=-1), err.unflatten(-1, (-1, 32)).amax(dim=-1)

    def smallest(v):
        e = torch.ceil(torch.log2(v.clamp(min=1e-300) / 448))
        e = torch.where(v / torch.exp2(e) > 448, e + 1, e)
        e = torch.where(v / torch.exp2(e - 1) <= 448, e - 1, e)
        return torch.exp2(e.clamp(min=-127))

    ok = ((s >= smallest((a - d).clamp(min=0))) & (s <= smallest(a + d))) | ~finite
    assert ok.all(), f"{what}: {int((~ok).sum())} scales off"
    step = s.repeat_interleave(32, dim=-1)
    keep = finite.repeat_interleave(32, dim=-1)
    tol = torch.maximum(2.0 ** -4 * (want.abs() + err), 2.0 ** -10 * step) + err
    bad = ((got - want).abs() > tol) & keep
    assert not bad.any(), f"{what}: {int(bad.sum())} elements off, first at {bad.nonzero()[0].tolist()}"
    row = a2av.a2av_row_bytes(a2av.MX8, n)
    assert (rows[..., n + n // 32:row].cpu() == 0).all(), f"{what}: padding"


def product(x, w, swiglu, eights=False):
    """Rows times weight rows in float64 with the bound of the arithmetic (eights: 8-bit rows, see
    above): returns (result, error before the output's rounding)."""
    k = x.shape[-1]
    v, m = x @ w.t(), x.abs() @ w.abs().t()
    err = 2 * (k + 2) * EPS32 * m
    if eights:
        err = err + 7 * 2.0 ** -13 * (x.abs().unflatten(-1, (-1, 8)).amax(-1) @ w.abs().unflatten(-1, (-1, 8)).amax(-1).t())
    if not swiglu:
        return v, err
    h = v.shape[-1] // 2
    g, u, eg, eu = v[:, :h], v[:, h:], err[:, :h], err[:, h:]
    act = g / (1 + torch.exp(-g))
    # |silu'| <= 1.1; the exponential's argument g * log2(e) is rounded (|g| * 2 eps32 in the
    # exponential, with a step or two of its own), then an addition, a division and a product
    ea = 1.1 * eg + act.abs() * (8 + 4 * g.abs()) * EPS32
    return act * u, ea * u.abs() + (act.abs() + ea) * eu + act.abs() * u.abs() * 2 * EPS32


def offsets_of(counts):
    c = np.asarray(counts)
    off = np.zeros((c.shape[0], c.shape[1] + 1), np.int32)
    off[:, 1:] = np.cumsum(c, axis=1)
    return torch.from_numpy(off)
