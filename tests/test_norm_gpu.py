"""a2av_rmsnorm against its definition in 64 bits."""
import pytest
import torch

from moe_alltoallv_resident_amd import a2av
from tests.gpu_util import banner
from tests.layer_util import EPS32, HALF_STEP, TORCH, assert_close, assert_mx8_close, mx8_values

pytestmark = pytest.mark.gpu
EPS = 1e-5


def reference(x, residual, weight, eps=EPS):
    s = x.cpu().double() + (residual.cpu().double() if residual is not None else 0)
    v = s / torch.sqrt((s * s).mean(dim=-1, keepdim=True) + eps)
    v = v * (weight.cpu().double() if weight is not None else 1)
    return s, v


def bound(v):
    # a thread sums at most 128 squares, then 6 lane steps and 16 wavefronts: relative error of
    # the sum 2 * 150 eps32, halved by the root; the addition, its square (counted), the division,
    # root, reciprocal and two products add a step each
    return v.abs() * (150 + 10) * EPS32 * 2 + 2.0 ** -149


def make(rows, hidden, dtype, seed=0, offset=0):
    g = torch.Generator().manual_seed(seed)
    big = torch.randn(rows * hidden + offset, generator=g).to(TORCH[dtype]).cuda()
    return big[offset:].view(rows, hidden)


def check(x, residual, weight, ro, y, y8, dtype, what):
    s, v = reference(x, residual, weight)
    if ro is not None:
        assert_close(ro.cpu().double(), s, s.abs() * (HALF_STEP[dtype] * (1 + 2 * EPS32) + EPS32), what + " residual_out")
    if y is not None:
        e = bound(v)
        assert_close(y.cpu().double(), v, e + (v.abs() + e) * HALF_STEP[dtype], what + " y")
    if y8 is not None:
        assert_mx8_close(y8, v, bound(v), what + " y8")


@pytest.mark.parametrize("dtype", [a2av.F32, a2av.BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", [(1, 1), (1, 32), (1, 5120), (2, 65536), (3, 2047), (5, 96), (4, 7), (7, 4099),
                                         (9, 4128), (130, 2048), (33, 512), (6, 544), (2, 65535), (3, 16416), (1027, 64),
                                         (3, 8192), (2, 16384), (2, 32800), (600, 7168), (1500, 5120)])
def test_norm(rows, hidden, dtype):
    banner(f"rmsnorm {rows}x{hidden} dtype {dtype}")
    x, r, w = make(rows, hidden, dtype), make(rows, hidden, dtype, 1), make(1, hidden, dtype, 2)[0]
    x *= 3
    for residual in (None, r):
        for weight in (None, w):
            ro = torch.full_like(x, 9) if residual is not None else None
            y = torch.full_like(x, 9)
            y8 = None
            if hidden % 32 == 0:
                y8 = torch.full((rows, a2av.a2av_row_bytes(a2av.MX8, hidden)), 0xAA, dtype=torch.uint8, device="cuda")
            a2av.rmsnorm(x, weight, EPS, residual, ro, y, y8)
            check(x, residual, weight, ro, y, y8, dtype, f"{residual is not None} {weight is not None}")


@pytest.mark.parametrize("dtype", [a2av.F32, a2av.BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("hidden", [64, 5120, 24])
def test_addresses_that_are_not_16_byte_aligned(hidden, dtype):
    x, r = make(5, hidden, dtype, 0, 1), make(5, hidden, dtype, 1, 3)
    w = make(1, hidden, dtype, 2, 1)[0]
    ro, y = make(5, hidden, dtype, 3, 1), make(5, hidden, dtype, 4, 5)
    a2av.rmsnorm(x, w, EPS, r, ro, y)
    check(x, r, w, ro, y, None, dtype, "offset")


def test_each_output_alone_and_nothing_else_is_written():
    rows, hidden = 37, 1056
    x, r, w = make(rows, hidden, a2av.BF16), make(rows, hidden, a2av.BF16, 1), make(1, hidden, a2av.BF16, 2)[0]
    row8 = a2av.a2av_row_bytes(a2av.MX8, hidden)
    for which in range(3):
        guard = torch.full((rows + 2, hidden), 7, dtype=torch.bfloat16, device="cuda")
        guard8 = torch.full((rows + 2, row8), 7, dtype=torch.uint8, device="cuda")
        out, out8 = guard[1:-1], guard8[1:-1]
        a2av.rmsnorm(x, w, EPS, r, out if which == 0 else None, out if which == 1 else None, out8 if which == 2 else None)
        check(x, r, w, out if which == 0 else None, out if which == 1 else None, out8 if which == 2 else None, a2av.BF16,
              "alone")
        assert (guard[0] == 7).all() and (guard[-1] == 7).all() and (guard8[0] == 7).all() and (guard8[-1] == 7).all()


@pytest.mark.parametrize("hidden", [512, 5120, 24576])
def test_in_place(hidden):
    for dtype in (a2av.F32, a2av.BF16):
        x, r, w = make(40, hidden, dtype), make(40, hidden, dtype, 1), make(1, hidden, dtype, 2)[0]
        ro, y = torch.empty_like(x), torch.empty_like(x)
        a2av.rmsnorm(x, w, EPS, r, ro, y)
        x1, r1 = x.clone(), r.clone()
        a2av.rmsnorm(x1, w, EPS, r1, r1, x1)
        assert torch.equal(r1, ro) and torch.equal(x1, y)
        x1, r1 = x.clone(), r.clone()
        a2av.rmsnorm(x1, w, EPS, r1, x1, r1)
        assert torch.equal(x1, ro) and torch.equal(r1, y)


def test_rows_of_zeros_infinities_and_nan():
    hidden = 320
    for dtype in (a2av.F32, a2av.BF16):
        x = make(6, hidden, dtype)
        x[0] = 0
        x[1, 5] = float("inf")
        x[2, 300] = float("nan")
        x[3] *= 1e-18
        x[4, 64:96] = 0                                     # a scale's 32 elements all zero
        x[5, 0] = -float("inf")
        y = torch.empty_like(x)
        y8 = torch.empty((6, a2av.a2av_row_bytes(a2av.MX8, hidden)), dtype=torch.uint8, device="cuda")
        a2av.rmsnorm(x, None, EPS, y=y, y8=y8)
        _, v = reference(x, None, None)
        e = bound(v)
        assert_close(y.cpu().double(), v, e + (v.abs() + e) * HALF_STEP[dtype], "y")
        assert_mx8_close(y8, v, e, "y8")
        # eps = 0: a row of zeros divides by zero
        a2av.rmsnorm(x, None, 0.0, y=y)
        assert torch.isnan(y[0]).all()


def test_scales_at_the_borders():
    """Elements right at 448 * 2^e and past it.  A row of ones has the root mean square 1 (eps =
    0), so the weight itself comes out and the scale bytes are known exactly."""
    hidden = 64
    for at, byte in ((448.0, 127), (448.0 * 2 ** -20, 107), (448.00003, 128), (1.75, 119), (1.875, 120), (256.0, 127),
                     (512.0, 128), (2.0 ** -126, 0), (2.0 ** -118, 1), (1.75 * 2.0 ** -119, 0), (3e38, 247), (1e38, 245)):
        w = torch.zeros(hidden, device="cuda")
        w[3] = at
        x = torch.ones((1, hidden), device="cuda")
        y8 = torch.empty((1, a2av.a2av_row_bytes(a2av.MX8, hidden)), dtype=torch.uint8, device="cuda")
        a2av.rmsnorm(x, w, 0.0, y8=y8)
        got = y8.cpu()[0]
        at = float(w[3])
        assert 448 * 2.0 ** (byte - 127) >= at and (byte == 0 or 448 * 2.0 ** (byte - 128) < at), "the test's own bytes"
        assert int(got[hidden]) == byte, (at, int(got[hidden]))
        assert int(got[hidden + 1]) == 0                     # a group of zeros: the smallest scale
        v, _, _ = mx8_values(y8, hidden)
        assert abs(float(v[0, 3]) - at) <= at * 2.0 ** -4


def test_strided_and_host_tensors_are_refused():
    x = make(4, 64, a2av.BF16)
    with pytest.raises(ValueError):
        a2av.rmsnorm(x[:, ::2], None, EPS, y=x[:, ::2])
    with pytest.raises(ValueError):
        a2av.rmsnorm(x, None, EPS, y=x.cpu())
    with pytest.raises(TypeError):
        a2av.rmsnorm(x, x[0].float(), EPS, y=torch.empty_like(x))
    with pytest.raises(ValueError):
        a2av.rmsnorm(x, None, EPS, y8=torch.empty((4, 64), dtype=torch.uint8, device="cuda"))
    with pytest.raises(a2av.A2AVError):
        a2av.rmsnorm(x, None, EPS)                           # no output


def test_no_rows():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    a2av.rmsnorm(x, None, EPS, y=torch.empty_like(x))


def test_other_stream_and_graph():
    x, w = make(64, 5120, a2av.BF16), make(1, 5120, a2av.BF16, 2)[0]
    y, y8 = torch.empty_like(x), torch.empty((64, 5280), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a2av.rmsnorm(x, w, EPS, y=y, y8=y8)
    torch.cuda.current_stream().wait_stream(side)
    check(x, None, w, None, y, y8, a2av.BF16, "side stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a2av.rmsnorm(x, w, EPS, y=y, y8=y8)
    for i in range(3):
        x.copy_(make(64, 5120, a2av.BF16, 10 + i))
        y.zero_()
        y8.zero_()
        g.replay()
        torch.cuda.synchronize()
        check(x, None, w, None, y, y8, a2av.BF16, f"replay {i}")
        e, e8 = torch.empty_like(y), torch.empty_like(y8)
        a2av.rmsnorm(x, w, EPS, y=e, y8=e8)
        assert torch.equal(e, y) and torch.equal(e8, y8)
