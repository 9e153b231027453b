"""The norm before the exchange and the experts' products: what their entry points refuse,
checked on the host before anything touches a GPU (the pointers below are never
dereferenced), row sizes, and the 8-bit row type's configurations.  Runs without a GPU."""
import ctypes

import pytest
import torch

from moe_alltoallv_resident_amd import a2av

vp = ctypes.c_void_p
A = 1 << 20          # distinct, far apart, aligned stand-ins for device addresses


def P(i, off=0):
    return vp((i + 1) * (A << 8) + off)


def test_row_bytes():
    assert a2av.a2av_row_bytes(a2av.F32, 7) == 28
    assert a2av.a2av_row_bytes(a2av.BF16, 7) == 14
    assert a2av.a2av_row_bytes(a2av.MX8, 32) == 48         # 32 + 1, padded
    assert a2av.a2av_row_bytes(a2av.MX8, 512) == 528
    assert a2av.a2av_row_bytes(a2av.MX8, 5120) == 5280
    for dtype, n in ((a2av.MX8, 33), (a2av.MX8, 0), (a2av.F32, 0), (a2av.BF16, -1), (a2av.MX4, 32), (9, 32)):
        assert a2av.a2av_row_bytes(dtype, n) == -1


def norm(x=P(0), residual=P(1), weight=P(2), residual_out=P(3), y=P(4), y8=P(5), rows=2, hidden=64, dtype=a2av.BF16,
         eps=1e-5):
    return a2av.lib().a2av_rmsnorm(x, residual, weight, residual_out, y, y8, rows, hidden, dtype, eps, None)


@pytest.mark.parametrize("bad", [
    dict(dtype=a2av.MX8), dict(dtype=9), dict(rows=-1), dict(rows=1 << 31), dict(hidden=0), dict(hidden=65537),
    dict(eps=-1.0), dict(eps=float("nan")), dict(x=None), dict(residual=None),       # residual_out without residual
    dict(residual_out=None, y=None, y8=None), dict(hidden=48), dict(y8=P(5, 8)),
    dict(x=P(0, 1)), dict(weight=P(2, 1)), dict(x=P(0, 2), dtype=a2av.F32), dict(y=P(4, 3)),
    dict(y=P(3)), dict(y8=P(0)), dict(y8=P(4, 128)), dict(y=P(2)), dict(y=P(0, 128)), dict(residual_out=P(1, 2)),
])
def test_norm_refuses(bad):
    assert norm(**bad) == a2av.ERR_INVALID


def test_norm_of_no_rows_is_nothing():
    assert norm(rows=0) == a2av.OK
    assert norm(rows=0, x=None, residual=None, weight=None, residual_out=None, y8=None) == a2av.OK


def matmul(inp=P(0), off=P(1), weight=P(2), scales=None, out=P(3), status=P(4), **over):
    c = dict(num_ranks=2, experts_per_rank=3, capacity_rows=8, k=64, n=64, in_dtype=a2av.BF16, weight_dtype=a2av.BF16,
             out_dtype=a2av.BF16, activation=a2av.ACT_NONE)
    c.update(over)
    cfg = a2av.Matmul(*(c[f] for f, _ in a2av.Matmul._fields_))
    return a2av.lib().a2av_expert_matmul(ctypes.byref(cfg), inp, off, weight, scales, out, status, None)


MXW = dict(in_dtype=a2av.MX8, weight_dtype=a2av.MX8, scales=P(5))
FPW = dict(weight_dtype=a2av.MX4, scales=P(5))


@pytest.mark.parametrize("bad", [
    dict(num_ranks=0), dict(experts_per_rank=0), dict(num_ranks=64, experts_per_rank=65), dict(capacity_rows=-1),
    dict(capacity_rows=1 << 31), dict(capacity_rows=1 << 30), dict(k=0), dict(n=0), dict(k=(1 << 20) + 1), dict(n=(1 << 20) + 1),
    dict(in_dtype=a2av.F32), dict(in_dtype=a2av.MX4), dict(weight_dtype=a2av.F32), dict(weight_dtype=a2av.MX8, scales=P(5)),
    dict(out_dtype=a2av.F32), dict(out_dtype=a2av.MX8), dict(activation=2), dict(n=65, activation=a2av.ACT_SWIGLU),
    dict(MXW, k=48), dict(FPW, k=48), dict(MXW, n=48, out_dtype=a2av.MX8),
    dict(MXW, n=96, out_dtype=a2av.MX8, activation=a2av.ACT_SWIGLU), dict(MXW, scales=None), dict(scales=P(5)),
    dict(off=None), dict(weight=None), dict(status=None), dict(inp=None), dict(out=None),
    dict(off=P(1, 2)), dict(status=P(4, 1)), dict(inp=P(0, 1)), dict(out=P(3, 1)), dict(weight=P(2, 1)),
    dict(MXW, inp=P(0, 8)), dict(MXW, weight=P(2, 8)), dict(FPW, weight=P(2, 4)), dict(MXW, out=P(3, 8), out_dtype=a2av.MX8),
    dict(k=1 << 15, n=1 << 15), dict(FPW, k=1 << 16, n=1 << 16),      # an expert's weight of 2 GiB
    dict(out=P(0)), dict(out=P(0, 1024)), dict(out=P(2)), dict(out=P(1, -8)), dict(FPW, out=P(5)),
])
def test_matmul_refuses(bad):
    assert matmul(**bad) == a2av.ERR_INVALID


def test_matmul_without_a_configuration():
    assert a2av.lib().a2av_expert_matmul(None, P(0), P(1), P(2), None, P(3), P(4), None) == a2av.ERR_INVALID


def test_matmul_of_an_empty_capacity_is_nothing():
    assert matmul(capacity_rows=0) == a2av.OK
    assert matmul(capacity_rows=0, inp=None, out=None) == a2av.OK


def test_mx8_workspace_holds_the_returned_rows():
    # staged: the send buffer holds 8-bit rows on the way out and bfloat16 rows on the way back
    R, T, H, epr, k = 8, 128, 5120, 16, 2
    mx = a2av.a2av_workspace_bytes(a2av.make_config(R, T, H, a2av.MX8, epr, k))
    assert mx == a2av.a2av_workspace_bytes(a2av.make_config(R, T, H, a2av.BF16, epr, k))
    assert a2av.a2av_workspace_bytes(a2av.make_config(R, T, H + 16, a2av.MX8, epr, k)) == -1    # not in 32s
    assert a2av.a2av_workspace_bytes(a2av.make_config(R, T, H, a2av.MX4, epr, k)) == -1


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        a2av.rmsnorm(x, None, 1e-5, y=torch.empty_like(x))
    with pytest.raises(TypeError):
        a2av.rmsnorm([1.0], None, 1e-5)
    off, st = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        a2av.expert_matmul(x[None], off, torch.zeros(1, 8, 64, dtype=torch.bfloat16), x[None, :, :8], st)
