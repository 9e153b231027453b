"""a2av_expert_matmul against its definition in 64 bits: every element type, ragged groups
from none to several tiles, odd sizes and addresses, dropped rows, bad group starts; and the
whole layer (norm, 8-bit dispatch, two products, combine) as it would be used."""
import numpy as np
import pytest
import torch

from moe_alltoallv_resident_amd import a2av
from tests.gpu_util import banner
from tests.layer_util import (HALF_STEP, TORCH, assert_close, assert_mx8_close, encode_mx8, mx8_values, offsets_of, product,
                              values)

pytestmark = pytest.mark.gpu
F32, BF16, MX8, MX4 = a2av.F32, a2av.BF16, a2av.MX8, a2av.MX4
NAME = {F32: "f32", BF16: "bf16", MX8: "mx8", MX4: "mx4"}
KINDS = [(F32, F32, F32), (BF16, BF16, BF16), (BF16, MX4, BF16), (MX8, MX8, BF16), (MX8, MX8, MX8), (MX8, MX4, BF16),
         (MX8, MX4, MX8)]
kinds = pytest.mark.parametrize("kind", KINDS, ids=["-".join(NAME[k] for k in ks) for ks in KINDS])


def rows_of(shape, kind, seed, offset=0):
    """Rows N(0, 1) of an element type on the GPU; `offset`: elements before the first, so that the
    address is not a multiple of 16 bytes."""
    v = torch.randn(shape, generator=torch.Generator().manual_seed(seed))
    if kind == MX8:
        return encode_mx8(v).cuda()
    flat = torch.zeros(v.numel() + offset, dtype=TORCH[kind], device="cuda")
    flat[offset:] = v.flatten().to(TORCH[kind])
    return flat[offset:].view(shape)


def weights_of(shape, kind, seed, offset=0):
    g = torch.Generator().manual_seed(seed)
    k = shape[-1]
    if kind == MX4:
        return (torch.randint(0, 256, shape[:-1] + (k // 2,), generator=g, dtype=torch.uint8).cuda(),
                torch.randint(119, 128, shape[:-1] + (k // 32,), generator=g, dtype=torch.uint8).cuda())
    if kind == MX8:
        rows = encode_mx8(torch.randn(shape, generator=g))
        return rows[..., :k].contiguous().cuda(), rows[..., k:k + k // 32].contiguous().cuda()
    return rows_of(shape, kind, seed, offset), None


class Case:
    def __init__(self, counts, k, n, kind, swiglu, cap=None, seed=0, offset=0):
        self.kind, self.k, self.n, self.swiglu = kind, k, n, swiglu
        self.off_host = offsets_of(counts)
        self.R, self.epr = len(counts), len(counts[0])
        self.cap = int(self.off_host.max()) + 3 if cap is None else cap
        self.width = n // 2 if swiglu else n
        i, w, o = kind
        self.x = rows_of((self.R, self.cap, k), i, seed, offset)
        self.w, self.ws = weights_of((self.R * self.epr, n, k), w, seed + 1, offset)
        cols = a2av.a2av_row_bytes(MX8, self.width) if o == MX8 else self.width
        flat = torch.full((self.R * self.cap * cols + offset,), 77, dtype=a2av.TORCH_DTYPE[o], device="cuda")
        self.out = flat[offset:].view(self.R, self.cap, cols)
        self.off = self.off_host.cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, stream=None):
        i, w, o = self.kind
        a2av.expert_matmul(self.x, self.off, self.w, self.out, self.status, self.ws, i, w, o,
                           a2av.ACT_SWIGLU if self.swiglu else a2av.ACT_NONE, stream)
        return self

    def check(self, status=0, groups=None):
        i, w, o = self.kind
        assert int(self.status.item()) == status
        out = self.out.cpu()
        untouched = torch.ones(self.R, self.cap, dtype=torch.bool)
        owners = torch.zeros(self.R, self.cap, dtype=torch.int32)   # groups that a row is in
        for d in range(self.R):
            for a, b in zip(self.off_host[d, :-1].tolist(), self.off_host[d, 1:].tolist()):
                if 0 <= a <= b:
                    owners[d, a:b] += 1
        for d in range(self.R):
            for le in range(self.epr):
                a, b = (int(v) for v in self.off_host[d, le:le + 2])
                if a < 0 or b < a:
                    continue
                a, b = min(a, self.cap), min(b, self.cap)
                if a == b:
                    continue
                e = d * self.epr + le
                untouched[d, a:b] = False
                x = values(self.x[d, a:b], i, self.k)
                wt = values(self.w[e], w, self.k, None if self.ws is None else self.ws[e])
                want, err = product(x, wt, self.swiglu, i == MX8)
                what = f"rank {d} expert {le} rows {a}:{b}"
                # after a bad start two groups may share rows: those hold either's, so nothing is said of them
                one = owners[d, a:b] == 1
                assert status or one.all()
                rows, want, err = out[d, a:b][one], want[one], err[one]
                if o == MX8:
                    assert_mx8_close(rows, want, err, what)
                else:
                    # an infinite product stays one; bfloat16's smallest numbers are steps of 2^-133
                    assert_close(rows.double(), want, err + (want.abs() + err) * HALF_STEP[o] + 2.0 ** -134, what)
        assert (out[untouched] == 77).all(), "rows in no group were written"
        return self


SMALL = [[0, 1, 5], [16, 0, 2], [0, 0, 0]]
RAGGED = [[1, 17, 0, 33], [64, 0, 129, 2], [0, 31, 257, 65]]
LONG = [[700, 3], [0, 1025]]


@kinds
@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("counts,k,n", [(SMALL, 32, 64), (SMALL, 160, 192), (SMALL, 2048, 320), (RAGGED, 96, 128),
                                        (RAGGED, 512, 576), (RAGGED, 1056, 64), (LONG, 256, 512), (LONG, 416, 448),
                                        ([[1]], 5120, 1024), ([[3, 1, 0, 2, 1, 1, 4, 0]], 7168, 128)],
                         ids=lambda v: str(v) if isinstance(v, int) else "c%d" % sum(map(sum, v)))
def test_products(kind, swiglu, counts, k, n):
    banner(f"experts {kind} swiglu {swiglu} rows {sum(map(sum, counts))} k {k} n {n}")
    Case(counts, k, n, kind, swiglu).run().check()


# groups of every tile height and row tiles for more than half of the GPU's units
BIG = [[300, 1100, 700, 20], [257, 129, 65, 600]]


@kinds
@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("k,n", [(32, 2112), (96, 2112), (416, 2112), (128, 2560), (640, 2112)])
def test_many_rows(kind, swiglu, k, n):
    banner(f"many rows {kind} swiglu {swiglu} k {k} n {n}")
    Case(BIG, k, n, kind, swiglu).run().check()


def test_many_rows_repeat_bit_for_bit():
    for kind in (KINDS[0], KINDS[1], KINDS[2], KINDS[4], KINDS[5]):
        c = Case(BIG, 1024, 2112, kind, True).run()
        torch.cuda.synchronize()
        want = c.out.clone()
        for _ in range(5):
            c.out.fill_(77)
            c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want)


@pytest.mark.parametrize("kind", [KINDS[0], KINDS[1]], ids=["f32", "bf16"])
def test_many_rows_of_odd_widths(kind):
    for k, n, swiglu in ((104, 2090, False), (104, 2090, True), (200, 2051, False), (64, 2050, True)):
        Case(BIG, k, n, kind, swiglu).run().check()


@pytest.mark.parametrize("kind", [KINDS[0], KINDS[1]], ids=["f32", "bf16"])
@pytest.mark.parametrize("k,n,offset", [(1, 2, 0), (7, 6, 0), (33, 34, 0), (130, 154, 0), (1001, 70, 0), (64, 66, 1),
                                        (256, 128, 3), (72, 10, 0), (200, 130, 0)])
def test_odd_sizes_and_addresses(kind, k, n, offset):
    for swiglu in (False, True):
        banner(f"odd {kind} k {k} n {n} offset {offset} swiglu {swiglu}")
        Case(RAGGED, k, n, kind, swiglu, offset=offset).run().check()


@pytest.mark.parametrize("kind", [KINDS[2], KINDS[3], KINDS[5]], ids=["bf16-mx4", "mx8-mx8", "mx8-mx4"])
def test_odd_widths_of_scaled_weights(kind):
    for n, swiglu in ((1, False), (2, True), (37, False), (74, True), (131, False)):
        banner(f"odd width {kind} n {n}")
        Case(RAGGED, 224, n, kind, swiglu).run().check()


@kinds
def test_rows_past_the_capacity_are_dropped(kind):
    counts = [[5, 40, 20], [0, 0, 3], [70, 1, 1]]
    for cap in (1, 44, 45, 60, 64):
        banner(f"capacity {cap}")
        Case(counts, 128, 64, kind, False, cap=cap).run().check()


@kinds
def test_bad_group_starts(kind):
    c = Case([[5, 9, 20], [2, 0, 3]], 64, 64, kind, False)
    c.off_host = torch.tensor([[0, 5, 3, 20], [-4, 2, 2, 1 << 30]], dtype=torch.int32)
    c.off = c.off_host.cuda()
    c.run().check(status=a2av.ST_OFFSETS)
    c.off_host = torch.tensor([[-2147483648, 2147483647, -1, 3], [7, 7, 7, 7]], dtype=torch.int32)
    c.off = c.off_host.cuda()
    c.out.fill_(77)
    c.run().check(status=a2av.ST_OFFSETS)


def test_more_groups_than_threads():
    rng = np.random.default_rng(3)
    counts = rng.integers(0, 3, (64, 64))
    counts[5] = 0
    counts[63, 63] = 40
    for kind in (KINDS[1], KINDS[6]):
        Case(counts, 64, 64, kind, False).run().check()
    Case(np.zeros((4, 8), np.int64), 64, 64, KINDS[1], False).run().check()


@pytest.mark.parametrize("kind,k", [(KINDS[1], 64), (KINDS[4], 128), (KINDS[0], 33), (KINDS[1], 33)],
                         ids=["bf16", "mx8", "f32-odd", "bf16-odd"])
def test_many_groups_with_many_rows(kind, k):
    """More groups than the list of row tiles has entries, some of several tiles."""
    rng = np.random.default_rng(4)
    counts = rng.integers(0, 2, (75, 16))
    for at in (3, 599, 600, 607, 1100):
        counts.flat[at] = 700 + at % 7
    counts[74, 15] = 300
    Case(counts, k, 2112, kind, False).run().check()


@pytest.mark.parametrize("kind", KINDS[2:], ids=["-".join(NAME[k] for k in ks) for ks in KINDS[2:]])
@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("k,shift", [(32, 0), (160, 0), (416, 0), (1056, 0), (512, 1), (640, 2), (160, 3)])
def test_scale_rows_of_any_length_and_address(kind, swiglu, k, shift):
    """Rows of scales that are not whole words: by their length or because they start `shift` bytes
    past a word, the last ones next to the allocation's end; few rows, few rows of enough groups for
    every unit of the GPU, many rows."""
    many = np.random.default_rng(6).integers(0, 33, (16, 8))
    for counts, n in ((SMALL, 192), (many, 832), (BIG, 2112)):
        banner(f"scales {kind} swiglu {swiglu} k {k} shift {shift} n {n}")
        c = Case(counts, k, n, kind, swiglu)
        flat = torch.full((c.ws.numel() + shift,), 255, dtype=torch.uint8, device="cuda")   # NaN in front
        flat[shift:] = c.ws.flatten()
        c.ws = flat[shift:].view(c.ws.shape)
        c.run().check()


@pytest.mark.parametrize("kind", [KINDS[0], KINDS[1]], ids=["f32", "bf16"])
@pytest.mark.parametrize("k", [3, 31, 65, 127, 191, 193, 257, 515])
def test_rows_of_any_length(kind, k):
    """Rows of no whole step and of one to many, with and without a rest shorter or longer than a
    load, for groups of 1, 16 and more rows."""
    for counts in ([[1]], [[16, 17], [0, 130]]):
        for swiglu in (False, True):
            banner(f"odd rows {kind} k {k} {counts} swiglu {swiglu}")
            Case(counts, k, 70, kind, swiglu).run().check()
            Case(counts, k, 70, kind, swiglu, offset=1).run().check()


@kinds
def test_infinities_and_nan_stay_in_their_row(kind):
    """A NaN in a row or an infinity in it reaches that row's outputs and no other's."""
    i, w, o = kind
    c = Case([[40, 3]], 256, 64, kind, False)
    if i == MX8:
        c.x[0, 7, 256 + 3] = 255                             # a scale that is NaN
        c.x[0, 41, 9] = 0x7F                                 # an element that is
    else:
        c.x[0, 7, 100] = float("nan")
        c.x[0, 41, 9] = float("inf")
    c.run()
    got = mx8_values(c.out, 64)[0] if o == MX8 else c.out.cpu().double()
    bad = ~torch.isfinite(got[0])
    rows = torch.zeros(43, dtype=torch.bool)
    rows[[7, 41]] = True
    assert bad[:43].any(dim=1).equal(rows)
    assert bad[7].all()


@pytest.mark.parametrize("kind", [KINDS[2], KINDS[5], KINDS[3]], ids=["bf16-mx4", "mx8-mx4", "mx8-mx8"])
def test_scales_over_their_range(kind):
    for rows in (3, 40):
        c = Case([[rows, 2]], 128, 64, kind, False)
        c.ws[0, 0] = 127 + 100                               # 2^100
        c.ws[0, 1] = 127 - 100
        c.ws[0, 2, 1] = 255                                  # NaN
        c.ws[0, 3] = 1                                       # 2^-126
        c.ws[0, 4] = 127
        c.run().check()


def test_other_stream_and_graph():
    """Captured once, replayed with other rows and group starts: what a decode step does."""
    for kind in (KINDS[1], KINDS[2], KINDS[6]):
        c = Case(RAGGED, 512, 256, kind, True, cap=400)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        c.run(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        c.check()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        rng = np.random.default_rng(1)
        for i in range(4):
            counts = rng.integers(0, (3, 20, 100, 1)[i] + 1, (c.R, c.epr))
            c.off_host = offsets_of(counts)
            c.off.copy_(c.off_host)
            c.x.copy_(rows_of((c.R, c.cap, c.k), kind[0], 50 + i))
            c.out.fill_(77)
            g.replay()
            torch.cuda.synchronize()
            c.check()
            eager = c.out.clone()
            c.out.fill_(77)
            c.run()
            torch.cuda.synchronize()
            assert torch.equal(eager, c.out), "a replay and an eager call differ"


def test_calls_repeat_bit_for_bit_and_two_streams_do_not_meet():
    a, b = Case(LONG, 1024, 512, KINDS[1], False), Case(RAGGED, 1024, 512, KINDS[6], True, seed=9)
    a.run(), b.run()
    torch.cuda.synchronize()
    wa, wb = a.out.clone(), b.out.clone()
    a.out.fill_(77), b.out.fill_(77)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.run(stream=s1)
        b.run(stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(a.out, wa) and torch.equal(b.out, wb)


def test_rows_past_4_gib():
    """The last rank's slice and the last expert's weight start past 2^32 bytes."""
    R, cap, k, n = 3, 900_000, 1024, 2048
    x = torch.zeros((R, cap, k), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((R, cap, n), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros((R, 401), dtype=torch.int32)
    off[2, :400], off[2, 400] = cap - 40, cap - 3            # the last group alone has rows, 37 of them
    w = torch.zeros((R * 400, n, k), dtype=torch.bfloat16, device="cuda")
    x[2, cap - 40:] = rows_of((40, k), BF16, 1)
    w[-1] = rows_of((n, k), BF16, 2)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    a2av.expert_matmul(x, off.cuda(), w, out, st)
    want, err = product(values(x[2, cap - 40:cap - 3], BF16, k), values(w[-1], BF16, k), False)
    assert_close(out[2, cap - 40:cap - 3].cpu().double(), want, err + (want.abs() + err) * HALF_STEP[BF16], "far rows")
    assert not out[2, cap - 3:].any() and not out[2, cap - 50:cap - 40].any() and not out[0, :64].any()
    assert int(st.item()) == 0


def test_tensors_are_checked():
    c = Case([[3]], 64, 64, KINDS[1], False)
    with pytest.raises(ValueError):
        a2av.expert_matmul(c.x[:, :, ::2], c.off, c.w, c.out, c.status)
    with pytest.raises(ValueError):
        a2av.expert_matmul(c.x, c.off, c.w[:, :32].contiguous(), c.out, c.status)
    with pytest.raises(TypeError):
        a2av.expert_matmul(c.x, c.off.long(), c.w, c.out, c.status)
    with pytest.raises(TypeError):
        a2av.expert_matmul(c.x, c.off, c.w, c.out, c.status, weight_dtype=MX8)
    with pytest.raises(ValueError):
        a2av.expert_matmul(c.x, c.off.cpu(), c.w, c.out, c.status)
    with pytest.raises(a2av.A2AVError):
        a2av.expert_matmul(c.x, c.off, c.w, c.x, c.status)


@pytest.mark.parametrize("path", [a2av.PATH_STAGED, a2av.PATH_DIRECT], ids=["staged", "direct"])
@pytest.mark.parametrize("R,T,epr,top_k,cap", [(4, 24, 2, 2, 0), (8, 128, 4, 1, 0), (4, 600, 4, 2, 0), (4, 24, 2, 2, 20)])
def test_8_bit_rows_through_the_exchange(path, R, T, epr, top_k, cap):
    """8-bit rows are moved as they are: the same tables and receive bytes as a bfloat16 session
    whose rows have those bytes; the combine then takes bfloat16 rows of the hidden size."""
    H = 288
    g = torch.Generator().manual_seed(4)
    row = a2av.a2av_row_bytes(MX8, H)
    x = torch.randint(0, 256, (R, T, row), generator=g, dtype=torch.uint8).cuda()
    ids = torch.randint(0, R * epr, (R, T, top_k), generator=g, dtype=torch.int32).cuda()
    gates = torch.rand((R, T, top_k), generator=g).cuda()
    for layout in (a2av.LAYOUT_SOURCE_MAJOR, a2av.LAYOUT_EXPERT_MAJOR):
        m = a2av.Session(R, T, H, MX8, epr, top_k, cap, path, layout)
        b = a2av.Session(R, T, row // 2, BF16, epr, top_k, cap, path, layout)
        o = a2av.Session(R, T, H, BF16, epr, top_k, cap, path, layout)
        for s in (m, b, o):
            s.recv.zero_()
        m.dispatch(x, ids)
        b.dispatch(x.view(torch.bfloat16), ids)
        o.dispatch(torch.zeros((R, T, H), dtype=torch.bfloat16, device="cuda"), ids)
        torch.cuda.synchronize()
        assert torch.equal(m.recv, b.recv.view(torch.uint8).view(m.recv.shape))
        assert torch.equal(m.recv_offsets, b.recv_offsets) and torch.equal(m.split, b.split)
        assert torch.equal(m.positions(), b.positions()) and torch.equal(m.status, b.status)
        expert_out = torch.randn((R, m.cap, H), generator=g).to(torch.bfloat16).cuda()
        y, yo = torch.empty((R, T, H), dtype=torch.bfloat16, device="cuda"), torch.empty((R, T, H), dtype=torch.bfloat16,
                                                                                        device="cuda")
        m.combine(expert_out, gates, y)
        o.combine(expert_out, gates, yo)
        torch.cuda.synchronize()
        assert torch.equal(y, yo)
        with pytest.raises(a2av.A2AVError):
            a2av.a2av_expert_apply(m.handle, m.recv, m.recv, a2av.EXPERT_IDENTITY)
        for s in (m, b, o):
            s.close()


def test_8_bit_rows_through_the_bare_collective():
    R, T, H = 4, 40, 96
    row = a2av.a2av_row_bytes(MX8, H)
    g = torch.Generator().manual_seed(6)
    send = torch.randint(0, 256, (R, T, row), generator=g, dtype=torch.uint8).cuda()
    counts = torch.tensor([[10, 0, 20, 5], [0, 0, 0, 40], [1, 2, 3, 4], [0, 0, 0, 0]], dtype=torch.int32).cuda()
    out = []
    for dtype, hidden in ((MX8, H), (BF16, row // 2)):
        cfg = a2av.make_config(R, T, hidden, dtype, 1, 1)
        recv = torch.zeros((R, R * T, row), dtype=torch.uint8, device="cuda")
        again = torch.zeros_like(recv)
        rc, st = torch.zeros((R, R), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        h = a2av.a2av_create(cfg)
        a2av.a2av_alltoallv(h, send, counts, recv, rc, None, st)
        a2av.a2av_alltoallv_noalloc(cfg, send, counts, again, rc, None, st)
        torch.cuda.synchronize()
        a2av.a2av_destroy(h)
        assert int(st.item()) == 0 and torch.equal(recv, again)
        out.append(recv)
    assert torch.equal(out[0], out[1]) and out[0].any()


def test_group_starts_of_the_handle():
    """The handle's own table is what the copy gives, before and after a dispatch, and only
    expert-major handles have one."""
    s = a2av.Session(2, 8, 64, BF16, 3, 2, recv_layout=a2av.LAYOUT_EXPERT_MAJOR)
    x = rows_of((2, 8, 64), BF16, 0)
    ids = torch.randint(0, 6, (2, 8, 2), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    w = rows_of((6, 32, 64), BF16, 1)
    out = torch.full((2, s.cap, 32), 77, dtype=torch.bfloat16, device="cuda")
    s.expert_matmul(s.recv, w, out)                          # nothing dispatched yet: every group is empty
    torch.cuda.synchronize()
    assert (out == 77).all()
    s.dispatch(x, ids)
    s.expert_matmul(s.recv, w, out)
    want = torch.full_like(out, 77)
    a2av.expert_matmul(s.recv, s.recv_expert_offsets(), w, want, s.status)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and not (out == 77).all() and int(s.status.item()) == 0
    assert int(s.recv_expert_offsets()[:, -1].sum()) == 2 * 8 * 2
    t = a2av.Session(2, 8, 64, BF16, 3, 2)
    assert not a2av.a2av_recv_expert_offsets(t.handle)
    with pytest.raises(ValueError):
        t.expert_matmul(t.recv, w, out)
    s.close(), t.close()


@pytest.mark.parametrize("weight", [MX8, MX4], ids=["mx8", "mx4"])
def test_the_layer_captured_and_replayed(weight):
    """Norm with the residual, 8-bit dispatch, gate and up with SwiGLU into 8-bit rows, down,
    combine: one graph, replayed with routing that changes on the device.  Checked step by step
    from the values that each step was given, so that every bound is one step's own."""
    R, T, epr, top_k, H, F = 4, 12, 4, 2, 256, 192
    E = R * epr
    s = a2av.Session(R, T, H, MX8, epr, top_k, path=a2av.PATH_DIRECT, recv_layout=a2av.LAYOUT_EXPERT_MAJOR)
    x, r = rows_of((R, T, H), BF16, 0), rows_of((R, T, H), BF16, 1)
    nw = rows_of((H,), BF16, 2)
    w1, s1 = weights_of((E, 2 * F, H), weight, 3)
    w2, s2 = weights_of((E, H, F), weight, 4)
    ro, y = torch.empty_like(x), torch.empty_like(x)
    x8 = torch.empty((R, T, a2av.a2av_row_bytes(MX8, H)), dtype=torch.uint8, device="cuda")
    mid = torch.zeros((R, s.cap, a2av.a2av_row_bytes(MX8, F)), dtype=torch.uint8, device="cuda")
    out = torch.zeros((R, s.cap, H), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros((R, T, top_k), dtype=torch.int32, device="cuda")
    gates = torch.rand((R, T, top_k), generator=torch.Generator().manual_seed(5)).cuda()

    def layer():
        a2av.rmsnorm(x, nw, 1e-5, residual=r, residual_out=ro, y8=x8)
        s.dispatch(x8, ids)
        s.expert_matmul(s.recv, w1, mid, s1, MX8, weight, MX8, a2av.ACT_SWIGLU)
        s.expert_matmul(mid, w2, out, s2, MX8, weight, BF16)
        s.combine(out, gates, y)

    layer()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    for i in range(4):
        ids.copy_(torch.randint(0, E if i else 1, (R, T, top_k), generator=torch.Generator().manual_seed(i),
                                dtype=torch.int32))
        x.copy_(rows_of((R, T, H), BF16, 60 + i))
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        off = s.recv_expert_offsets().cpu()
        assert int(s.status.item()) == 0
        v = (x.cpu().double() + r.cpu().double())
        n = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * nw.cpu().double()
        assert_mx8_close(x8.cpu(), n, n.abs() * 320 * 2.0 ** -24, "norm")
        want_y = torch.zeros(R, T, H, dtype=torch.float64)
        rows = {}
        for d in range(R):
            for le in range(epr):
                a, b = int(off[d, le]), int(off[d, le + 1])
                if a == b:
                    continue
                e = d * epr + le
                h, err = product(values(s.recv[d, a:b], MX8, H), values(w1[e], weight, H, s1[e]), True, True)
                assert_mx8_close(mid[d, a:b].cpu(), h, err, f"up {d} {le}")
                o, err = product(values(mid[d, a:b], MX8, F), values(w2[e], weight, F, s2[e]), False, True)
                assert_close(out[d, a:b].cpu().double(), o, err + (o.abs() + err) * HALF_STEP[BF16], f"down {d} {le}")
                # this expert's rows stand in the order (source, token, slot)
                at = (ids.cpu().flatten() == e).nonzero().flatten()
                assert len(at) == b - a
                for j, src in enumerate(at.tolist()):
                    rows[src] = out[d, a + j].cpu().double()
        mags = torch.zeros(R * T, H, dtype=torch.float64)
        yv = want_y.view(R * T, H)
        for src, row in rows.items():
            yv[src // top_k] += gates.flatten()[src].cpu().double() * row
            mags[src // top_k] += (gates.flatten()[src].cpu().double() * row).abs()
        assert_close(y.cpu().double().view(R * T, H), yv, yv.abs() * 2.0 ** -8 + mags * 4 * 2.0 ** -24, "combine")
    s.close()
