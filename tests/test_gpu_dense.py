"""The dense MoE operators (include/msb_dense.h) against plain 64-bit formulas on the GPU.

Tolerances, derived before the first run.  A rounding to bf16 is off by at most 2^-8 of the
value, one to float32 by 2^-24.  A sum of k products in float32 adds at most one unit of 2^-23
of the sum of magnitudes A = |x| . |w| per addition: k 2^-23 A (a bound; errors are far
smaller).  Each test states what it adds to these.
"""
import numpy as np
import pytest

import oracle
import synth
from parity import device_layer, from_bf16_tensor, require_gpu, to_bf16_tensor

pytestmark = pytest.mark.gpu

BF16, F32 = 2.0 ** -8, 2.0 ** -24
TINY = 2.0 ** -126  # below the normal range values round to multiples of 2^-133 (bf16)


@pytest.fixture(scope="module")
def msb():
    return require_gpu()


@pytest.fixture(autouse=True)
def checked(msb):
    """No kernel of the test gave up waiting."""
    import torch
    yield
    torch.cuda.synchronize()
    msb.dense_check()


def rnd(seed, *shape, scale=1.0, dtype=None):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype or torch.bfloat16)


def within(got, want, tol, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g where %.3g is allowed" % (
        what, int(bad.sum()), bad.numel(), float(err[bad].max()), float(tol[bad].min()))


def offsets_of(counts, first=0):
    import torch
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def product64(x, w, offs, rows):
    """(sums, sums of magnitudes) of every row with its group's weight [n][k]; zeros for rows
    of no group, for a row index outside x."""
    import torch
    x = x.double()
    if rows is not None:
        ok = (rows >= 0) & (rows < x.shape[0])
        x = torch.where(ok[:, None], x[rows.long().clamp(0, x.shape[0] - 1)], 0.0)
    out = torch.zeros((x.shape[0], w.shape[1]), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    at = offs.tolist()
    for e, (lo, hi) in enumerate(zip(at, at[1:])):
        if hi > lo:
            we = w[e].double()
            out[lo:hi], mag[lo:hi] = x[lo:hi] @ we.t(), x[lo:hi].abs() @ we.abs().t()
    return out, mag


def weight(seed, groups, n, k, layout):
    """bf16 [groups][n][k]: k contiguous (rows padded to 16 bytes), n contiguous, or the down
    columns of channel records."""
    if layout == "k":
        return rnd(seed, groups, n, (k + 7) // 8 * 8, scale=0.1)[:, :, :k]
    if layout == "n":
        return rnd(seed, groups, k, (n + 7) // 8 * 8, scale=0.1)[:, :, :n].transpose(1, 2)
    return rnd(seed, groups, k, 3, (n + 7) // 8 * 8, scale=0.1)[:, :, 2, :n].transpose(1, 2)


COUNTS = {"one": [1], "edges": [31, 0, 32, 33, 1, 0], "pieces": [255, 256, 257, 513],
          "empty": [0, 0, 0], "skew": [0, 700, 3, 0, 0, 64, 65]}


@pytest.mark.parametrize("layout", ["k", "n", "records"])
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("n,k", [(1, 8), (7, 33), (128, 64), (257, 200), (640, 1000)])
def test_grouped_matmul(msb, counts, n, k, layout):
    import torch
    c = COUNTS[counts]
    offs, R = offsets_of(c), sum(c)
    x = rnd(1, R, (k + 7) // 8 * 8)[:, :k]
    w = weight(2, len(c), n, k, layout)
    want, mag = product64(x, w, offs, None)
    for dtype, step in ((torch.bfloat16, BF16), (torch.float32, F32)):
        got = msb.grouped_matmul(x, w, offs, out_dtype=dtype)
        assert got.shape == (R, n) and got.dtype == dtype
        within(got, want, step * want.abs() + k * 2 * F32 * mag + TINY, dtype)


@pytest.mark.parametrize("record", [False, True])
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("n,k", [(1, 8), (33, 64), (130, 192), (500, 1024)])
def test_grouped_swiglu(msb, counts, n, k, record):
    """h = silu(g) u: with |silu'| < 1.1 an error dg, du of the sums moves h by at most
    1.1 dg |u| + |silu(g)| du + 1.1 dg du; the exponential and the quotient add 2^-20 |h|."""
    import torch
    c = COUNTS[counts]
    offs, R, T = offsets_of(c), sum(c), 50
    x = rnd(3, T, k)
    rows = torch.randint(0, T, (R,), device="cuda", dtype=torch.int32)
    if record:
        w = rnd(4, len(c), n, 3, k, scale=0.1)[:, :, :2].permute(0, 2, 1, 3)
    else:
        w = rnd(4, len(c), 2, n, k, scale=0.1)
    g, ga = product64(x, w[:, 0], offs, rows)
    u, ua = product64(x, w[:, 1], offs, rows)
    dg, du = k * 2 * F32 * ga, k * 2 * F32 * ua
    s = torch.nn.functional.silu(g)
    tol = (BF16 + 2.0 ** -20) * (s * u).abs() + 1.1 * dg * u.abs() + s.abs() * du + 1.1 * dg * du + TINY
    within(msb.grouped_swiglu(x, w, offs, rows=rows), s * u, tol)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("R,n,k", [(9, 100, 1000), (64, 640, 4096), (65, 300, 2050), (200, 1000, 1024), (3, 64, 20000)])
def test_one_group_with_few_tiles(msb, R, n, k, gather):
    """One weight and few rows: the tiles' k is shared out and joined.  Tolerances as above; 8-bit
    sums stay exact."""
    import torch
    T = 40 if gather else R
    rows = torch.randint(-1, T + 1, (R,), device="cuda", dtype=torch.int32) if gather else None
    offs = offsets_of([R])
    x = rnd(40, T, (k + 7) // 8 * 8)[:, :k]
    for layout in ("k", "n"):
        w = weight(41, 1, n, k, layout)
        want, mag = product64(x, w, offs, rows)
        for dtype, step in ((torch.bfloat16, BF16), (torch.float32, F32)):
            got = msb.grouped_matmul(x, w, rows=rows, out_dtype=dtype)
            within(got, want, step * want.abs() + k * 2 * F32 * mag + TINY, (layout, dtype))
    w2 = weight(42, 2, n, k, "k")[None]
    (g, ga), (u, ua) = (product64(x, w2[:, p], offs, rows) for p in range(2))
    dg, du, sg = k * 2 * F32 * ga, k * 2 * F32 * ua, torch.nn.functional.silu(g)
    tol = (BF16 + 2.0 ** -20) * (sg * u).abs() + 1.1 * dg * u.abs() + sg.abs() * du + 1.1 * dg * du + TINY
    within(msb.grouped_swiglu(x, w2, rows=rows), sg * u, tol + 2.0 ** -117 * u.abs(), "swiglu")
    gen = torch.Generator(device="cuda").manual_seed(43)
    q = torch.randint(-128, 128, (T, (k + 15) // 16 * 16), device="cuda", generator=gen).to(torch.int8)[:, :k]
    w8 = torch.randint(-128, 128, (n, (k + 15) // 16 * 16), device="cuda", generator=gen).to(torch.int8)[:, :k]
    one, ones = torch.ones(T, device="cuda"), torch.ones(n, device="cuda")
    want, _ = product64(q, w8[None], offs, rows)
    within(msb.matmul_int8(q, one, w8, ones, rows=rows, out_dtype=torch.float32), want, F32 * want.abs())
    within(msb.matmul_int8(q, one, w8, ones, rows=rows), want, (BF16 + F32) * want.abs())


@pytest.mark.parametrize("counts", [[600, 0, 513, 257, 1300], [2670], [256, 512, 33, 700, 300, 1024, 1, 640]])
def test_large_groups(msb, counts):
    """Groups of several pieces and of two accumulators, enough of them for the largest tiles: each
    kind of product, in order and gathered.  Tolerances as above."""
    import torch
    k, T, E, R = 136, 900, len(counts), sum(counts)
    offs = offsets_of(counts)
    rows = torch.randint(-1, T + 1, (R,), device="cuda", dtype=torch.int32)
    xs, xg = rnd(70, R, k), rnd(71, T, k)
    for x, idx in ((xs, None), (xg, rows)):
        for layout in ("k", "records"):
            n = 4104
            w = weight(72, E, n, k, layout)
            want, mag = product64(x, w, offs, idx)
            within(msb.grouped_matmul(x, w, offs, rows=idx), want, BF16 * want.abs() + k * 2 * F32 * mag + TINY, layout)
        n = 2072
        w = weight(73, 2 * E, n, k, "k").unflatten(0, (E, 2))
        (g, ga), (u, ua) = (product64(x, w[:, p], offs, idx) for p in range(2))
        dg, du, sg = k * 2 * F32 * ga, k * 2 * F32 * ua, torch.nn.functional.silu(g)
        tol = (BF16 + 2.0 ** -20) * (sg * u).abs() + 1.1 * dg * u.abs() + sg.abs() * du + 1.1 * dg * du + TINY
        within(msb.grouped_swiglu(x, w, offs, rows=idx), sg * u, tol + 2.0 ** -117 * u.abs(), "swiglu")
        n = 4104
        q, qs = msb.quantize_int8(x)
        w8 = torch.randint(-127, 128, (E, n, 144), device="cuda").to(torch.int8)[..., :k]
        ws = rnd(74, E, n, dtype=torch.float32)
        want = product64(q, w8, offs, idx)[0]
        if idx is None:
            want = want * qs.double()[:, None]
        else:
            ok = (idx >= 0) & (idx < T)
            want = want * torch.where(ok, qs[idx.long().clamp(0, T - 1)], 0.0).double()[:, None]
        for e, (lo, hi) in enumerate(zip(offs.tolist(), offs.tolist()[1:])):
            want[lo:hi] *= ws[e].double()
        for dtype, step in ((torch.bfloat16, BF16), (torch.float32, 0)):
            got = msb.matmul_int8(q, qs, w8, ws, offs, rows=idx, out_dtype=dtype)
            within(got, want, (step + 3.1 * F32) * want.abs() + TINY, ("int8", dtype))


def test_float_outputs_keep_float_precision(msb):
    """Float outputs at k = 8192: the sum is cut off every 256 k only, each time by less than 2^-23
    of a part's size per addition; relative L2 below 1e-6 (the bf16 output's rounding is 2e-3)."""
    import torch
    for layout in ("k", "n"):
        x, w = rnd(44, 500, 8192), weight(45, 1, 256, 8192, layout)
        want, _ = product64(x, w, offsets_of([500]), None)
        got = msb.grouped_matmul(x, w, out_dtype=torch.float32)
        assert (got.double() - want).norm() < 1e-6 * want.norm()


def whole(seed, *shape, most=2):
    """bf16 whole numbers -most .. most: sums of their products below 2^24 are exact in float32,
    in any order and however an addition is cut off."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(torch.bfloat16)


def long_weight(seed, lead, n, k, layout):
    """whole() of [*lead][n][k], k or n contiguous on a pitch of whole 16 bytes."""
    if layout == "k":
        return whole(seed, *lead, n, (k + 7) // 8 * 8)[..., :k]
    return whole(seed, *lead, k, (n + 7) // 8 * 8)[..., :n].transpose(-1, -2)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("R,n,k", [(128, 4096, 2048), (64, 8192, 4100), (129, 2500, 2090), (200, 1000, 20000),
                                   (3, 64, 20000), (17, 4100, 8192), (33, 9000, 4104), (128, 4096, 4104),
                                   (129, 2500, 4200), (40, 5000, 8200), (64, 2048, 2560)])
def test_shared_k_loses_nothing(msb, R, n, k, gather):
    """One weight whose tiles' k is shared by two or four pairs: whole numbers, exact sums (of 8-bit
    values in float64), so that a stage that is lost or counted twice shows in every output."""
    import torch
    T = 40
    rows = torch.randint(-1, T + 1, (R,), device="cuda", dtype=torch.int32) if gather else None
    offs = offsets_of([R])
    x = whole(92, T if gather else R, (k + 7) // 8 * 8)[:, :k]
    for layout in ("k", "n"):
        w = long_weight(93, (1,), n, k, layout)
        want, _ = product64(x, w, offs, rows)
        assert torch.equal(msb.grouped_matmul(x, w, rows=rows, out_dtype=torch.float32), want.float()), layout
        assert torch.equal(msb.grouped_matmul(x, w, rows=rows), want.bfloat16()), layout
    w = long_weight(94, (1, 2), n, k, "k").mul_(2.0 ** -6)  # gates of up to a few dozen
    (g, _), (u, _) = (product64(x, w[:, p], offs, rows) for p in range(2))
    want = torch.nn.functional.silu(g) * u
    # exact sums: the exponential and the quotient (2^-16 at most), one rounding
    within(msb.grouped_swiglu(x, w, rows=rows), want, (BF16 + 2.0 ** -16) * want.abs() + 2.0 ** -117 * u.abs() + TINY)
    gen = torch.Generator(device="cuda").manual_seed(89)
    eight = lambda *s: torch.randint(-128, 128, (*s, (k + 15) // 16 * 16), device="cuda", generator=gen).to(torch.int8)[..., :k]  # noqa: E731
    q, w8 = eight(T if gather else R), eight(2, n)
    one, ones = torch.ones(q.shape[0], device="cuda"), torch.ones(2, n, device="cuda")
    want, _ = product64(q, w8[:1], offs, rows)
    assert torch.equal(msb.matmul_int8(q, one, w8[0], ones[0], rows=rows, out_dtype=torch.float32), want.float())
    # bf16: of the sum's float
    assert torch.equal(msb.matmul_int8(q, one, w8[0], ones[0], rows=rows), want.float().bfloat16())
    up, _ = product64(q, w8[1:], offs, rows)
    scale = torch.full((2, n), 2.0 ** -18, device="cuda")  # gates of a few, exact but for the sums' float
    g, u = want * 2.0 ** -18, up * 2.0 ** -18
    h = torch.nn.functional.silu(g) * u
    tol = (BF16 + 2.0 ** -16) * h.abs() + 2.2 * F32 * g.abs() * u.abs() + 2.0 ** -117 * u.abs() + TINY
    within(msb.matmul_int8(q, one, w8, scale, rows=rows, swiglu=True), h, tol, "8-bit swiglu")


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,n,k", [([60, 0, 70], 300, 40000), ([100], 3000, 131136), ([100], 1500, 131136), ([70], 300, 140000)])
def test_long_sums_lose_nothing(msb, counts, n, k, gather):
    """k beyond one accumulator, with and without pairs that share it: sums of whole numbers come
    out exact, rounded once to bf16, so that no part of k is lost or counted twice."""
    import torch
    R, E, T = sum(counts), len(counts), 40
    offs = offsets_of(counts)
    rows = torch.randint(-1, T + 1, (R,), device="cuda", dtype=torch.int32) if gather else None
    x = whole(95, T if gather else R, k)
    for layout in ("k", "n"):
        w = long_weight(96, (E,), n, k, layout)
        want, _ = product64(x, w, offs, rows)
        assert torch.equal(msb.grouped_matmul(x, w, offs, rows=rows), want.bfloat16()), layout
    w = long_weight(97, (E, 2), n, k, "k") * 2.0 ** -8  # gates of up to a few dozen
    (g, _), (u, _) = (product64(x, w[:, p], offs, rows) for p in range(2))
    want = torch.nn.functional.silu(g) * u
    # exact sums: the exponential and the quotient (2^-16 at most), one rounding
    within(msb.grouped_swiglu(x, w, offs, rows=rows), want, (BF16 + 2.0 ** -16) * want.abs() + 2.0 ** -117 * u.abs() + TINY)


@pytest.mark.parametrize("counts,n,k", [([0, 100], 256, 1 << 18), ([100], 3000, 131136), ([64], 128, 1 << 20)])
def test_long_sums_are_not_cut_off(msb, counts, n, k):
    """Values of one sign, where every addition that is cut off errs the same way.  An accumulator's
    32768 k take 2048 additions of less than 2^-23 each: the mean relative error of bf16 outputs stays
    below 2.4e-4 (SwiGLU of large gates: twice that), plus the mean of N roundings of at most 2^-8
    each, 6 standard deviations: 6 2^-8 / sqrt(3 N)."""
    import torch
    R, E = sum(counts), len(counts)
    offs = offsets_of(counts)
    gen = torch.Generator(device="cuda").manual_seed(98)
    uni = lambda *s: torch.rand(*s, generator=gen, device="cuda")  # noqa: E731
    x = (uni(R, k) * (1 + torch.linspace(0, 1, R, device="cuda"))[:, None]).bfloat16()
    noise = 6 * BF16 / (3 * R * n) ** 0.5
    for layout in ("k", "n"):
        w = (uni(E, n, k) if layout == "k" else uni(E, k, n).transpose(1, 2)).bfloat16()
        want, _ = product64(x, w, offs, None)
        err = (msb.grouped_matmul(x, w, offs).double() - want) / want
        assert err.mean().abs() < 2.4e-4 + noise, (layout, float(err.mean()))
    if E == 2 or k >= 1 << 20:  # gate and up of the same values
        w2 = torch.stack([w.contiguous()] * 2, 1)
        x2 = x * 2.0 ** -9
        g, _ = product64(x2, w, offs, None)
        err = (msb.grouped_swiglu(x2, w2, offs).double() - g * g) / (g * g)
        assert err.mean().abs() < 4.8e-4 + noise, float(err.mean())


def test_swiglu_of_extreme_gates(msb):
    """Gates of +-300: silu is the gate itself and a zero of either sign, never NaN."""
    import torch
    x = torch.zeros((2, 8), device="cuda", dtype=torch.bfloat16)
    x[0, 0], x[1, 0] = 300.0, -300.0
    w = torch.zeros((1, 2, 3, 8), device="cuda", dtype=torch.bfloat16)
    w[0, :, :, 0] = 1.0
    h = msb.grouped_swiglu(x, w).float()
    assert torch.equal(h[0], torch.full((3,), 90112.0, device="cuda"))  # 300^2 = 90000 in bf16
    assert torch.equal(h[1], torch.zeros(3, device="cuda"))


@pytest.mark.parametrize("R", [1, 40])
def test_swiglu_over_the_range_of_gates(msb, R):
    """Gates of -87 to 87 in quarters, exact: the exponential is within (2 + 1.173 |g|) 2^-23, its sum
    with 1, the quotient and the product add 3 2^-23; one rounding to bf16."""
    import torch
    g = torch.arange(-348, 349, device="cuda") / 4.0
    n = g.numel()
    x = torch.ones((R, 8), device="cuda", dtype=torch.bfloat16)
    w = torch.zeros((1, 2, n, 8), device="cuda", dtype=torch.bfloat16)
    w[0, 0, :, 0], w[0, 0, :, 1] = g.floor().bfloat16(), (g - g.floor()).bfloat16()
    w[0, 1, :, 2] = 2.0 ** 20
    want = torch.nn.functional.silu(g.double()).expand(R, n) * 2.0 ** 20
    tol = (BF16 + (5 + 1.173 * g.double().abs()) * 2 * F32) * want.abs()
    within(msb.grouped_swiglu(x, w), want, tol)


@pytest.mark.parametrize("R", [1, 2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("k", [8, 33, 520, 2056, 4100])
def test_few_rows(msb, R, k):
    """Single tokens: rows of several groups and of one, indices outside x among them."""
    import torch
    n, T = 71, 5
    x = rnd(50, T, (k + 7) // 8 * 8)[:, :k]
    rows = torch.randint(-1, T + 1, (R,), device="cuda", dtype=torch.int32)
    for counts in ([R], [0, R // 2, 0, R - R // 2, 0]):
        offs, E = offsets_of(counts), len(counts)
        w = weight(51, 2 * E, n, k, "k").unflatten(0, (E, 2))
        want, mag = product64(x, w[:, 0], offs, rows)
        for dtype, step in ((torch.bfloat16, BF16), (torch.float32, F32)):
            got = msb.grouped_matmul(x, w[:, 0], offs, rows=rows, out_dtype=dtype)
            within(got, want, step * want.abs() + k * 2 * F32 * mag + TINY, dtype)
        u, ua = product64(x, w[:, 1], offs, rows)
        s = torch.nn.functional.silu(want)
        dg, du = k * 2 * F32 * mag, k * 2 * F32 * ua
        tol = (BF16 + 2.0 ** -20) * (s * u).abs() + 1.1 * dg * u.abs() + s.abs() * du + 1.1 * dg * du + TINY
        within(msb.grouped_swiglu(x, w, offs, rows=rows), s * u, tol + 2.0 ** -117 * u.abs(), "swiglu")
        q, qs = msb.quantize_int8(x)
        w8 = torch.randint(-127, 128, (E, n, (k + 15) // 16 * 16), device="cuda").to(torch.int8)[..., :k]
        ws = rnd(52, E, n, dtype=torch.float32)
        want = product64(q, w8, offs, rows)[0]
        ok = (rows >= 0) & (rows < T)
        want = want * torch.where(ok, qs[rows.long().clamp(0, T - 1)], 0.0).double()[:, None]
        for e, (lo, hi) in enumerate(zip(offs.tolist(), offs.tolist()[1:])):
            want[lo:hi] *= ws[e].double()
        within(msb.matmul_int8(q, qs, w8, ws, offs, rows=rows), want, (BF16 + 3.1 * F32) * want.abs() + TINY, "int8")


def test_rows_of_no_group_and_bad_indices(msb):
    """Rows before the first offset, behind the last and spare rows of out stay as they were; a
    row index outside x reads zeros; offsets out of order or out of range touch nothing else."""
    import torch
    k, n = 128, 96
    x, w = rnd(5, 40, k), rnd(6, 3, n, k)
    offs = offsets_of([5, 0, 20], first=7)
    rows = torch.arange(40, device="cuda", dtype=torch.int32)
    rows[9], rows[12], rows[13] = -1, 40, 2 ** 31 - 1
    out = torch.full((50, n), 7.0, device="cuda", dtype=torch.bfloat16)
    msb.grouped_matmul(x, w, offs, rows=rows, out=out)
    want, mag = product64(x, w, offs, rows)
    within(out[7:32], want[7:32], BF16 * want[7:32].abs() + k * 2 * F32 * mag[7:32])
    assert (out[:7] == 7).all() and (out[32:] == 7).all()
    assert (out[9] == 0).all() and (out[12] == 0).all() and (out[13] == 0).all()
    for bad in ([-5, 3, 2, 1000], [2 ** 31 - 1, 0, -2 ** 31, 4], [40, 30, 20, 10]):
        for R in (40, 6):
            out.fill_(7.0)
            msb.grouped_matmul(x, w, torch.tensor(bad, dtype=torch.int32, device="cuda"), rows=rows[:R], out=out)
            assert (out[R:] == 7).all()


def test_wide_pitches_and_strided_views(msb):
    """x, out and the weights as column slices of wider buffers: nothing outside is read into the
    result (the rest is NaN) or written."""
    import torch
    k, n, R = 72, 40, 70
    xb = torch.full((R, 128), float("nan"), device="cuda", dtype=torch.bfloat16)
    wb = torch.full((2, n, 128), float("nan"), device="cuda", dtype=torch.bfloat16)
    x, w = xb[:, 16:16 + k], wb[:, :, 8:8 + k]
    x.copy_(rnd(7, R, k)), w.copy_(rnd(8, 2, n, k))
    offs = offsets_of([33, 37])
    want, mag = product64(x, w, offs, None)
    for dtype, step in ((torch.bfloat16, BF16), (torch.float32, F32)):
        ob = torch.full((R, 60), 5.0, device="cuda", dtype=dtype)
        msb.grouped_matmul(x, w, offs, out=ob[:, 3:3 + n])
        within(ob[:, 3:3 + n], want, step * want.abs() + k * 2 * F32 * mag)
        assert (ob[:, :3] == 5).all() and (ob[:, 3 + n:] == 5).all()


def test_inner_length_of_one(msb):
    """k = 1: either dimension of the weight may be the contiguous one."""
    import torch
    x = rnd(60, 20, 8)[:, :1]
    for w in (rnd(61, 1, 24, 8)[:, :, :1], rnd(62, 1, 24, 1), rnd(63, 1, 1, 24).transpose(1, 2)):
        want = x.double() @ w[0].double().t()
        within(msb.grouped_matmul(x, w), want, (BF16 + F32) * want.abs() + TINY)


def test_nothing_to_do(msb):
    """Calls of no tokens or rows return empty tensors."""
    import torch
    w = synth.TINY
    layer = device_layer(w, rank=0)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    none = torch.empty((0, w.d), **bf)
    assert msb.moe_dense_block(none, layer).shape == (0, w.d)
    assert msb.moe_dense_block(none, msb.Int8Layer.from_packed(layer)).shape == (0, w.d)
    q, s = msb.quantize_int8(none)
    assert q.shape == (0, w.d) and s.shape == (0,)
    assert msb.linear_int8(none, torch.ones(8, w.d, device="cuda", dtype=torch.int8), torch.ones(8, device="cuda")).shape == (0, 8)
    assert msb.grouped_matmul(none, torch.ones((8, w.d), **bf)).shape == (0, 8)
    r = msb.route(torch.empty((0, 8), device="cuda"), 2)
    assert (r.offsets == 0).all()
    assert msb.combine(none, r).shape == (0, w.d)
    h, x = msb.block_norm(none, none)
    assert x.shape == (0, w.d)


def test_many_groups(msb):
    """512 groups, most of them empty."""
    import torch
    rng = np.random.default_rng(1)
    c = np.where(rng.random(512) < 0.1, rng.integers(1, 40, 512), 0)
    offs, k, n = offsets_of(c), 64, 130
    x, w = rnd(9, int(c.sum()), k), rnd(10, 512, n, k)
    want, mag = product64(x, w, offs, None)
    within(msb.grouped_matmul(x, w, offs), want, BF16 * want.abs() + k * 2 * F32 * mag)


def test_output_offsets_pass_32_bits(msb):
    """Rows of out on a pitch of 2^26 elements: the last starts 2^32 elements in."""
    import torch
    x, w = rnd(11, 65, 64), rnd(12, 1, 8, 64)
    out = torch.empty((65, 1 << 26), device="cuda", dtype=torch.bfloat16)[:, :8]
    out.fill_(0)
    msb.grouped_matmul(x, w, out=out)
    want, mag = product64(x, w, offsets_of([65]), None)
    within(out, want, BF16 * want.abs() + 64 * 2 * F32 * mag)


# ------------------------------------------------------------------ 8 bits

@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("R,k", [(1, 1), (3, 17), (70, 256), (5, 5000), (2, 20000), (1300, 1032), (1201, 2048),
                                 (1185, 4096)])
def test_quantize_int8(msb, R, k, dtype):
    """Bit for bit the stated float32 steps."""
    import torch
    x = rnd(13, R, k, scale=3.0, dtype=getattr(torch, dtype))
    x[0, 0] = 0
    q, s = msb.quantize_int8(x)
    # numpy's float32 quotient is the rounded one (torch multiplies by a rounded reciprocal)
    xf = x.float().cpu().numpy()
    big = np.abs(xf).max(1)
    live = big >= np.float32(2.0 ** -119)
    safe = np.where(live, big, np.float32(1))
    np.testing.assert_array_equal(s.cpu().numpy(), np.where(live, safe / np.float32(127), np.float32(0)))
    inv = np.where(live, np.float32(127) / safe, np.float32(0))
    np.testing.assert_array_equal(q.cpu().numpy(), np.rint(xf * inv[:, None]).astype(np.int8))


def test_quantize_special_rows(msb):
    import torch
    x = torch.zeros((6, 40), device="cuda")
    x[1, 3] = float("inf")
    x[2, 39] = float("nan")
    x[3, 0] = 1e-38
    x[4, 7] = -3e38
    x[5, :] = 2.0 ** -119
    q, s = msb.quantize_int8(x)
    assert (q[:4] == 0).all() and q[4, 7] == -127 and (q[5] == 127).all()
    assert s[0] == 0 and s[3] == 0 and torch.isnan(s[1]) and torch.isnan(s[2])
    w = torch.ones((1, 8, 48), device="cuda", dtype=torch.int8)[:, :, :40]
    y = msb.matmul_int8(q, s, w, torch.ones((1, 8), device="cuda"))
    assert torch.isnan(y[1:3].float()).all() and (y[0] == 0).all() and (y[3] == 0).all()


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("n,k", [(1, 16), (7, 33), (257, 200), (300, 1040)])
def test_matmul_int8(msb, counts, n, k):
    """The sum is exact; float32 of it and two products: 3 x 2^-24, and the output's rounding."""
    import torch
    c = COUNTS[counts]
    offs, R = offsets_of(c), sum(c)
    g = torch.Generator(device="cuda").manual_seed(14)
    q = torch.randint(-128, 128, (R, (k + 15) // 16 * 16), device="cuda", generator=g).to(torch.int8)[:, :k]
    w = torch.randint(-128, 128, (len(c), n, (k + 15) // 16 * 16), device="cuda", generator=g).to(torch.int8)[:, :, :k]
    qs, ws = rnd(15, R, dtype=torch.float32).abs(), rnd(16, len(c), n, dtype=torch.float32)
    want, _ = product64(q, w, offs, None)
    for e, (lo, hi) in enumerate(zip(offs.tolist(), offs.tolist()[1:])):
        want[lo:hi] *= ws[e].double()
    want *= qs.double()[:, None]
    for dtype, step in ((torch.bfloat16, BF16), (torch.float32, 0)):
        got = msb.matmul_int8(q, qs, w, ws, offs, out_dtype=dtype)
        within(got, want, (step + 3.1 * F32) * want.abs() + TINY, dtype)


def test_matmul_int8_largest_sums(msb):
    """k = 131056 products of -128 x -128: the sum 2147221504 is below 2^31 and exact."""
    import torch
    k = 131056
    q = torch.full((2, k), -128, device="cuda", dtype=torch.int8)
    q[1] = 127
    w = torch.full((1, 3, k), -128, device="cuda", dtype=torch.int8)
    one = torch.ones(2, device="cuda")
    y = msb.matmul_int8(q, one, w, torch.ones((1, 3), device="cuda"), out_dtype=torch.float32)
    want = torch.tensor([128 * 128 * k, -127 * 128 * k], device="cuda", dtype=torch.float64)[:, None].expand(2, 3)
    within(y, want, F32 * want.abs())


@pytest.mark.parametrize("n,k", [(33, 64), (200, 1024)])
def test_swiglu_int8(msb, n, k):
    """As the bf16 form with the sums' errors 3 x 2^-24 of the scaled sum."""
    import torch
    c = COUNTS["skew"]
    offs, R, T = offsets_of(c), sum(c), 90
    x = rnd(17, T, k)
    w = torch.randint(-127, 128, (len(c), 2, n, k), device="cuda").to(torch.int8)
    ws = rnd(18, len(c), 2, n, dtype=torch.float32).abs() * 1e-3
    rows = torch.randint(0, T, (R,), device="cuda", dtype=torch.int32)
    q, qs = msb.quantize_int8(x)
    # the integer sums are exact in 64 bits (a sum of zero stays zero); then the scales
    group = torch.repeat_interleave(torch.arange(len(c), device="cuda"), torch.tensor(c, device="cuda"))
    g, u = (product64(q, w[:, p], offs, rows)[0] * qs.double()[rows.long(), None] * ws[group, p].double()
            for p in range(2))
    s = torch.nn.functional.silu(g)
    dg, du = 3.1 * F32 * g.abs(), 3.1 * F32 * u.abs()
    tol = (BF16 + 2.0 ** -20) * (s * u).abs() + 1.1 * dg * u.abs() + s.abs() * du + TINY
    got = msb.swiglu_int8(x, w, ws, offs, rows=rows)
    within(got, s * u, tol)
    assert torch.equal(got, msb.matmul_int8(q, qs, w, ws, offs, rows=rows, swiglu=True))


@pytest.mark.parametrize("R", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("k", [16, 33, 1023, 1032, 2048, 4096])
@pytest.mark.parametrize("f32,lead,pitch", [(False, 0, 0), (True, 0, 8), (False, 1, 8), (True, 3, 5)])
def test_linear_int8_is_quantize_and_matmul(msb, R, k, f32, lead, pitch):
    """The same bits, whichever kernel rounds x; strided and unaligned rows in a buffer of NaN, a
    row of zeros, one with a NaN."""
    import torch
    dtype = torch.float32 if f32 else torch.bfloat16
    buf = torch.full((lead + R * (k + pitch),), float("nan"), device="cuda", dtype=dtype)
    x = buf[lead:].view(R, k + pitch)[:, :k]
    x.copy_(rnd(27, R, k, dtype=dtype))
    if R > 3:
        x[2] = 0
        x[3, k // 2] = float("nan")
    n, E = 37, 5
    q, qs = msb.quantize_int8(x)
    w = torch.randint(-128, 128, (E, 2, n, (k + 15) // 16 * 16), device="cuda").to(torch.int8)[..., :k]
    ws = rnd(28, E, 2, n, dtype=torch.float32).abs() * 1e-3
    same = lambda a, b: torch.equal(a, b) or torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())  # noqa: E731
    for o in (torch.bfloat16, torch.float32):
        assert same(msb.linear_int8(x, w[1, 0], ws[1, 0], out_dtype=o), msb.matmul_int8(q, qs, w[1, 0], ws[1, 0], out_dtype=o))
    # grouped: a group of none, rows taken twice, one outside x
    rows = torch.arange(6, device="cuda", dtype=torch.int32) % R
    rows[4] = R
    offs = torch.tensor([0, 1, 1, 4, 5, 6], device="cuda", dtype=torch.int32)
    assert same(msb.linear_int8(x, w[:, 0], ws[:, 0].contiguous(), offs, rows=rows),
                msb.matmul_int8(q, qs, w[:, 0], ws[:, 0].contiguous(), offs, rows=rows))
    assert same(msb.swiglu_int8(x, w, ws, offs, rows=rows),
                msb.matmul_int8(q, qs, w, ws, offs, rows=rows, swiglu=True))


@pytest.mark.parametrize("R", [2, 700])
def test_linear_int8_with_scratch_of_the_caller(msb, R):
    """out and workspace given: the same bits, on a raw stream handle too; nothing behind the
    workspace is written; one that is too small is refused."""
    import torch
    n, k, E = 96, 520, 3
    x = rnd(90, R, k)
    w = torch.randint(-127, 128, (E, 2, n, 528), device="cuda").to(torch.int8)[..., :k]
    ws = rnd(91, E, 2, n, dtype=torch.float32).abs() * 1e-3
    rows = torch.arange(R, device="cuda", dtype=torch.int32)
    offs = offsets_of([R // 2, 0, R - R // 2])
    need = msb.load_library().msb_int8_linear_workspace_size(R, k)
    buf = torch.full((need + 64,), 7, device="cuda", dtype=torch.uint8)
    side = torch.cuda.Stream()
    for f, at, kw in ((msb.linear_int8, (w[1, 0], ws[1, 0]), {}), (msb.swiglu_int8, (w, ws, offs), dict(rows=rows))):
        want = f(x, *at, **kw)
        out = torch.zeros_like(want)
        torch.cuda.synchronize()
        for stream in (None, side, side.cuda_stream):
            out.zero_()
            torch.cuda.synchronize()
            assert f(x, *at, out=out, workspace=buf[:need], stream=stream, **kw) is out
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        assert (buf[need:] == 7).all()
        with pytest.raises(msb.MsbError):
            f(x, *at, out=out, workspace=buf[:need - 1], **kw)
        with pytest.raises(ValueError):
            f(x, *at, out=out, stream=side.cuda_stream, **kw)
        with pytest.raises(ValueError):
            f(x, *at, out=out, workspace=torch.zeros(need, dtype=torch.uint8), **kw)


# ------------------------------------------------------------------ routing

def route_ref(l, top_e, renorm, mask):
    """Plain loops over float64 logits."""
    T, E = l.shape
    ids, wts = -np.ones((T, top_e), np.int64), np.zeros((T, top_e))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        v = np.minimum(l[t], np.float64(np.finfo(np.float32).max))
        cand = [e for e in range(E) if v[e] > -np.inf]
        best = sorted(cand, key=lambda e: (-v[e], e))[:top_e]
        if not best:
            continue
        p = np.exp(v - v[best[0]])
        den = p[best].sum() if renorm else p[cand].sum()
        ids[t, :len(best)], wts[t, :len(best)] = best, p[best] / den
    pairs = sorted((ids[t, k], t, k) for t in range(T) for k in range(top_e) if ids[t, k] >= 0)
    rows, pos = -np.ones(T * top_e, np.int64), -np.ones((T, top_e), np.int64)
    for p, (e, t, k) in enumerate(pairs):
        rows[p], pos[t, k] = t, p
    counts = np.bincount([e for e, _, _ in pairs], minlength=E) if pairs else np.zeros(E, np.int64)
    return ids, wts, np.concatenate([[0], np.cumsum(counts)]), rows, pos


@pytest.mark.parametrize("T", [0, 1, 33, 64, 65, 700])
@pytest.mark.parametrize("E,K", [(1, 1), (8, 2), (60, 4), (128, 8), (300, 16), (512, 16)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(msb, T, E, K, renorm):
    """Ids and plan exact (logits on a coarse grid: many ties); weights: the difference, the
    exponential (2 ulp), the sum and the quotient: (E + 8) 2^-24 is a bound, |l - max| 2^-24 more
    from the rounded difference (below 10 here)."""
    import torch
    rng = np.random.default_rng(T + E)
    l = np.round(rng.standard_normal((T, E)) * 4) / 4
    if T > 8:
        l[1], l[2, 1:], l[3, ::2], l[4, 0] = -np.inf, -np.inf, np.nan, np.inf
        l[5, :], l[6, 0] = np.inf, -np.finfo(np.float32).max
    mask = rng.random(T) < 0.8 if T % 2 else None
    for dtype in (torch.float32, torch.bfloat16):
        lt = torch.tensor(l, device="cuda").to(dtype)
        mt = None if mask is None else torch.tensor(mask, device="cuda")
        got = msb.route(lt, K, renorm=renorm, mask=mt)
        with np.errstate(all="ignore"):
            ids, wts, offs, rows, pos = route_ref(lt.double().cpu().numpy(), K, renorm, mask)
        for a, b in ((got.ids, ids), (got.offsets, offs), (got.rows, rows), (got.pos, pos)):
            np.testing.assert_array_equal(a.cpu().numpy(), b)
        np.testing.assert_allclose(got.weights.cpu().numpy(), wts, rtol=(E + 20) * F32, atol=1e-38)


def test_route_many_tokens(msb):
    """More pairs per block than one chunk holds; strided logits."""
    import torch
    T, E, K = 70000, 24, 16
    l = rnd(19, T, 40, dtype=torch.float32)[:, 3:3 + E]
    got = msb.route(l, K)
    ids = torch.argsort(l, dim=1, descending=True, stable=True)[:, :K]
    assert torch.equal(got.ids.long(), ids)
    order = torch.argsort(ids.reshape(-1), stable=True)
    assert torch.equal(got.rows.long(), order // K)
    assert torch.equal(got.pos.reshape(-1)[order].long(), torch.arange(T * K, device="cuda"))
    assert torch.equal(got.offsets[1:].long(), torch.cumsum(torch.bincount(ids.reshape(-1), minlength=E), 0))


@pytest.mark.parametrize("d", [1, 100, 2048])
def test_combine(msb, d):
    """K products and sums in float32: (K + 1) 2^-24 of the sum of magnitudes, one rounding."""
    import torch
    T, K, R = 37, 5, 120
    pos = torch.randint(-1, R, (T, K), device="cuda", dtype=torch.int32)
    pos[3], pos[4, 0], pos[5, 1] = -1, R, 2 ** 31 - 1
    w = rnd(20, T, K, dtype=torch.float32)
    r = msb.Routing(None, w, None, None, pos)
    for dtype in (torch.bfloat16, torch.float32):
        y = rnd(21, R, d + 3, dtype=dtype)[:, :d]
        ok = ((pos >= 0) & (pos < R))
        terms = torch.where(ok, w, 0.0).double()[..., None] * y.double()[pos.long().clamp(0, R - 1)]
        want = terms.sum(1)
        got = msb.combine(y, r)
        within(got, want, BF16 * want.abs() + (K + 1) * F32 * terms.abs().sum(1) + TINY)
        assert (got[3] == 0).all()


@pytest.mark.parametrize("T,K", [(1185, 1), (2369, 2), (1191, 3), (1300, 4), (1201, 5), (1184, 9), (2400, 16)])
@pytest.mark.parametrize("d", [8, 2056])
def test_combine_many_tokens(msb, T, K, d):
    """Blocks that take several tokens: as test_combine, pitches wider than the rows, rows left out."""
    import torch
    R = 500
    pos = torch.randint(-1, R + 1, (T, K), device="cuda", dtype=torch.int32)
    w = rnd(29, T, K, dtype=torch.float32)
    r = msb.Routing(None, w, None, None, pos)
    ok = (pos >= 0) & (pos < R)
    for dtype in (torch.bfloat16, torch.float32):
        y = rnd(30, R, d + 8, dtype=dtype)[:, :d]
        want, mag = torch.zeros(T, d, device="cuda", dtype=torch.float64), torch.zeros(T, d, device="cuda", dtype=torch.float64)
        for k in range(K):
            term = torch.where(ok[:, k], w[:, k], 0.0).double()[:, None] * y.double()[pos[:, k].long().clamp(0, R - 1)]
            want += term
            mag += term.abs()
        out = torch.full((T + 1, d + 16), 3.0, device="cuda", dtype=torch.bfloat16)
        got = msb.combine(y, r, out=out[:T, :d])
        within(got, want, BF16 * want.abs() + (K + 1) * F32 * mag + TINY)
        assert (out[T] == 3).all() and (out[:, d:] == 3).all()


def test_longest_rows(msb):
    """Rows of 2^28 - 1 (and - 8) elements, the longest that are taken: bit for bit."""
    import torch
    d = (1 << 28) - 8
    y = rnd(88, 2, d)
    w = torch.tensor([[0.5, 2.0]], device="cuda")
    r = msb.Routing(None, w, None, None, torch.tensor([[1, 0]], device="cuda", dtype=torch.int32))
    got = msb.combine(y, r)
    # powers of two: the products are exact, the sum is rounded once to float and once to bf16
    assert torch.equal(got[0], (0.5 * y[1].float() + 2.0 * y[0].float()).bfloat16())
    k = (1 << 28) - 1
    x = y.view(-1)[:k].view(1, k)
    x[0, 5] = 16.0  # the maximum: 127 / 16 is exact
    q, s = msb.quantize_int8(x)
    assert abs(float(s[0]) - 16.0 / 127.0) <= F32 * 16.0 / 127.0
    assert torch.equal(q[0], torch.round(x[0].float() * (127.0 / 16.0)).to(torch.int8))


# ------------------------------------------------------------------ block norm

@pytest.mark.parametrize("R,d", [(1, 1), (4, 64), (3, 433), (70, 1000), (5, 2048), (9, 4096), (2, 8192), (2, 16384)])
@pytest.mark.parametrize("h32,y32", [(True, False), (False, False), (True, True)])
@pytest.mark.parametrize("gate", [None, "channel", "token", "full", "row"])
def test_block_norm(msb, R, d, h32, y32, gate):
    """Float32 steps: the mean of squares within (d + 2) 2^-24 relative (half of that after the
    root), a dozen roundings more; h' besides by those of its terms' magnitudes; one rounding of
    each output."""
    import torch
    t = lambda f: torch.float32 if f else torch.bfloat16  # noqa: E731
    h, y = rnd(22, R, d + 8, scale=4.0, dtype=t(h32))[:, :d], rnd(23, R, d, dtype=t(y32))
    shape = {None: None, "channel": (d,), "token": (R, 1), "full": (R, d), "row": (1, d)}[gate]
    post = gate != "full"
    g = None if shape is None else rnd(24, *shape, dtype=t(gate == "token"))
    pre, pw = rnd(25, d, dtype=t(y32)), (rnd(26, d, dtype=t(y32)) if gate != "row" and post else None)
    rms = lambda v: v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    b = rms(y.double()) if post else y.double()
    b = b if pw is None else b * pw.double()
    b = b if g is None else b * g.double()
    hw = 0.5 * h.double() + 0.22 * b
    mag = 0.5 * h.double().abs() + 0.22 * b.abs()
    xw = rms(hw) * pre.double()
    h0 = h.clone()
    ho, x = msb.block_norm(h, y, h_out=torch.empty_like(h0), pre_weight=pre, post_norm=post, post_weight=pw,
                           gate=g, skip_scale=0.5, residual_scale=0.22)
    assert torch.equal(h, h0)
    eps = (d / 2 + 14) * F32
    within(ho, hw, (F32 if h32 else BF16) * hw.abs() + eps * mag, "h")
    # x: the norm sees h' off by eps mag; relative to the row's root mean square
    scale = (hw.square().mean(1, keepdim=True) + 1e-6).sqrt()
    far = eps * (mag / scale + 2 * xw.abs() / pre.double().abs().clamp(min=1e-30)
                 + (mag.square().mean(1, keepdim=True).sqrt() / scale) * rms(hw).abs()) * pre.double().abs()
    within(x, xw, BF16 * xw.abs() + far + TINY, "x")
    ho2, x2 = msb.block_norm(h, y, x=torch.empty_like(x), pre_weight=pre, post_norm=post, post_weight=pw, gate=g,
                             skip_scale=0.5, residual_scale=0.22)
    assert ho2 is h and torch.equal(h, ho) and torch.equal(x2, x)


@pytest.mark.parametrize("R,d", [(1183, 2048), (1184, 1032), (2500, 1536), (1500, 768), (1300, 264)])
@pytest.mark.parametrize("h32,y32", [(True, False), (False, False), (True, True), (False, True)])
def test_block_norm_many_rows(msb, R, d, h32, y32):
    """Row counts on both sides of the choice of threads, blocks that take several rows."""
    for gate in ("token", "full"):
        test_block_norm(msb, R, d, h32, y32, gate)


def test_block_norm_is_residual_rmsnorm(msb):
    """Without weights, gate and scales it is the decode stack's glue."""
    import torch
    h, y = rnd(27, 5, 2048, dtype=torch.float32), rnd(28, 5, 2048)
    h1, x1 = h.clone(), torch.empty_like(y)
    msb.residual_rmsnorm(h1, y, x1)
    h2, x2 = msb.block_norm(h.clone(), y)
    assert torch.equal(h1, h2)
    # the two kernels' sums run in different orders: a value may fall on the other side of a rounding
    within(x2, x1.double(), 2 * BF16 * x1.double().abs())
    h3, x3 = msb.block_norm(h.clone())
    assert torch.equal(h3, h)


def test_block_norm_special_rows(msb):
    """A row of zeros gives zeros, NaN and infinity stay in their row."""
    import torch
    h, y = rnd(29, 4, 300), rnd(30, 4, 300)
    h[0], y[0] = 0, 0
    y[1, 7], h[2, 9] = float("nan"), float("inf")
    ho, x = msb.block_norm(h, y, post_norm=True)
    assert (x[0] == 0).all() and (ho[0] == 0).all()
    assert torch.isnan(x[1].float()).all() and torch.isfinite(x[3].float()).all()
    assert torch.isinf(ho[2, 9].float()) and torch.isnan(x[2, 9].float()) and (x[2, :9] == 0).all()


@pytest.mark.parametrize("R,d", [(3, 40), (5, 33), (4, 433), (3, 1000), (6, 1001), (3, 2048), (5, 4097), (1500, 264), (2, 16384)])
@pytest.mark.parametrize("h32", [True, False])
def test_block_norm_strided_gates(msb, R, d, h32):
    """A gate of any strides (transposed, every third column, one row or column of a matrix) gives
    the bits of its contiguous copy: the same steps on the same values.  What lies between is NaN."""
    import torch
    h, y = rnd(80, R, d, dtype=torch.float32 if h32 else None), rnd(81, R, d)
    pre, pw = rnd(82, d), rnd(83, d)

    def views(dtype):
        nan = lambda *s: torch.full(s, float("nan"), device="cuda", dtype=dtype)  # noqa: E731
        g = rnd(84, R, d, dtype=dtype)
        b = nan(d, R + 3)
        yield "transposed", g, b[:, 1:R + 1].t()
        b = nan(R, 3 * d + 5)
        yield "every third", g, b[:, 2:2 + 3 * d:3]
        yield "one row", g[:1], nan(d, 7)[:, 2:3].t()
        yield "channel", g[0], nan(d, 5)[:, 3]
        yield "token", g[:, :1], nan(R, 9)[:, 4:5]

    for dtype in (torch.bfloat16, torch.float32):
        for name, g, v in views(dtype):
            v.copy_(g)
            kw = dict(pre_weight=pre, post_norm=True, post_weight=pw, skip_scale=0.5, residual_scale=0.22)
            want = msb.block_norm(h, y, h_out=torch.empty_like(h), gate=g.contiguous(), **kw)
            got = msb.block_norm(h, y, h_out=torch.empty_like(h), gate=v, **kw)
            assert torch.isfinite(want[0]).all()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (name, dtype)


@pytest.mark.parametrize("d,stride", [(33, 1 << 26), (513, 1 << 23)])
def test_block_norm_gate_columns_far_apart(msb, d, stride):
    """Columns of a transposed gate 2^23 and 2^26 elements apart: their offsets pass 32 bits."""
    import torch
    R = 2
    buf = torch.empty((d, stride), device="cuda", dtype=torch.bfloat16)
    gate = buf.t()[:R]
    g = rnd(85, R, d)
    gate.copy_(g)
    h, y = rnd(86, R, d), rnd(87, R, d)
    want = msb.block_norm(h, y, h_out=torch.empty_like(h), gate=g)
    got = msb.block_norm(h, y, h_out=torch.empty_like(h), gate=gate)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ the block

@pytest.mark.parametrize("tokens", [1, 3, 300])
def test_dense_block_against_the_oracle(msb, tokens):
    """moe_dense_block against the oracle's dense block on sampled tokens.  Three roundings to
    bf16 along the way (h, the experts' rows, the output), each 2^-8 at most: 2e-2 relative L2 as
    for the decode block is far outside."""
    w = synth.TINY
    lw = synth.layer_weights(w)
    lay = oracle.ArrayLayer(lw.gate, lw.up, lw.down, lw.router, lw.lr_a, lw.lr_b)
    layer = device_layer(w)
    xb = synth.activations(w, 3, batch=tokens)
    y = msb.moe_dense_block(to_bf16_tensor(xb), layer)
    got = oracle.bf16_to_f64(from_bf16_tensor(y))
    for t in sorted({0, tokens // 2, tokens - 1}):
        ref = oracle.moe_block(xb[t:t + 1], lay, w.top_e, w.inter, rank=0, mode="dense")["y"][0]
        rel = np.linalg.norm(got[t] - ref) / np.linalg.norm(ref)
        assert rel < 2e-2, (t, rel)


@pytest.mark.parametrize("workload,tokens", [(synth.TINY, 4), (synth.QWEN30B_BLOCK, 16), (synth.QWEN30B_BLOCK, 256)])
def test_dense_block_is_the_decode_block(msb, workload, tokens):
    """The same tokens through moe_sparse_block with k = I and rank 0: each side within the
    roundings above of the same value (a token whose K-th and next logit are equal to float32
    accuracy may route differently: none of these)."""
    w = workload
    layer = device_layer(w, rank=0)
    x = to_bf16_tensor(synth.activations(w, 5, batch=tokens))
    a = msb.moe_dense_block(x, layer).double()
    b = msb.moe_sparse_block(x, layer, w.inter).double()
    rel = (a - b).norm(dim=1) / b.norm(dim=1)
    assert rel.max() < 2e-2, rel.max()


def test_dense_block_padded_and_int8(msb):
    """A padded batch gives each prompt what it gives alone, and zeros for the padding; the 8-bit
    layer stays within the 8-bit error: each of the two products' operands is off by at most half
    a step of its row's maximum, 1/254, against typical values of a third of it."""
    import torch
    w = synth.QWEN30B_BLOCK
    layer = device_layer(w, rank=0)
    x = to_bf16_tensor(synth.activations(w, 6, batch=120))
    mask = torch.arange(120, device="cuda") % 60 < 47
    alone = torch.cat([msb.moe_dense_block(x[i:i + 47].contiguous(), layer) for i in (0, 60)])
    both = msb.moe_dense_block(x, layer, mask=mask)
    # other group sizes, same sums: the products' order along k does not depend on them
    assert torch.equal(both[mask], alone)
    assert (both[~mask] == 0).all()
    y8 = msb.moe_dense_block(x, msb.Int8Layer.from_packed(layer), mask=mask)
    rel = (y8.double() - both.double())[mask].norm() / both.double()[mask].norm()
    assert rel < 0.05, rel
    assert (y8[~mask] == 0).all()


@pytest.mark.parametrize("tokens", [1, 2, 9])
def test_dense_block_int8_is_its_parts(msb, tokens):
    """The 8-bit block bit for bit as its operators one after the other, eager and replayed."""
    import torch
    w = synth.QWEN30B_BLOCK
    layer = msb.Int8Layer.from_packed(device_layer(w, rank=0))
    x = to_bf16_tensor(synth.activations(w, 7, batch=tokens))
    router = layer.router_t.view(torch.bfloat16).view(w.experts, w.d)
    r = msb.route(msb.grouped_matmul(x, router, out_dtype=torch.float32), w.top_e, renorm=bool(layer.dims.renorm))
    h = msb.swiglu_int8(x, layer.gate_up, layer.gate_up_scale, r.offsets, rows=r.rows)
    y = msb.linear_int8(h, layer.down[..., :w.inter], layer.down_scale, r.offsets)
    want = msb.combine(y, r)
    assert torch.equal(msb.moe_dense_block(x, layer), want)
    out, space = torch.empty_like(x), msb.DenseWorkspace(layer.dims, tokens, int8=True)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        msb.moe_dense_block(x, layer, out=out, workspace=space)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    msb.dense_check()


def test_prompt_step_with_norms_captured(msb):
    """Two layers of a stack, block_norm around moe_dense_block, as a user runs them: eager and
    replayed from a graph on another stream, the same bits; a second graph beside it does not
    disturb the first."""
    import torch
    w = synth.TINY
    layer = device_layer(w, rank=0)
    T = 77
    hs = [rnd(31 + i, T, w.d, dtype=torch.float32) for i in range(2)]
    pre, post = rnd(33, w.d), rnd(34, w.d)

    def step(h, ws):
        h, x = msb.block_norm(h, None, h_out=torch.empty_like(h), pre_weight=pre)
        for _ in range(2):
            y = msb.moe_dense_block(x, layer, workspace=ws)
            h, x = msb.block_norm(h, y, h_out=torch.empty_like(h), pre_weight=pre, post_norm=True,
                                  post_weight=post, residual_scale=0.5)
        return h, x

    ws = [msb.DenseWorkspace(layer.dims, T) for _ in range(2)]
    want = [step(h, ws[0]) for h in hs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs, outs, ins = [], [], []
    for i in range(2):
        ins.append(torch.zeros_like(hs[i]))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(step(ins[i], ws[i]))
        graphs.append(g)
    for i in range(2):
        ins[i].copy_(hs[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for (h, x), (hw, xw) in zip(outs, want):
        assert torch.equal(h, hw) and torch.equal(x, xw)


def test_calls_on_another_stream(msb):
    """Outputs allocated for a call on another stream are ordered for it."""
    import torch
    w = synth.TINY
    layer = device_layer(w, rank=0)
    x = to_bf16_tensor(synth.activations(w, 9, batch=40))
    want = msb.moe_dense_block(x, layer)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = msb.moe_dense_block(x, layer, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    with pytest.raises(ValueError):
        msb.moe_dense_block(x, layer, stream=side.cuda_stream)


def test_repeatable(msb):
    """The same call twice gives the same bits."""
    import torch
    w = synth.QWEN30B_BLOCK
    layer = device_layer(w, rank=0)
    x = to_bf16_tensor(synth.activations(w, 10, batch=200))
    assert torch.equal(msb.moe_dense_block(x, layer), msb.moe_dense_block(x, layer))


def test_dense_block_ignores_rank(msb):
    """dims.rank does not matter to the dense block."""
    import torch
    w = synth.TINY
    x = to_bf16_tensor(synth.activations(w, 11, batch=9))
    a = msb.moe_dense_block(x, device_layer(w))
    b = msb.moe_dense_block(x, device_layer(w, rank=0))
    assert torch.equal(a, b)
