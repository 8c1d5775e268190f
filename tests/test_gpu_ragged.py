"""The products over ragged groups (bf16 forward, dgrad, wgrad; int8 forward) and the
int8 row quantiser against float64 on the device.

Tolerances, per element, S = sum of |a| |b| over the contraction: a product of two
bf16 values is exact in float32; the tensor cores add 16 products at a time to the
running sum and may cut off up to two units in its last place (2 * 2^-23 of at most S)
a step. A float32 result moves its sum to registers every 512 elements (32 steps) and
rounds there once a part (2^-24). The result's own rounding is half a step, 2^-8 of
the value for bf16 and 2^-24 for float32:
    |y - exact| <= half * |exact| + (2 * steps + parts) * 2^-23 * S,
steps = K / 16 for bf16, 32 for float32.
int8: sums are exact below 2^24; the scales' product and its product with the sum round
once each (2^-24): half * |exact| + 3 * 2^-24 * |exact|.
"""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8


@pytest.fixture(scope="module")
def mgq():
    from fp8_grouped_gemm_gb300 import mgq
    mgq.load()
    return mgq


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(BF)


def _bounds(counts, lead):
    b = [lead]
    for c in counts:
        b.append(b[-1] + c)
    return b


def _off(bounds):
    return torch.tensor(bounds, dtype=torch.int32, device="cuda")


def _tol(dt, ref, S, K):
    parts = math.ceil(K / 512)
    steps = 32 if dt is F32 else math.ceil(K / 16)
    half = 2.0 ** -24 if dt is F32 else 2.0 ** -8
    return half * ref.abs() + (2 * steps + parts) * 2.0 ** -23 * S + 1e-38


def _close(out, ref, tol, what):
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), out[bad][:4], ref[bad][:4])


# groups (sizes; a first row and rows behind the last group in `lead`, `tail`), N, K
SHAPES = [
    ([1], 0, 0, 8, 16),
    ([5, 0, 33, 1, 64, 17, 16], 3, 5, 264, 144),          # few rows: one small tile a group
    ([0, 0, 3], 0, 0, 136, 2064),                         # contraction split over a cluster, a ragged end
    ([64, 65, 63, 0, 128], 1, 2, 520, 528),               # either side of a token tile
    ([2] * 40, 0, 7, 128, 512),
    ([300] + [0] * 30, 0, 0, 256, 512),
    ([1300, 513, 0, 77, 256, 257], 9, 30, 2056, 656),     # the large form: tiles of 256 tokens, short last ones
    ([1024, 1025, 1023], 0, 1, 1544, 1040),
    ([31, 0, 700, 1900, 1], 2, 0, 1800, 136),
]
IDS = [str(i) for i in range(len(SHAPES))]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("op", ["fwd", "dgrad"])
def test_rows(mgq, op, shape, dt):
    counts, lead, tail, N, K = shape
    g = _gen(1)
    b = _bounds(counts, lead)
    R, E = b[-1] + tail, len(counts)
    M, C = (N, K) if op == "fwd" else (K, N)
    x, w = _randn(g, R, C), _randn(g, E, N, K)
    x[:lead] = float("nan")                               # rows of no group reach nothing
    x[b[-1]:] = float("inf")
    out = torch.full((R, M), 7.0, dtype=dt, device="cuda")
    (mgq.ragged_gemm_fwd if op == "fwd" else mgq.ragged_gemm_dgrad)(x, w, _off(b), out)
    assert mgq.get_error() == mgq.OK
    assert (out[:lead] == 7).all() and (out[b[-1]:] == 7).all()
    for e in range(E):
        r = slice(b[e], b[e + 1])
        we = w[e].double() if op == "dgrad" else w[e].double().t()
        ref, S = x[r].double() @ we, x[r].double().abs() @ we.abs()
        _close(out[r], ref, _tol(dt, ref, S, C), (op, e))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES + [([15, 1, 47, 48, 49, 64, 79, 0, 80, 129], 5, 3, 128, 264)],
                         ids=IDS + ["steps"])
def test_wgrad(mgq, shape, dt):
    counts, lead, tail, N, K = shape
    g = _gen(2)
    b = _bounds(counts, lead)
    R, E = b[-1] + tail, len(counts)
    dy, x = _randn(g, R, N), _randn(g, R, K)
    dw = torch.full((E, N, K), float("nan"), dtype=dt, device="cuda")      # beta 0 does not read it
    mgq.ragged_gemm_wgrad(dy, x, _off(b), dw)
    assert mgq.get_error() == mgq.OK
    for e in range(E):
        r = slice(b[e], b[e + 1])
        ref = dy[r].double().t() @ x[r].double()
        S = dy[r].double().abs().t() @ x[r].double().abs()
        _close(dw[e], ref, _tol(dt, ref, S, max(1, counts[e])), e)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("R,C,M", [(13, 14344, 520), (290, 4104, 5128), (1307, 4104, 2568)])
@pytest.mark.parametrize("op", ["fwd", "dgrad", "wgrad"])
def test_sums_of_one_sign(mgq, op, R, C, M, dt):
    """Operands of one sign, for which every bit that is cut off counts the same way. A step aligns its 16 products
    and the running sum to the largest of them, cuts each off two bits below its 24 (16 * 2^-25 of it) and the sum
    to 24 bits (2^-23): at most 5 * 2^-23 of the sum a step, float32 results 32 steps of a part of it and then a
    rounding for each part (2^-24)."""
    g = _gen(28)
    pos = lambda *s: (torch.rand(s, device="cuda", generator=g) + 1).to(BF)
    if op == "wgrad":                                     # contraction over C rows, R of them another group's
        a, c, out = pos(C + R, 264), pos(C + R, 136), torch.empty(2, 264, 136, dtype=dt, device="cuda")
        mgq.ragged_gemm_wgrad(a, c, _off([0, R, R + C]), out)
        out, ref = out[1], a[R:].double().t() @ c[R:].double()
    else:
        x, w = pos(R, C), pos(1, *((M, C) if op == "fwd" else (C, M)))
        out = torch.empty(R, M, dtype=dt, device="cuda")
        (mgq.ragged_gemm_fwd if op == "fwd" else mgq.ragged_gemm_dgrad)(x, w, None, out)
        ref = x.double() @ (w[0].double().t() if op == "fwd" else w[0].double())
    steps, parts = (32, math.ceil(C / 512)) if dt is F32 else (math.ceil(C / 16), 0)
    half = 2.0 ** -24 if dt is F32 else 2.0 ** -8
    _close(out, ref, (half + 5 * steps * 2.0 ** -23 + parts * 2.0 ** -24) * ref, op)


@pytest.mark.parametrize("beta", [1.0, 0.5, -2.0])
def test_wgrad_accumulates(mgq, beta):
    g = _gen(3)
    counts, N, K = [70, 0, 5, 260], 392, 264
    b = _bounds(counts, 0)
    dy, x = _randn(g, b[-1], N), _randn(g, b[-1], K)
    old = torch.randn(4, N, K, device="cuda", generator=g)
    dw = old.clone()
    mgq.ragged_gemm_wgrad(dy, x, _off(b), dw, beta=beta)
    for e in range(4):
        r = slice(b[e], b[e + 1])
        prod = dy[r].double().t() @ x[r].double()
        S = dy[r].double().abs().t() @ x[r].double().abs()
        ref = prod + beta * old[e].double()
        _close(dw[e], ref, _tol(F32, ref, S, 512) + 2.0 ** -24 * prod.abs(), e)
    assert torch.equal(dw[1], beta * old[1])              # an empty group


@pytest.mark.parametrize("beta", [0.0, 1.0, 0.5])
def test_wgrad_without_rows(mgq, beta):
    old = torch.randn(2, 16, 24, device="cuda")
    dw = old.clone() if beta else torch.full_like(old, float("nan"))
    e = torch.empty(0, 16, dtype=BF, device="cuda"), torch.empty(0, 24, dtype=BF, device="cuda")
    mgq.ragged_gemm_wgrad(*e, _off([0, 0, 0]), dw, beta=beta)
    assert torch.equal(dw, beta * old)


@pytest.mark.parametrize("R", [5, 4000])
def test_all_groups_empty(mgq, R):
    """Rows, but none in a group: nothing is written but the empty groups' zeros."""
    off, N, K = _off([2, 2, 2]), 1032, 48
    x, dy, w = (torch.full(s, float("nan"), dtype=BF, device="cuda") for s in ((R, K), (R, N), (2, N, K)))
    y, dx = torch.full((R, N), 7.0, device="cuda"), torch.full((R, K), 7.0, dtype=BF, device="cuda")
    dw = torch.full((2, N, K), 7.0, device="cuda")
    mgq.ragged_gemm_fwd(x, w, off, y)
    mgq.ragged_gemm_dgrad(dy, w, off, dx)
    mgq.ragged_gemm_wgrad(dy, x, off, dw)
    mgq.ragged_gemm_int8(torch.ones(R, K, dtype=I8, device="cuda"), y[:, 0].contiguous(),
                         torch.ones(2, N, K, dtype=I8, device="cuda"), dw[:, :, 0].contiguous(), off, y)
    assert mgq.get_error() == mgq.OK
    assert (y == 7).all() and (dx == 7).all() and (dw == 0).all()


@pytest.mark.parametrize("small", [True, False])
def test_foreign_nan_stays_out(mgq, small):
    """NaN and infinity of one group's rows and weight reach no other group."""
    g = _gen(4)
    counts = [7, 9, 30, 3] if small else [300, 261, 1000, 700]
    N, K = (136, 136) if small else (1544, 136)
    b = _bounds(counts, 0)
    x, dy, w = _randn(g, b[-1], K), _randn(g, b[-1], N), _randn(g, 4, N, K)
    runs = []
    for poison in (False, True):
        if poison:
            x[b[1]:b[2]], dy[b[1]:b[2]], w[1] = float("nan"), float("inf"), float("nan")
        y, dx, dw = (torch.empty(s, dtype=BF, device="cuda") for s in ((b[-1], N), (b[-1], K), (4, N, K)))
        mgq.ragged_gemm_fwd(x, w, _off(b), y)
        mgq.ragged_gemm_dgrad(dy, w, _off(b), dx)
        mgq.ragged_gemm_wgrad(dy, x, _off(b), dw)
        runs.append((y, dx, dw))
    (y0, dx0, dw0), (y1, dx1, dw1) = runs
    for r in (slice(0, b[1]), slice(b[2], b[4])):
        assert torch.equal(y0[r], y1[r]) and torch.equal(dx0[r], dx1[r])
    assert torch.equal(dw0[[0, 2, 3]], dw1[[0, 2, 3]])
    assert y1[b[1]:b[2]].isnan().all() and dw1[1].isnan().all()


@pytest.mark.parametrize("R", [3, 3000])
def test_row_pitch(mgq, R):
    """Activations and results inside wider buffers; the columns beside them stay as they were."""
    g = _gen(5)
    N, K, E = 1032, 72, 3
    b = [0, R // 3, R // 3, R]
    wide_x, wide_dy = _randn(g, R, K + 40), _randn(g, R, N + 8)
    x, dy, w = wide_x[:, 8:8 + K], wide_dy[:, 8:], _randn(g, E, N, K)
    for dt in (BF, F32):
        wide_y = torch.full((R, N + 16), 3.0, dtype=dt, device="cuda")
        wide_dx = torch.full((R, K + 24), 3.0, dtype=dt, device="cuda")
        y, dx = wide_y[:, 8:8 + N], wide_dx[:, 16:16 + K]
        mgq.ragged_gemm_fwd(x, w, _off(b), y)
        mgq.ragged_gemm_dgrad(dy, w, _off(b), dx)
        y2, dx2 = torch.empty(R, N, dtype=dt, device="cuda"), torch.empty(R, K, dtype=dt, device="cuda")
        mgq.ragged_gemm_fwd(x.contiguous(), w, _off(b), y2)
        mgq.ragged_gemm_dgrad(dy.contiguous(), w, _off(b), dx2)
        assert torch.equal(y, y2) and torch.equal(dx, dx2)
        assert (wide_y[:, :8] == 3).all() and (wide_y[:, 8 + N:] == 3).all()
        assert (wide_dx[:, :16] == 3).all() and (wide_dx[:, 16 + K:] == 3).all()
    dw, dw2 = (torch.empty(E, N, K, device="cuda") for _ in range(2))
    mgq.ragged_gemm_wgrad(dy, x, _off(b), dw)
    mgq.ragged_gemm_wgrad(dy.contiguous(), x.contiguous(), _off(b), dw2)
    assert torch.equal(dw, dw2)


def _int8(g, *shape):
    return torch.randint(-128, 128, shape, device="cuda", generator=g, dtype=I8)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_int8(mgq, shape, dt):
    counts, lead, tail, N, K = shape
    K = K // 16 * 16
    g = _gen(6)
    b = _bounds(counts, lead)
    R, E = b[-1] + tail, len(counts)
    x, w = _int8(g, R, K), _int8(g, E, N, K)
    xs = torch.rand(R, device="cuda", generator=g) + 0.01
    ws = torch.rand(E, N, device="cuda", generator=g) - 0.5
    y = torch.full((R, N), 7.0, dtype=dt, device="cuda")
    mgq.ragged_gemm_int8(x, xs, w, ws, _off(b), y)
    assert mgq.get_error() == mgq.OK
    assert (y[:lead] == 7).all() and (y[b[-1]:] == 7).all()
    half = 2.0 ** -24 if dt is F32 else 2.0 ** -8
    for e in range(E):
        r = slice(b[e], b[e + 1])
        acc = x[r].double() @ w[e].double().t()
        assert acc.numel() == 0 or acc.abs().max() < 2 ** 24
        ref = acc * xs[r, None].double() * ws[e].double()
        _close(y[r], ref, (half + 3 * 2.0 ** -24) * ref.abs() + 1e-38, e)


@pytest.mark.parametrize("N,K", [(32, 768), (136, 1040), (32, 4096)])
@pytest.mark.parametrize("op", ["fwd", "dgrad", "int8"])
def test_many_groups_of_few_rows(mgq, op, N, K):
    """More short tiles than the GPU holds at once, and places for tiles that turn out not to exist behind them: a
    ring's slot is refilled from L2 right after it is given back, so that a read of it that is still under way shows."""
    E = 1024
    counts = torch.randint(0, 3, (E,), generator=torch.Generator().manual_seed(3))
    b = _bounds(counts.tolist(), 0)
    R, g = b[-1], _gen(23)
    group = torch.repeat_interleave(torch.arange(E), counts).cuda()
    if op == "int8":
        x, w = _int8(g, R, K), _int8(g, E, N, K)
        ones = (torch.ones(R, device="cuda"), torch.ones(E, N, device="cuda"))
        run, wt, C = lambda o: mgq.ragged_gemm_int8(x, ones[0], w, ones[1], _off(b), o), w.transpose(1, 2), K
    elif op == "fwd":
        x, w = _randn(g, R, K), _randn(g, E, N, K)
        run, wt, C = lambda o: mgq.ragged_gemm_fwd(x, w, _off(b), o), w.transpose(1, 2), K
    else:
        x, w = _randn(g, R, K), _randn(g, E, K, N)
        run, wt, C = lambda o: mgq.ragged_gemm_dgrad(x, w, _off(b), o), w, K
    ref, S = torch.empty(R, N, dtype=torch.float64, device="cuda"), torch.empty(R, N, dtype=torch.float64, device="cuda")
    for r in range(0, R, 128):
        xr, wr = x[r:r + 128, None].double(), wt[group[r:r + 128]].double()
        ref[r:r + 128], S[r:r + 128] = torch.bmm(xr, wr)[:, 0], torch.bmm(xr.abs(), wr.abs())[:, 0]
    for _ in range(4):
        y = torch.full((R, N), 7.0, device="cuda")
        run(y)
        assert mgq.get_error() == mgq.OK
        if op == "int8":
            _close(y, ref, torch.where(S < 2 ** 24, 0.0, (K / 16) * 2.0 ** -23 * S), op)
        else:
            _close(y, ref, _tol(F32, ref, S, C), op)


@pytest.mark.parametrize("R", [2, 40, 5000])
def test_int8_sums_exact_whatever_the_codes(mgq, R):
    """K of 1024, all codes at the ends of their range: |sum| up to 2^24, every one an integer."""
    g = _gen(7)
    N, K = 512, 1024
    x = torch.where(torch.rand(R, K, device="cuda", generator=g) < 0.5, -128, 127).to(I8)
    w = torch.where(torch.rand(1, N, K, device="cuda", generator=g) < 0.5, -128, 127).to(I8)
    x[0], w[0, 0] = -128, -128                            # 2^24 itself
    y = torch.empty(R, N, device="cuda")
    mgq.ragged_gemm_int8(x, torch.ones(R, device="cuda"), w, torch.ones(1, N, device="cuda"), None, y)
    assert torch.equal(y.double(), x.double() @ w[0].double().t())


def test_int8_long_sums(mgq):
    """Beyond 2^24: within 2^-23 of the running sum a step of 16 (the header's bound), plus the scales' roundings."""
    for R in (3, 4000):
        K, N = 14336, 512
        x, w = torch.full((R, K), 127, dtype=I8, device="cuda"), torch.full((1, N, K), 127, dtype=I8, device="cuda")
        y = torch.empty(R, N, device="cuda")
        mgq.ragged_gemm_int8(x, torch.ones(R, device="cuda"), w, torch.ones(1, N, device="cuda"), None, y)
        ref = 127.0 * 127.0 * K
        assert ((y.double() - ref).abs() <= (K / 16 + 4) * 2.0 ** -23 * ref).all()


# R, E, N of the few-row form with a split contraction, without a split, and of the large form
LONG_SUMS = [(13, 1, 520), (37, 2, 10240), (1307, 1, 1544), (1307, 2, 1544)]


@pytest.mark.parametrize("K", [1040, 2048, 14352])
@pytest.mark.parametrize("R,E,N", LONG_SUMS)
def test_int8_float32_sums_of_any_codes(mgq, R, E, N, K):
    """Codes of one sign, so that sums pass 2^24 and their last bits count: parts of 1024 elements are integers up to
    2^24, exact; each part is added with one rounding (at most one more a part where a cluster splits the contraction),
    and the scales take two roundings, so every one is at most 2^-24 of the final sum."""
    g = _gen(26)
    b = _bounds([R] if E == 1 else [R // 3, R - R // 3], 0)
    x = torch.randint(64, 128, (R, K), device="cuda", generator=g).to(I8)
    w = torch.randint(64, 128, (E, N, K), device="cuda", generator=g).to(I8)
    # products of 97 to 127 in every place: each step of 16 then cuts off the same
    x[::2] = (97 + torch.arange(R, device="cuda") % 31).to(I8)[::2, None]
    w[:, ::2] = (97 + torch.arange(N, device="cuda") % 31).to(I8)[None, ::2, None]
    x[R // 2:] = -x[R // 2:]
    xs = torch.rand(R, device="cuda", generator=g) + 0.5
    ws = torch.rand(E, N, device="cuda", generator=g) + 0.5
    y = torch.empty(R, N, device="cuda")
    mgq.ragged_gemm_int8(x, xs, w, ws, _off(b), y)
    assert mgq.get_error() == mgq.OK
    for e in range(E):
        r = slice(b[e], b[e + 1])
        ref = (x[r].double() @ w[e].double().t()) * xs[r, None].double() * ws[e].double()
        _close(y[r], ref, (2 * math.ceil(K / 1024) + 2) * 2.0 ** -24 * ref.abs(), e)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_int8_float32_in_parts(mgq, shape):
    """Contractions of more than 1024 elements, whose sums leave the accumulator in parts: every group and tile."""
    counts, lead, tail, N, _ = shape
    test_int8(mgq, (counts, lead, tail, N, 2576), F32)


def test_int8_nan_scale(mgq):
    g = _gen(8)
    for R in (6, 3000):
        x, w = _int8(g, R, 64), _int8(g, 1, 1032, 64)
        xs, ws = torch.ones(R, device="cuda"), torch.ones(1, 1032, device="cuda")
        xs[1], ws[0, 5] = float("nan"), float("nan")
        y = torch.empty(R, 1032, device="cuda")
        mgq.ragged_gemm_int8(x, xs, w, ws, None, y)
        nan = torch.zeros(R, 1032, dtype=torch.bool, device="cuda")
        nan[1], nan[:, 5] = True, True
        assert torch.equal(y.isnan(), nan)


def test_int8_row_pitch(mgq):
    g = _gen(9)
    for R in (5, 3000):
        wide, w = _int8(g, R, 96 + 64), _int8(g, 2, 1032, 96)
        x = wide[:, 16:112]
        b = _off([0, R // 2, R])
        xs, ws = torch.rand(R, device="cuda"), torch.rand(2, 1032, device="cuda")
        wide_y = torch.full((R, 1048), 3.0, dtype=BF, device="cuda")
        y2 = torch.empty(R, 1032, dtype=BF, device="cuda")
        mgq.ragged_gemm_int8(x, xs, w, ws, b, wide_y[:, 8:1040])
        mgq.ragged_gemm_int8(x.contiguous(), xs, w, ws, b, y2)
        assert torch.equal(wide_y[:, 8:1040], y2) and (wide_y[:, :8] == 3).all() and (wide_y[:, 1040:] == 3).all()


def _quant_ref(x):
    xd = x.double()
    amax = xd.abs().amax(-1, keepdim=True)
    return torch.round(127 * xd / torch.where(amax == 0, 1.0, amax)), amax[:, 0] / 127


@pytest.mark.parametrize("T,K", [(1, 16), (3, 512), (130, 1024), (7, 1040), (33, 4096), (5, 4112), (9, 14336), (2, 40000)])
@pytest.mark.parametrize("kind", ["normal", "ties", "tiny", "huge"])
def test_quantiser(mgq, T, K, kind):
    g = _gen(10)
    x = torch.randn(T, K, device="cuda", generator=g)
    if kind == "ties":        # small integers over powers of two: quotients that end in a half, and just beside one
        x = torch.randint(-255, 256, (T, K), device="cuda", generator=g).float()
        x *= 2.0 ** -torch.randint(0, 9, (T, K), device="cuda", generator=g).float()
        x[:, 0] = torch.randint(1, 256, (T,), device="cuda", generator=g).float() * 2.0
    elif kind == "tiny":      # subnormal bf16 values among them
        x *= 2.0 ** -130
    elif kind == "huge":
        x = (x * 2.0 ** 126).clamp(-3.3e38, 3.3e38)
    x = x.to(BF)
    codes, scale = torch.empty(T, K, dtype=I8, device="cuda"), torch.empty(T, device="cuda")
    mgq.rows_quantize_int8(x, codes, scale)
    ref, s = _quant_ref(x)
    assert torch.equal(codes.double(), ref)
    assert torch.equal(scale, s.float())


def test_quantiser_odd_rows(mgq):
    """Rows of zeros, with a NaN, with an infinity; a row pitch; nothing behind the last row is written."""
    g = _gen(11)
    for K in (64, 2048, 20000):
        wide = _randn(g, 6, K + 24)
        x = wide[:, 8:8 + K]
        x[1], x[2, 3], x[3, 0], x[4, K - 1] = 0, float("nan"), float("inf"), float("-inf")
        codes, scale = torch.full((8, K), 9, dtype=I8, device="cuda"), torch.full((8,), 9.0, device="cuda")
        mgq.rows_quantize_int8(x, codes[:6], scale[:6])
        ref, s = _quant_ref(x[[0, 1, 5]])
        assert torch.equal(codes[[0, 1, 5]].double(), ref) and torch.equal(scale[[0, 1, 5]], s.float())
        assert (codes[2:5] == 0).all() and scale[2:5].isnan().all()
        assert (codes[6:] == 9).all() and (scale[6:] == 9).all()


@pytest.mark.parametrize("bad", [[0, 5, 4, 10], [-1, 2, 5, 10], [0, 2, 5, 5000], [7, 2, 5, 10]])
@pytest.mark.parametrize("R", [10, 4000])
def test_offsets_that_are_no_partition(mgq, bad, R):
    """Reported, with nothing written; the next call works."""
    g = _gen(12)
    N, K = 1032, 64
    x, dy, w = _randn(g, R, K), _randn(g, R, N), _randn(g, 3, N, K)
    if bad[-1] == 10:
        bad = bad[:-1] + [R]
    good = _off([0, 2, 5, R])
    y, dx = torch.full((R, N), 7.0, dtype=BF, device="cuda"), torch.full((R, K), 7.0, device="cuda")
    dw = torch.full((3, N, K), 7.0, device="cuda")
    x8, w8, s = x.to(I8), w.to(I8), torch.ones(R, device="cuda")
    calls = [lambda o: mgq.ragged_gemm_fwd(x, w, o, y), lambda o: mgq.ragged_gemm_dgrad(dy, w, o, dx),
             lambda o: mgq.ragged_gemm_wgrad(dy, x, o, dw),
             lambda o: mgq.ragged_gemm_int8(x8, s, w8, torch.ones(3, N, device="cuda"), o, y)]
    for call in calls:
        call(_off(bad))
        assert mgq.get_error() == mgq.ERR_INVALID_ARG
        assert (y == 7).all() and (dx == 7).all() and (dw == 7).all()
    for call, out in zip(calls, (y, dx, dw, y)):
        call(good)
        assert mgq.get_error() == mgq.OK and not (out == 7).all()


def test_plain_products(mgq):
    """offsets None: one group of all rows, and nothing to do without rows."""
    g = _gen(13)
    for R in (1, 33, 2700):
        N, K = 1032, 80
        x, dy, w = _randn(g, R, K), _randn(g, R, N), _randn(g, 1, N, K)
        outs = []
        for off in (None, _off([0, R])):
            y, dx = torch.empty(R, N, device="cuda"), torch.empty(R, K, device="cuda")
            dw, z = torch.empty(1, N, K, device="cuda"), torch.empty(R, N, device="cuda")
            mgq.ragged_gemm_fwd(x, w, off, y)
            mgq.ragged_gemm_dgrad(dy, w, off, dx)
            mgq.ragged_gemm_wgrad(dy, x, off, dw)
            mgq.ragged_gemm_int8((x * 10).to(I8), y[:, 0].contiguous(), (w * 10).to(I8), dw[:, :, 0].contiguous(), off, z)
            outs.append((y, dx, dw, z))
        assert all(torch.equal(a, b) for a, b in zip(*outs))
        ref, S = x.double() @ w[0].double().t(), x.double().abs() @ w[0].double().abs().t()
        _close(outs[0][0], ref, _tol(F32, ref, S, K), R)
    empty = torch.empty(0, 16, dtype=BF, device="cuda")
    mgq.ragged_gemm_fwd(empty, torch.empty(3, 8, 16, dtype=BF, device="cuda"), _off([0, 0, 0, 0]),
                        torch.empty(0, 8, dtype=BF, device="cuda"))
    with pytest.raises(mgq.MGQError):
        mgq.ragged_gemm_fwd(x, torch.cat([w, w]), None, torch.empty(R, N, device="cuda"))


def test_refusals(mgq):
    """Tensors that do not fit together, on the device."""
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")
    off = _off([0, 2, 4])
    bad = [
        lambda: mgq.ragged_gemm_fwd(z(4, 16), z(2, 8, 16), _off([0, 4]), z(4, 8)),            # offsets of another E
        lambda: mgq.ragged_gemm_fwd(z(4, 16), z(2, 8, 16), off.long(), z(4, 8)),
        lambda: mgq.ragged_gemm_fwd(z(4, 16), z(2, 8, 16), off.cpu(), z(4, 8)),
        lambda: mgq.ragged_gemm_fwd(z(4, 24), z(2, 8, 16), off, z(4, 8)),
        lambda: mgq.ragged_gemm_fwd(z(4, 16), z(2, 8, 16), off, z(3, 8)),
        lambda: mgq.ragged_gemm_fwd(z(16, 4).t(), z(2, 8, 16), off, z(4, 8)),                 # columns contiguous
        lambda: mgq.ragged_gemm_fwd(z(4, 16), z(2, 16, 8).transpose(1, 2), off, z(4, 8)),
        lambda: mgq.ragged_gemm_fwd(z(4, 12), z(2, 8, 12), off, z(4, 8)),                     # K not a multiple of 8
        lambda: mgq.ragged_gemm_fwd(z(4, 20)[:, :16], z(2, 8, 16), off, z(4, 8)),             # row pitch 20
        lambda: mgq.ragged_gemm_dgrad(z(4, 8), z(2, 8, 16), off, z(4, 8)),
        lambda: mgq.ragged_gemm_wgrad(z(4, 8), z(4, 16), off, z(2, 16, 8)),
        lambda: mgq.ragged_gemm_wgrad(z(4, 8), z(4, 16), off, z(2, 8, 16), beta=1.0),         # bf16 accumulates nothing
        lambda: mgq.ragged_gemm_int8(z(4, 16, dtype=I8), z(4, dtype=F32), z(2, 8, 16, dtype=I8), z(2, 16, dtype=F32), off,
                                     z(4, 8)),
        lambda: mgq.ragged_gemm_int8(z(4, 16, dtype=I8), z(5, dtype=F32), z(2, 8, 16, dtype=I8), z(2, 8, dtype=F32), off,
                                     z(4, 8)),
        lambda: mgq.ragged_gemm_int8(z(4, 24, dtype=I8), z(4, dtype=F32), z(2, 8, 24, dtype=I8), z(2, 8, dtype=F32), off,
                                     z(4, 8)),
        lambda: mgq.rows_quantize_int8(z(4, 24), z(4, 24, dtype=I8), z(4, dtype=F32)),
        lambda: mgq.rows_quantize_int8(z(4, 16), z(4, 32, dtype=I8)[:, :16], z(4, dtype=F32)),
        lambda: mgq.rows_quantize_int8(z(4, 16), z(4, 16, dtype=I8), z(4, 1, dtype=F32)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(mgq.MGQError) as e:
            call()
        assert e.value.status == mgq.ERR_INVALID_ARG, i


def test_differences_of_the_forward(mgq):
    """Small integers, for which every sum is exact: the forward is linear, so its differences along a
    direction equal the gradients' products with it, to the bit."""
    g = _gen(14)
    counts, N, K = [40, 0, 300, 7], 264, 136
    b = _bounds(counts, 0)
    i = lambda *s: torch.randint(-3, 4, s, device="cuda", generator=g).to(BF)
    x, dx_, w, dw_, dy = i(b[-1], K), i(b[-1], K), i(4, N, K), i(4, N, K), i(b[-1], N)

    def loss(x, w):
        y = torch.empty(b[-1], N, device="cuda")
        mgq.ragged_gemm_fwd(x, w, _off(b), y)
        return (y.double() * dy.double()).sum()

    gx, gw = torch.empty(b[-1], K, device="cuda"), torch.empty(4, N, K, device="cuda")
    mgq.ragged_gemm_dgrad(dy, w, _off(b), gx)
    mgq.ragged_gemm_wgrad(dy, x, _off(b), gw)
    assert loss(x + dx_, w) - loss(x - dx_, w) == 2 * (gx.double() * dx_.double()).sum()
    assert loss(x, w + dw_) - loss(x, w - dw_) == 2 * (gw.double() * dw_.double()).sum()


def test_offsets_past_32_bits(mgq):
    """Results and activations of more than 2^31 elements: the last rows."""
    g = _gen(15)
    R, N, K = 40000, 57344, 16
    x, w = _randn(g, R, K), _randn(g, 2, N, K)
    y = torch.empty(R, N, dtype=BF, device="cuda")
    off = _off([0, R - 5, R])
    mgq.ragged_gemm_fwd(x, w, off, y)
    for e, r in ((0, slice(R - 40, R - 5)), (1, slice(R - 5, R))):
        ref, S = x[r].double() @ w[e].double().t(), x[r].double().abs() @ w[e].double().abs().t()
        _close(y[r], ref, _tol(BF, ref, S, K), e)
    v = _randn(g, 2, 16, N)                               # y as the input: contraction N, 16 outputs
    z = torch.empty(R, 16, device="cuda")
    mgq.ragged_gemm_fwd(y, v, off, z)
    for e, r in ((0, slice(R - 40, R - 5)), (1, slice(R - 5, R))):
        ref, S = y[r].double() @ v[e].double().t(), y[r].double().abs() @ v[e].double().abs().t()
        _close(z[r], ref, _tol(F32, ref, S, N), e)
    codes, scale = torch.empty(R, N, dtype=I8, device="cuda"), torch.empty(R, device="cuda")
    mgq.rows_quantize_int8(y, codes, scale)
    ref, s = _quant_ref(y[-7:])
    assert torch.equal(codes[-7:].double(), ref) and torch.equal(scale[-7:], s.float())
    w8, ws = _int8(g, 2, 16, N), torch.ones(2, 16, device="cuda")
    mgq.ragged_gemm_int8(codes, scale, w8, ws, off, z)
    acc = codes[-5:].double() @ w8[1].double().t()
    assert acc.abs().max() < 2 ** 24
    _close(z[-5:], acc * scale[-5:, None].double(), 4 * 2.0 ** -24 * (acc * scale[-5:, None].double()).abs() + 1e-38, "int8")


def test_streams_graphs_and_repeats(mgq):
    """Two streams at once, and a captured graph replayed on new inputs, give the bits of a call by itself."""
    g = _gen(16)
    for counts, N, K in (([3, 0, 14, 1], 264, 2064), ([700, 33, 0, 1500], 1544, 520)):
        b = _bounds(counts, 0)
        R, off = b[-1], _off(b)
        x, dy, w = _randn(g, R, K), _randn(g, R, N), _randn(g, 4, N, K)
        K16 = K // 16 * 16
        x8, w8 = _int8(g, R, K16), _int8(g, 4, N, K16)
        xs, ws = torch.rand(R, device="cuda"), torch.rand(4, N, device="cuda")
        make = lambda: (torch.empty(R, N, dtype=BF, device="cuda"), torch.empty(R, K, device="cuda"),
                        torch.empty(4, N, K, device="cuda"), torch.empty(R, N, device="cuda"))

        def run(o, s=None):
            mgq.ragged_gemm_fwd(x, w, off, o[0], stream=s)
            mgq.ragged_gemm_dgrad(dy, w, off, o[1], stream=s)
            mgq.ragged_gemm_wgrad(dy, x, off, o[2], stream=s)
            mgq.ragged_gemm_int8(x8, xs, w8, ws, off, o[3], stream=s)

        first = make()
        run(first)
        torch.cuda.synchronize()
        streams, outs = [torch.cuda.Stream() for _ in range(2)], [make() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(3):
            for s, o in zip(streams, outs):
                run(o, s)
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, c) for a, c in zip(first, o))
        graph, held = torch.cuda.CUDAGraph(), make()
        with torch.cuda.graph(graph):
            run(held)
        old = x.clone()
        x.copy_(_randn(g, R, K))
        for _ in range(2):
            graph.replay()
        again = make()
        run(again)
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(again, held)) and not torch.equal(first[0], held[0])
        x.copy_(old)
        assert mgq.get_error() == mgq.OK


@pytest.mark.parametrize("R", [24, 3000])
def test_first_calls_inside_a_capture(R):
    """A process whose first call of each operator is captured; the replay gives the bits of a later call."""
    code = f"""
import torch
from fp8_grouped_gemm_gb300 import mgq
R, N, K, E = {R}, 264, 1040, 3
x, dy, w = (torch.randn(s, device="cuda").bfloat16() for s in ((R, K), (R, N), (E, N, K)))
x8, w8 = (torch.randint(-128, 128, s, device="cuda", dtype=torch.int8) for s in ((R, K), (E, N, K)))
xs, ws, off = torch.rand(R, device="cuda"), torch.rand(E, N, device="cuda"), torch.tensor([0, R // 3, R // 2, R]).int().cuda()
new = lambda: [torch.zeros(s, device="cuda", dtype=d) for s, d in (((R, N), torch.bfloat16), ((R, K), torch.float32),
               ((E, N, K), torch.float32), ((R, N), torch.float32), ((R, K), torch.int8), ((R,), torch.float32))]
def run(o):
    mgq.ragged_gemm_int8(x8, xs, w8, ws, off, o[3])
    mgq.rows_quantize_int8(x, o[4], o[5])
    mgq.ragged_gemm_fwd(x, w, off, o[0])
    mgq.ragged_gemm_dgrad(dy, w, off, o[1])
    mgq.ragged_gemm_wgrad(dy, x, off, o[2])
a, b, g = new(), new(), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    run(a)
g.replay()
run(b)
torch.cuda.synchronize()
assert mgq.get_error() == mgq.OK and all(t.any() for t in a) and all(torch.equal(s, t) for s, t in zip(a, b))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_host_threads(mgq):
    """Four host threads on streams of their own, sizes of both forms: the bits of calls one after the other."""
    g = _gen(24)
    N, K = 520, 1040
    w, w8, ws = _randn(g, 4, N, K), _int8(g, 4, N, K), torch.rand(4, N, device="cuda")
    sets = []
    for R in (6, 40, 900, 2500):
        off = _off([0, R // 2, R // 2, R - 1, R])
        sets.append((_randn(g, R, K), _int8(g, R, K), torch.rand(R, device="cuda"), off, R))

    def run(i, out):
        x, x8, xs, off, R = sets[i]
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for y, y8 in out:
                mgq.ragged_gemm_fwd(x, w, off, y)
                mgq.ragged_gemm_int8(x8, xs, w8, ws, off, y8)
        s.synchronize()

    def new(n):
        return [[(torch.zeros(q[4], N, device="cuda"), torch.zeros(q[4], N, device="cuda")) for _ in range(n)] for q in sets]

    outs, one = new(20), new(1)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(i, outs[i])) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    for i in range(4):
        run(i, one[i])
        for y, y8 in outs[i]:
            assert torch.equal(y, one[i][0][0]) and torch.equal(y8, one[i][0][1])
    assert mgq.get_error() == mgq.OK


def test_first_calls_from_host_threads():
    """A process whose first call of each operator comes from several threads at once, each thread's first CUDA call
    at all being the library's (raw entry points, no stream of its own): the bits of later calls."""
    code = """
import ctypes, threading, torch
from fp8_grouped_gemm_gb300 import mgq
E, N, K = 4, 520, 2064
lib, work = mgq.load(), []
for R in (6, 900, 2500):
    x, dy, w = (torch.randn(s, device="cuda").bfloat16() for s in ((R, K), (R, N), (E, N, K)))
    x8, w8 = (torch.randint(-128, 128, s, device="cuda", dtype=torch.int8) for s in ((R, K), (E, N, K)))
    xs, ws, off = torch.rand(R, device="cuda"), torch.rand(E, N, device="cuda"), torch.tensor([0, R // 2, R // 2, R - 1, R]).int().cuda()
    p = lambda t: t.data_ptr()
    for f32 in (0, 1):
        dt = torch.float32 if f32 else torch.bfloat16
        new = lambda *s, dt=dt: torch.zeros(s, device="cuda", dtype=dt)
        hold = (x, dy, w, x8, w8, xs, ws, off)
        calls = [
            (lambda o, x=x, w=w, off=off, R=R, f32=f32: lib.mgq_ragged_gemm_fwd(p(x), K, p(w), p(off), E, R, N, K, p(o), N, f32, None), new, (R, N)),
            (lambda o, dy=dy, w=w, off=off, R=R, f32=f32: lib.mgq_ragged_gemm_dgrad(p(dy), N, p(w), p(off), E, R, N, K, p(o), K, f32, None), new, (R, K)),
            (lambda o, dy=dy, x=x, off=off, R=R, f32=f32: lib.mgq_ragged_gemm_wgrad(p(dy), N, p(x), K, p(off), E, R, N, K, 0.0, p(o), f32, None), new, (E, N, K)),
            (lambda o, x8=x8, xs=xs, w8=w8, ws=ws, off=off, R=R, f32=f32: lib.mgq_ragged_gemm_int8(p(x8), K, p(xs), p(w8), p(ws), p(off), E, R, N, K, p(o), N, f32, None), new, (R, N))]
        for call, new, shape in calls:
            work.append((call, [new(*shape) for _ in range(3)], hold))
torch.cuda.synchronize()
bad = []
def run(call, out, gate):
    gate.wait()
    rc = call(out)
    if rc:
        bad.append(rc)
for call, outs, _ in work:                       # two threads for every kernel, new ones each time
    gate = threading.Barrier(2)
    ts = [threading.Thread(target=run, args=(call, o, gate)) for o in outs[:2]]
    [t.start() for t in ts]
    [t.join() for t in ts]
for call, outs, _ in work:
    assert call(outs[2]) == 0
torch.cuda.synchronize()
assert not bad and mgq.get_error() == mgq.OK, bad
for call, (a, b, c), _ in work:
    assert c.any() and torch.equal(a, c) and torch.equal(b, c)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_rows_do_not_depend_on_other_groups(mgq):
    """A group's results with other groups around it, where both calls take the same form."""
    g = _gen(17)
    N, K = 1544, 264
    x, w = _randn(g, 3000, K), _randn(g, 3, N, K)
    y, z = torch.empty(3000, N, dtype=BF, device="cuda"), torch.empty(2000, N, dtype=BF, device="cuda")
    mgq.ragged_gemm_fwd(x, w, _off([0, 517, 2517, 3000]), y)
    mgq.ragged_gemm_fwd(x[517:2517], w[1:2], None, z)
    assert torch.equal(y[517:2517], z)


@pytest.mark.parametrize("R", [20, 4000])
def test_waits_run_out(mgq, R):
    """No loads are issued: every wait gives up, the call reports it, and the next one works."""
    g = _gen(18)
    N, K = 1544, 136
    b = _off([0, 5, R])
    x, dy, w = _randn(g, R, K), _randn(g, R, N), _randn(g, 2, N, K)
    K16 = 128
    x8, w8 = _int8(g, R, K16), _int8(g, 2, N, K16)
    s, t = torch.ones(R, device="cuda"), torch.ones(2, N, device="cuda")
    y, dx, dw = torch.empty(R, N, device="cuda"), torch.empty(R, K, device="cuda"), torch.empty(2, N, K, device="cuda")
    calls = [lambda: mgq.ragged_gemm_fwd(x, w, b, y), lambda: mgq.ragged_gemm_dgrad(dy, w, b, dx),
             lambda: mgq.ragged_gemm_wgrad(dy, x, b, dw), lambda: mgq.ragged_gemm_int8(x8, s, w8, t, b, y)]
    outs = [y, dx, dw, y]
    for call, out in zip(calls, outs):
        call()
        torch.cuda.synchronize()
        good = out.clone()
        mgq.set_gemm_option(mgq.GEMM_OPT_WAIT_MS, 20)
        mgq.set_gemm_option(mgq.GEMM_OPT_DEBUG_STALL, 1)
        try:
            call()
            assert mgq.get_error() == mgq.ERR_TIMEOUT
        finally:
            mgq.set_gemm_option(mgq.GEMM_OPT_DEBUG_STALL, 0)
            mgq.set_gemm_option(mgq.GEMM_OPT_WAIT_MS, 0)
        call()
        assert mgq.get_error() == mgq.OK and torch.equal(out, good)


@pytest.mark.parametrize("R", [20, 4000])
@pytest.mark.parametrize("dt", [BF, F32])
def test_waits_run_out_over_long_contractions(mgq, R, dt):
    """The same where a cluster splits the contraction (R 20) and where the sum leaves in parts (R 4000, float32)."""
    g = _gen(27)
    N, K = 1544, 4112
    b = _off([0, 5, R])
    x, w = _randn(g, R, K), _randn(g, 2, N, K)
    x8, w8, s, t = _int8(g, R, K), _int8(g, 2, N, K), torch.ones(R, device="cuda"), torch.ones(2, N, device="cuda")
    for run in (lambda o: mgq.ragged_gemm_fwd(x, w, b, o), lambda o: mgq.ragged_gemm_int8(x8, s, w8, t, b, o)):
        good, out = (torch.empty(R, N, dtype=dt, device="cuda") for _ in range(2))
        run(good)
        mgq.set_gemm_option(mgq.GEMM_OPT_WAIT_MS, 20)
        mgq.set_gemm_option(mgq.GEMM_OPT_DEBUG_STALL, 1)
        try:
            run(out)
            assert mgq.get_error() == mgq.ERR_TIMEOUT
        finally:
            mgq.set_gemm_option(mgq.GEMM_OPT_DEBUG_STALL, 0)
            mgq.set_gemm_option(mgq.GEMM_OPT_WAIT_MS, 0)
        run(out)
        assert mgq.get_error() == mgq.OK and torch.equal(out, good)


# ---------------------------------------------------------------------------
# together: the routed experts' layer over unpadded groups

def _route(mgq, idx, E):
    """Unpadded routing (align 1): token of each row, offsets, rows of each token."""
    T, k = idx.shape
    cap = mgq.r_cap(T, k, E, 1)
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")
    rim, src, off, cnt = i32(T, k), i32(cap), i32(E + 1), i32(E)
    ws = torch.empty(max(16, mgq.permute_workspace_size(T, k, E)), dtype=torch.uint8, device="cuda")
    mgq.moe_route(idx, E, 1, cap, rim, src, off, cnt, ws)
    return src[:T * k].long() // k, off, rim.long()


def _layer_inputs(g, T, E, k, H, F):
    x = _randn(g, T, H)
    w1, w2 = _randn(g, E, 2 * F, H, scale=0.05), _randn(g, E, H, F, scale=0.05)
    top = torch.topk(torch.randn(T, E, device="cuda", generator=g), k)
    return x, w1, w2, top.indices.int(), torch.softmax(top.values, -1)


def _layer_f64(x, w1, w2, idx, probs):
    out = torch.zeros_like(x)
    F = w2.shape[2]
    for e in range(w1.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        gu = x[t] @ w1[e].t()
        h = torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]
        out = out.index_add(0, t, (h @ w2[e].t()) * probs[t, j][:, None])
    return out


@pytest.mark.parametrize("T,E", [(1, 8), (50, 12), (900, 5)])
def test_bf16_layer_forward_and_backward(mgq, T, E):
    """Routing, both projections and all six gradients in bf16, against float64 autograd: every bf16 rounding
    on the way (gu, h, y, dy, dh, dgu and the result: relative 2^-9 rms at most each) adds in quadrature, so a
    relative Frobenius error of 2^-9 sqrt(8) < 2^-7 is an upper bound for each result."""
    g = _gen(19)
    k, H, F = 3, 264, 136
    x, w1, w2, idx, probs = _layer_inputs(g, T, E, k, H, F)
    dout = _randn(g, T, H)
    tok, off, rim = _route(mgq, idx, E)
    R = T * k
    bf = lambda *s: torch.empty(*s, dtype=BF, device="cuda")
    xp, gu, y = x[tok], bf(R, 2 * F), bf(R, H)
    mgq.ragged_gemm_fwd(xp, w1, off, gu)
    gate, up = gu[:, :F].float(), gu[:, F:].float()
    sg = torch.sigmoid(gate)
    h = (gate * sg * up).to(BF)
    mgq.ragged_gemm_fwd(h, w2, off, y)
    out = (y[rim].float() * probs[..., None]).sum(1)

    p_row = torch.empty(R, device="cuda").scatter_(0, rim.reshape(-1), probs.reshape(-1))
    dy = (dout[tok].float() * p_row[:, None]).to(BF)
    dh, dxp = torch.empty(R, F, device="cuda"), torch.empty(R, H, device="cuda")
    dw1, dw2 = torch.empty(E, 2 * F, H, device="cuda"), torch.empty(E, H, F, device="cuda")
    mgq.ragged_gemm_dgrad(dy, w2, off, dh)
    mgq.ragged_gemm_wgrad(dy, h, off, dw2)
    dgu = torch.cat([dh * up * sg * (1 + gate * (1 - sg)), dh * gate * sg], 1).to(BF)
    mgq.ragged_gemm_dgrad(dgu, w1, off, dxp)
    mgq.ragged_gemm_wgrad(dgu, xp, off, dw1)
    dx = dxp[rim].sum(1)
    assert mgq.get_error() == mgq.OK

    xd, w1d, w2d = (t.double().requires_grad_() for t in (x, w1, w2))
    ref = _layer_f64(xd, w1d, w2d, idx, probs.double())
    grads = torch.autograd.grad((ref * dout.double()).sum(), (xd, w1d, w2d))
    for name, a, r in (("out", out, ref.detach()), ("dx", dx, grads[0]), ("dw1", dw1, grads[1]), ("dw2", dw2, grads[2])):
        err = (a.double() - r).norm() / r.norm()
        assert err < 2.0 ** -7, (name, float(err))


@pytest.mark.parametrize("T,E", [(1, 8), (300, 6)])
def test_int8_layer_forward(mgq, T, E):
    """Weights quantised by channel, tokens and h by row, both products in int8: equal to the same layer in
    float64 on the quantised values, to the bf16 roundings of gu, h and the result (each under 2^-9 rms) and the
    codes of h that such a rounding moves by one (under 2^-8 of amax / 127 each)."""
    g = _gen(20)
    k, H, F = 2, 272, 144
    x, w1, w2, idx, probs = _layer_inputs(g, T, E, k, H, F)

    def quant(t):
        flat = t.reshape(-1, t.shape[-1])
        c, s = torch.empty(flat.shape, dtype=I8, device="cuda"), torch.empty(flat.shape[0], device="cuda")
        mgq.rows_quantize_int8(flat, c, s)
        return c.view(t.shape), s.view(t.shape[:-1])

    tok, off, rim = _route(mgq, idx, E)
    R = T * k
    (w1c, w1s), (w2c, w2s), (xc, xs) = quant(w1), quant(w2), quant(x)
    gu, y = torch.empty(R, 2 * F, dtype=BF, device="cuda"), torch.empty(R, H, dtype=BF, device="cuda")
    mgq.ragged_gemm_int8(xc[tok], xs[tok], w1c, w1s, off, gu)
    h = (torch.nn.functional.silu(gu[:, :F].float()) * gu[:, F:].float()).to(BF)
    hc, hs = quant(h)
    mgq.ragged_gemm_int8(hc, hs, w2c, w2s, off, y)
    out = (y[rim].float() * probs[..., None]).sum(1)
    assert mgq.get_error() == mgq.OK
    deq = lambda c, s: c.double() * s.double()[..., None]
    xd, w1d, w2d = deq(xc, xs), deq(w1c, w1s), deq(w2c, w2s)
    off = off.tolist()
    ref_y = torch.empty(R, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        r = slice(off[e], off[e + 1])
        z = xd[tok[r]] @ w1d[e].t()
        hd = torch.nn.functional.silu(z[:, :F]) * z[:, F:]
        amax = hd.abs().amax(-1, keepdim=True)
        ref_y[r] = torch.round(127 * hd / torch.where(amax == 0, 1.0, amax)) * amax / 127 @ w2d[e].t()
    ref = (ref_y[rim] * probs.double()[..., None]).sum(1)
    assert (out.double() - ref).norm() / ref.norm() < 2.0 ** -6
