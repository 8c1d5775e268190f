"""GPU parity of the residual addition + RMSNorm (+ quantised output) and its
gradient with the float64 definitions.

Error bounds, with u = 2^-24 (float32) and H <= 16384: the sum of squares is
taken over at most 32 serial terms a thread and a tree, so rstd is within 64 u
of the exact value and y within 72 u (three more products); a bf16 output adds
half a bf16 ulp. Codes are held to the interval that the cast of y (1 -+ 72 u)
spans with the kernel's own scale, scales to that of the block's amax. In the
gradient, mean(g xh) is within 64 u mean|g xh|; dw, a sum of T terms in any
order, within (T + 16) u sum|dy xh|."""
import numpy as np
import pytest
import torch

from oracle import block as OB
from oracle import formats as OF
from oracle import quant as OQ
from tests.layer_check import bf16_np, u8_np, ulp_bf16, untile_mx_scales

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5
CODE_MAX = {0: 448.0, 1: 57344.0}


def _inputs(T, H, seed, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g)
    if H >= 16:
        x[:, H // 3] *= 50.0                      # one large channel
    r = torch.randn(T, H, generator=g) * 2.0
    w = 1.0 + 0.25 * torch.randn(H, generator=g)
    return x.bfloat16(), (r.bfloat16() if residual else None), w


def _near_bf16(got, ref, slack):
    ulp = ulp_bf16(np.abs(ref) + slack)
    assert np.all(np.abs(got - ref) <= 0.5 * ulp * (1 + 1e-9) + slack)


def _run(x, r, w, q=None, **kw):
    from fp8_grouped_gemm_gb300 import mgq
    dev = lambda t: None if t is None else t.cuda()
    T, H = x.shape
    out = dict(y=torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda"),
               rstd=torch.full((T,), 7.0, device="cuda"))
    if r is not None:
        out["sum_out"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    mgq.add_rmsnorm_quantize(dev(x), w.cuda(), EPS, q, residual=dev(r), **out, **kw)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("T,H", [(1, 8), (3, 40), (1, 128), (5, 1000), (129, 2048), (7, 4096), (700, 5120),
                                 (2, 8200), (3, 16384)])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("wdt", [torch.bfloat16, torch.float32])
def test_forward_without_codes(T, H, residual, wdt):
    x, r, w = _inputs(T, H, T + H, residual)
    w = w.to(wdt)
    o = _run(x, r, w)
    s, rstd, y = OB.rmsnorm(bf16_np(x), None if r is None else bf16_np(r), w.double().numpy(), EPS)
    assert np.all(np.abs(o["rstd"].cpu().numpy() - rstd) <= 64 * U * rstd)
    _near_bf16(bf16_np(o["y"]), y, 72 * U * np.abs(y))
    if residual:
        _near_bf16(bf16_np(o["sum_out"]), s, U * np.abs(s))


@pytest.mark.parametrize("T,H,wdt", [(40000, 128, torch.float32), (6001, 1000, torch.bfloat16),
                                     (2003, 4096, torch.bfloat16), (1300, 5120, torch.float32),
                                     (700, 16384, torch.bfloat16)])
@pytest.mark.parametrize("residual", [True, False])
def test_forward_of_many_rows(T, H, wdt, residual):
    """Enough rows for the streamed form (two rows a CTA and more)."""
    test_forward_without_codes(T, H, residual, wdt)


@pytest.mark.parametrize("T,H", [(20001, 128), (2003, 4096), (1300, 5120)])
def test_mx_codes_of_many_rows(T, H):
    test_mx_codes(T, H, 0, "rceil")


@pytest.mark.parametrize("T,H", [(20001, 128), (3001, 1000), (2003, 4096), (1300, 5120), (700, 8200)])
@pytest.mark.parametrize("dsum", [True, False])
def test_backward_of_many_rows(T, H, dsum):
    test_backward(T, H, dsum)


@pytest.mark.parametrize("T,H", [(1, 128), (5, 384), (130, 2048), (33, 5120), (256, 4096), (3, 16384)])
@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("mode", ["rceil", "floor"])
def test_mx_codes(T, H, dt, mode):
    from fp8_grouped_gemm_gb300 import mgq
    x, r, w = _inputs(T, H, T * H + dt)
    x[0, :32], r[0, :32] = 0.0, 0.0                          # an all-zero block
    codes = torch.full((T, H), 0xAB, dtype=torch.uint8, device="cuda")
    sc = torch.full((mgq.mx_scale_bytes(T, H),), 0xAB, dtype=torch.uint8, device="cuda")
    q = mgq.qdesc(dt, mgq.MX32_E8M0, codes, sc, e8m0_mode=mgq.RCEIL if mode == "rceil" else mgq.FLOOR)
    _run(x, r, w.bfloat16(), q)
    _, _, y = OB.rmsnorm(bf16_np(x), bf16_np(r), bf16_np(w.bfloat16()), EPS)
    fmt = ["e4m3", "e5m2"][dt]
    # scales: the oracle's for an amax anywhere within its error
    tiled = u8_np(sc)
    got = untile_mx_scales(tiled, T, H).astype(np.int64)
    lo = OQ.quantize_mx(y * (1 - 72 * U), fmt, mode)[1].astype(np.int64)
    hi = OQ.quantize_mx(y * (1 + 72 * U), fmt, mode)[1].astype(np.int64)
    assert np.all((got == lo) | (got == hi))
    rp = (T + 127) // 128 * 128
    assert np.all(untile_mx_scales(tiled, rp, H)[T:] == 0)
    # codes: cast with the kernel's own scale, monotone in y
    m = np.repeat(np.exp2(got - 127.0), 32, axis=1)
    _between(u8_np(codes), y / m, fmt)


def _between(codes, v, fmt):
    fmt = OF.FORMATS[fmt]
    val = OF.decode(codes, fmt)
    a = OF.decode(OF.encode(v * (1 - 72 * U), fmt), fmt)
    b = OF.decode(OF.encode(v * (1 + 72 * U), fmt), fmt)
    assert np.all((val >= np.minimum(a, b)) & (val <= np.maximum(a, b)))


@pytest.mark.parametrize("T,H", [(1, 128), (37, 640), (200, 4096)])
def test_blockwise_codes(T, H):
    from fp8_grouped_gemm_gb300 import mgq
    x, r, w = _inputs(T, H, T * H)
    x[0, :128], r[0, :128] = 0.0, 0.0
    codes = torch.empty(T, H, dtype=torch.uint8, device="cuda")
    sc = torch.empty(H // 128, T, device="cuda")
    _run(x, r, w, mgq.qdesc(mgq.E4M3, mgq.BLK_1x128_F32, codes, sc))
    _, _, y = OB.rmsnorm(bf16_np(x), bf16_np(r), w.double().numpy(), EPS)
    amax = np.abs(y).reshape(T, H // 128, 128).max(-1)
    inv = np.where(amax == 0, 1.0, amax / 448.0)
    got = sc.cpu().numpy().T.astype(np.float64)
    assert np.all(np.abs(got - inv) <= 76 * U * inv)            # two more divisions
    s = 1.0 / np.repeat(got, 128, axis=1)
    # the kernel multiplies by s, whose stored inverse is one rounding away
    v = y * s
    a = OF.decode(OF.encode(v * (1 - 80 * U), OF.E4M3), OF.E4M3)
    b = OF.decode(OF.encode(v * (1 + 80 * U), OF.E4M3), OF.E4M3)
    val = OF.decode(u8_np(codes), OF.E4M3)
    assert np.all((val >= np.minimum(a, b)) & (val <= np.maximum(a, b)))


@pytest.mark.parametrize("T,H,dt", [(1, 128, 0), (65, 1024, 1), (300, 4096, 0)])
def test_per_tensor_codes_and_amax(T, H, dt):
    from fp8_grouped_gemm_gb300 import mgq
    x, r, w = _inputs(T, H, T + H)
    codes = torch.empty(T, H, dtype=torch.uint8, device="cuda")
    ts, am = torch.full((1,), 3.7, device="cuda"), torch.zeros(1, device="cuda")
    _run(x, r, w, mgq.qdesc(dt, mgq.TENSOR_F32, codes, tensor_scale=ts, amax_out=am))
    _, _, y = OB.rmsnorm(bf16_np(x), bf16_np(r), w.double().numpy(), EPS)
    assert abs(am.item() - np.abs(y).max()) <= 72 * U * np.abs(y).max()
    _between(u8_np(codes), y * float(np.float32(3.7)), ["e4m3", "e5m2"][dt])
    # amax is raised, never lowered; the outputs that are not asked for are not needed
    am.fill_(1e9)
    mgq.add_rmsnorm_quantize(x.cuda(), w.cuda(), EPS, mgq.qdesc(dt, mgq.TENSOR_F32, codes, tensor_scale=ts, amax_out=am),
                             residual=r.cuda())
    assert am.item() == 1e9


def test_sum_in_place_of_the_residual_and_side_stream():
    from fp8_grouped_gemm_gb300 import mgq
    x, r, w = _inputs(50, 1024, 9)
    a = _run(x, r, w)
    xd, rd, wd, y = x.cuda(), r.cuda(), w.cuda(), torch.empty(50, 1024, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    mgq.add_rmsnorm_quantize(xd, wd, EPS, residual=rd, sum_out=rd, y=y, stream=st)
    st.synchronize()
    assert torch.equal(rd, a["sum_out"]) and torch.equal(y, a["y"])


def test_nan_and_infinity_stay_in_their_row():
    x, r, w = _inputs(6, 256, 4)
    x[2, 5], x[4, 7] = float("nan"), float("inf")
    o = _run(x, r, w)
    y = bf16_np(o["y"])
    assert np.all(np.isnan(y[2])) and np.isnan(y[4, 7])
    assert np.all(y[4, :7] == 0) and np.all(np.isfinite(y[[0, 1, 3, 5]]))


@pytest.mark.parametrize("T,H", [(1, 8), (2, 40), (5, 1000), (129, 2048), (333, 4096), (64, 5120), (3, 8200),
                                 (2, 16384)])
@pytest.mark.parametrize("dsum", [True, False])
def test_backward(T, H, dsum):
    from fp8_grouped_gemm_gb300 import mgq
    x, r, w = _inputs(T, H, 3 * T + H)
    g = torch.Generator().manual_seed(5)
    dy = torch.randn(T, H, generator=g).bfloat16()
    ds = torch.randn(T, H, generator=g).bfloat16() if dsum else None
    s = (x.float() + r.float()).bfloat16()
    s64, w64, dy64 = bf16_np(s), bf16_np(w.bfloat16()), bf16_np(dy)
    rstd = torch.from_numpy(1.0 / np.sqrt((s64 ** 2).mean(-1) + EPS)).float()
    rs = rstd.double().numpy()
    dx = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((H,), float("nan"), device="cuda")
    ws = torch.empty(max(16, mgq.add_rmsnorm_bwd_workspace_size(T, H)), dtype=torch.uint8, device="cuda")
    args = (dy.cuda(), s.cuda(), w.bfloat16().cuda(), rstd.cuda())
    mgq.add_rmsnorm_bwd(*args, dx, dw, ws, dsum=None if ds is None else ds.cuda())
    rx, rw = OB.rmsnorm_bwd(dy64, s64, w64, rs, None if ds is None else bf16_np(ds))
    xh, gg = s64 * rs[:, None], dy64 * w64
    slack = U * (rs[:, None] * (8 * np.abs(gg) + 72 * np.abs(xh) * np.abs(gg * xh).mean(-1, keepdims=True))
                 + 2 * np.abs(rx))
    _near_bf16(bf16_np(dx), rx, slack)
    mag = np.abs(dy64 * xh).sum(0)
    assert np.all(np.abs(dw.cpu().numpy() - rw) <= (T + 16) * U * mag + 1e-30)
    # accumulation, in-place dsum, and the same bits again
    dw2, acc = torch.empty_like(dw), torch.full((H,), 2.0, device="cuda")
    dx2 = torch.zeros_like(dx) if ds is None else ds.cuda()
    mgq.add_rmsnorm_bwd(*args, dx2, dw2, ws, dsum=None if ds is None else dx2)
    assert torch.equal(dw, dw2) and torch.equal(dx, dx2)
    mgq.add_rmsnorm_bwd(*args, dx, acc, ws, dsum=None if ds is None else ds.cuda(), beta=0.5)
    assert np.all(np.abs(acc.cpu().numpy() - (rw + 1.0)) <= (T + 20) * U * (mag + 1.0))


def test_backward_against_differences():
    """dx and dw against central differences of the float64 forward (bf16 output: 2^-8 of each value,
    and 2^-8 of the saved sum's own rounding is avoided by inputs that bf16 holds exactly)."""
    from fp8_grouped_gemm_gb300 import mgq
    rng = np.random.default_rng(3)
    T, H = 2, 16
    s = torch.from_numpy(rng.normal(size=(T, H))).bfloat16()
    w = torch.from_numpy(rng.normal(size=H)).float()
    dy = torch.from_numpy(rng.normal(size=(T, H))).bfloat16()
    s64, w64, dy64 = bf16_np(s), w.double().numpy(), bf16_np(dy)
    loss = lambda a, b: (OB.rmsnorm(a, None, b, EPS)[2] * dy64).sum()
    rstd = torch.from_numpy(OB.rmsnorm(s64, None, w64, EPS)[1]).float()
    dx, dw = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(H, device="cuda")
    ws = torch.empty(mgq.add_rmsnorm_bwd_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    mgq.add_rmsnorm_bwd(dy.cuda(), s.cuda(), w.cuda(), rstd.cuda(), dx, dw, ws)
    h = 1e-6
    for i in range(T):
        for j in range(H):
            e = np.zeros((T, H))
            e[i, j] = h
            d = (loss(s64 + e, w64) - loss(s64 - e, w64)) / (2 * h)
            assert abs(bf16_np(dx)[i, j] - d) <= 2.0 ** -8 * abs(d) + 1e-5
    for j in range(H):
        e = np.zeros(H)
        e[j] = h
        d = (loss(s64, w64 + e) - loss(s64, w64 - e)) / (2 * h)
        assert abs(dw[j].item() - d) <= 1e-5


def test_no_rows():
    from fp8_grouped_gemm_gb300 import mgq
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, device="cuda")
    mgq.add_rmsnorm_quantize(e, w, EPS, y=e)
    dw = torch.full((256,), 3.0, device="cuda")
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    mgq.add_rmsnorm_bwd(e, e, w, torch.empty(0, device="cuda"), e, dw, ws, beta=1.0)
    assert torch.all(dw == 3.0)
    mgq.add_rmsnorm_bwd(e, e, w, torch.empty(0, device="cuda"), e, dw, ws)
    assert torch.all(dw == 0.0)


def test_refusals_of_the_binding():
    from fp8_grouped_gemm_gb300 import mgq
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, device="cuda")
    y = torch.empty_like(x)

    def refused(status, **kw):
        a = dict(x=x, w=w, eps=EPS, y=y)
        a.update(kw)
        with pytest.raises(mgq.MGQError) as e:
            mgq.add_rmsnorm_quantize(**a)
        assert e.value.status == status

    refused(mgq.ERR_INVALID_ARG, x=x.t().contiguous().t())                  # strides
    refused(mgq.ERR_INVALID_ARG, x=x.float())                               # type
    refused(mgq.ERR_INVALID_ARG, y=torch.empty(4, 128, dtype=torch.bfloat16, device="cuda"))
    refused(mgq.ERR_INVALID_ARG, x=x.cpu())                                 # place
    refused(mgq.ERR_UNSUPPORTED, w=w.half())
    refused(mgq.ERR_INVALID_ARG, y=None)                                    # nothing to write


def test_two_threads_with_rows_of_different_length():
    """Two host threads, streams of their own, one kernel and rings of 128 KB and more beside small ones."""
    import threading
    from fp8_grouped_gemm_gb300 import mgq
    failed = []

    def work(T, H):
        x, w = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), torch.ones(H, device="cuda")
        y, st = torch.empty_like(x), torch.cuda.Stream()
        dw, ws = torch.empty(H, device="cuda"), torch.empty(mgq.add_rmsnorm_bwd_workspace_size(T, H), dtype=torch.uint8,
                                                            device="cuda")
        rstd = torch.ones(T, device="cuda")
        torch.cuda.synchronize()
        start.wait()
        try:
            for _ in range(3000):
                mgq.add_rmsnorm_quantize(x, w, EPS, y=y, stream=st)
                mgq.add_rmsnorm_bwd(x, x, w, rstd, y, dw, ws, stream=st)
        except mgq.MGQError as e:
            failed.append((H, e))
        st.synchronize()

    start = threading.Barrier(2)
    threads = [threading.Thread(target=work, args=a) for a in ((5000, 2176), (700, 8192))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


# ---- enough rows for the streamed form, in every scaling -----------------------------

@pytest.mark.parametrize("T,H", [(20001, 128), (2003, 4096), (1300, 5120), (700, 16384)])
def test_blockwise_codes_of_many_rows(T, H):
    test_blockwise_codes(T, H)


@pytest.mark.parametrize("T,H,dt", [(20001, 128, 0), (2003, 4096, 1), (1300, 5120, 0), (700, 16384, 1)])
def test_per_tensor_codes_of_many_rows(T, H, dt):
    test_per_tensor_codes_and_amax(T, H, dt)


@pytest.mark.parametrize("T,H,dt,mode", [(2003, 4096, 1, "floor"), (1300, 5120, 1, "rceil"), (5003, 1024, 0, "floor")])
def test_mx_codes_of_many_rows_other_formats(T, H, dt, mode):
    test_mx_codes(T, H, dt, mode)


def _codes(T, H, scaling, dt=0):
    """(QDesc, its output tensors)"""
    from fp8_grouped_gemm_gb300 import mgq
    c = torch.full((T, H), 0xAB, dtype=torch.uint8, device="cuda")
    if scaling == "mx":
        s = torch.full((mgq.mx_scale_bytes(T, H),), 0xAB, dtype=torch.uint8, device="cuda")
        return mgq.qdesc(dt, mgq.MX32_E8M0, c, s), (c, s)
    if scaling == "blk":
        s = torch.full((H // 128, T), 7.0, device="cuda")
        return mgq.qdesc(dt, mgq.BLK_1x128_F32, c, s), (c, s)
    ts, am = torch.full((1,), 3.7, device="cuda"), torch.zeros(1, device="cuda")
    return mgq.qdesc(dt, mgq.TENSOR_F32, c, tensor_scale=ts, amax_out=am), (c, ts, am)


@pytest.mark.parametrize("scaling", ["mx", "blk", "tensor"])
def test_outputs_at_odd_16_byte_addresses(scaling):
    """bf16 outputs that are 16-byte but not 32-byte aligned, and sum_out in place of x: the same bits."""
    T, H = 2003, 1152
    x, r, w = _inputs(T, H, 21)
    q, a = _codes(T, H, scaling)
    ref = _run(x, r, w, q)
    from fp8_grouped_gemm_gb300 import mgq
    q, b = _codes(T, H, scaling)
    at = lambda: torch.full((T * H + 8,), 7.0, dtype=torch.bfloat16, device="cuda")[8:].view(T, H)
    y, s = at(), at()
    s.copy_(x)
    assert y.data_ptr() % 32 == 16
    mgq.add_rmsnorm_quantize(s, w.cuda(), EPS, q, residual=r.cuda(), sum_out=s, y=y)
    torch.cuda.synchronize()
    assert torch.equal(y, ref["y"]) and torch.equal(s, ref["sum_out"])
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("T", [9, 2003])
@pytest.mark.parametrize("scaling", ["mx", "blk", "tensor"])
def test_nan_and_infinity_with_codes_stay_in_their_row(T, scaling):
    """A NaN in a row makes all of its codes NaN, an infinity those of its block (the rest of
    y is 0); the codes and scales of other rows keep their bits."""
    H = 1152
    x, r, w = _inputs(T, H, 22)
    q, a = _codes(T, H, scaling)
    _run(x, r, w, q)
    bad = x.clone()
    bad[2, 5], bad[4, 7] = float("nan"), float("inf")
    q, b = _codes(T, H, scaling)
    _run(bad, r, w, q)
    rest = [t for t in range(T) if t not in (2, 4)]
    assert torch.equal(a[0][rest], b[0][rest])
    nan = (b[0] & 0x7F) == 0x7F                      # e4m3
    assert torch.all(nan[2]) and nan[4, 7]
    span = {"mx": 32, "blk": 128, "tensor": 1}[scaling]
    lo = 7 // span * span
    assert torch.all(nan[4, lo:lo + span])
    assert torch.all((b[0][4, lo + span:] & 0x7F) == 0)
    if scaling == "mx":
        u, v = (untile_mx_scales(u8_np(s), T, H) for s in (a[1], b[1]))
        assert np.array_equal(u[rest], v[rest]) and np.all(v[2] == 255) and v[4, 0] == 255 and np.all(v[4, 1:] == 0)
    elif scaling == "blk":
        assert torch.equal(a[1][:, rest], b[1][:, rest]) and torch.all(torch.isnan(b[1][:, 2]))
        assert torch.isnan(b[1][0, 4]) and torch.all(b[1][1:, 4] == 1.0)
    else:
        assert torch.isnan(b[2][0])
