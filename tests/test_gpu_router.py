"""GPU parity of the top-k router and its gradient with the float64 definitions.

Ids are equal. With u = 2^-24: a score is an exponential (2 ulp) over a sum of
at most 32 serial terms and a tree of the lanes, so probabilities are within
64 u; a gradient is within 96 u of the sum of the magnitudes it is made of
(and, for bf16 logits, half a bf16 ulp)."""
import numpy as np
import pytest
import torch

from oracle import block as OB
from tests.layer_check import ulp_bf16

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _mode(score):
    from fp8_grouped_gemm_gb300 import mgq
    return mgq.SCORE_SOFTMAX if score == "softmax" else mgq.SCORE_SIGMOID


def _check(logits, k, score, renorm, scale=1.0, seed=0):
    from fp8_grouped_gemm_gb300 import mgq
    T, E = logits.shape
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    probs = torch.full((T, k), 7.0, device="cuda")
    dp = torch.randn(T, k, generator=torch.Generator().manual_seed(seed))
    dl = torch.full((T, E), 7.0, dtype=logits.dtype, device="cuda")
    ld = logits.cuda()
    mgq.router_topk(ld, idx, probs, _mode(score), renorm, scale)
    mgq.router_topk_bwd(ld, idx, dp.cuda(), dl, _mode(score), renorm, scale)
    assert mgq.get_error() == mgq.OK
    l64 = logits.double().numpy()
    sc = float(np.float32(scale))
    ri, rp = OB.router_topk(l64, k, score, renorm, sc)
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert np.all(np.abs(probs.cpu().numpy() - rp) <= 64 * U * np.abs(rp) + 1e-37)
    rg, mag = OB.router_topk_bwd(l64, ri, dp.double().numpy(), score, renorm, sc)
    slack = 96 * U * mag + 1e-37
    if logits.dtype == torch.bfloat16:
        slack = slack + 0.5 * ulp_bf16(np.abs(rg) + slack) * (1 + 1e-9)
    assert np.all(np.abs(dl.double().cpu().numpy() - rg) <= slack)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (17, 8, 8), (9, 31, 3), (40, 64, 6), (7, 65, 1),
                                   (33, 128, 8), (5, 129, 4), (6, 256, 8), (4, 300, 8), (3, 1024, 7)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_router(T, E, k, score, renorm, dtype):
    g = torch.Generator().manual_seed(T * E + k)
    _check((torch.randn(T, E, generator=g) * 3).to(dtype), k, score, renorm, 2.5, E)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_ties_masks_and_extremes(score, renorm):
    inf, big = float("inf"), 3.4028234e38
    rows = [[1.0, 2.0, 2.0, 2.0, 0.0, -0.0],
            [0.0, -0.0, 0.0, -0.0, -1.0, -inf],
            [-inf, -inf, 3.0, -inf, -inf, -inf],
            [-inf] * 6,
            [float("nan"), 1.0, float("nan"), 2.0, -inf, 0.5],
            [-big] * 6,
            [90.0, -90.0, 100.0, -100.0, 0.0, 80.0],
            [1e-40, -1e-40, 0.0, 2e-40, -inf, -inf]]
    _check(torch.tensor(rows), 4, score, renorm)


def test_many_rows_and_a_side_stream():
    """More rows than the grid has warps, on another stream than the tensors'."""
    from fp8_grouped_gemm_gb300 import mgq
    T, E, k = 20000, 16, 2
    l = torch.randn(T, E, generator=torch.Generator().manual_seed(1))
    l = (l * 4).round() / 4                                 # ties in most rows
    _check(l, k, "softmax", True)
    ld = l.cuda()
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    probs = torch.empty(T, k, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mgq.router_topk(ld, idx, probs, stream=s)
    s.synchronize()
    assert np.array_equal(idx.cpu().numpy(), OB.router_topk(l.double().numpy(), k)[0])


@pytest.mark.parametrize("E,k", [(2, 1), (8, 8), (31, 3), (33, 8), (64, 6), (100, 8), (128, 8), (129, 4), (256, 8),
                                 (300, 5), (512, 8), (640, 8)])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
@pytest.mark.parametrize("dtype,shift", [(torch.float32, 0), (torch.bfloat16, 0), (torch.float32, 1)])
def test_a_row_is_the_same_in_any_batch(E, k, score, renorm, dtype, shift):
    """5003 rows at once (lanes share a warp's rows) and 100 at a time (a warp a
    row): the same bits, with ties, masked experts and NaN in some rows; rows
    at odd addresses (shift) as well."""
    from fp8_grouped_gemm_gb300 import mgq
    T = 5003
    g = torch.Generator().manual_seed(E + k)
    x = torch.randn(T, E, generator=g)
    x[::3] = (x[::3] * 2).round()                                      # ties
    x[1::7] = torch.where(torch.rand(x[1::7].shape, generator=g) < 0.5, -torch.inf, x[1::7])
    x[5::50] = -torch.inf
    x[6::50] = torch.nan
    x[7::50] = 0.0
    x[7::100] *= -1
    x[8::50, E // 2] = torch.inf
    flat = torch.empty(T * E + 1, dtype=dtype, device="cuda")
    logits = flat[shift:shift + T * E].view(T, E)
    logits.copy_(x.to(dtype))
    def route(l):
        i = torch.full((l.shape[0], k), -7, dtype=torch.int32, device="cuda")
        p = torch.full((l.shape[0], k), 7.0, device="cuda")
        mgq.router_topk(l, i, p, _mode(score), renorm, 1.5)
        return i, p
    i, p = route(logits)
    parts = [route(logits[t:t + 100]) for t in range(0, T, 100)]
    assert torch.equal(i, torch.cat([a for a, _ in parts]))
    assert torch.equal(p.view(torch.int32), torch.cat([b for _, b in parts]).view(torch.int32))
    clean = torch.nan_to_num(logits[:301].float().cpu(), nan=-torch.inf, posinf=torch.inf, neginf=-torch.inf)
    with np.errstate(invalid="ignore"):      # a logit of infinity has no softmax; its rank is looked at
        ri, _ = OB.router_topk(clean.double().numpy(), k, score, renorm, 1.5)
    assert np.array_equal(i[:301].cpu().numpy(), ri)


def test_probabilities_feed_the_unpermute_and_its_gradient_comes_back():
    """dprobs of mgq_moe_unpermute_bwd is what the router's backward takes: shapes and types as they are."""
    from fp8_grouped_gemm_gb300 import mgq
    l = torch.randn(12, 8, device="cuda")
    idx = torch.empty(12, 2, dtype=torch.int32, device="cuda")
    p = torch.empty(12, 2, device="cuda")
    mgq.router_topk(l, idx, p)
    assert torch.all((p.sum(1) - 1).abs() < 1e-6)


def test_gradient_against_differences():
    rng = np.random.default_rng(5)
    from fp8_grouped_gemm_gb300 import mgq
    l, d = rng.normal(size=(3, 9)), rng.normal(size=(3, 3))
    l, d = l.astype(np.float32), d.astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            idx = torch.empty(3, 3, dtype=torch.int32, device="cuda")
            p, dl = torch.empty(3, 3, device="cuda"), torch.empty(3, 9, device="cuda")
            ld = torch.from_numpy(l).cuda()
            mgq.router_topk(ld, idx, p, _mode(score), renorm)
            mgq.router_topk_bwd(ld, idx, torch.from_numpy(d).cuda(), dl, _mode(score), renorm)
            f = lambda v: (OB.router_topk(v, 3, score, renorm)[1] * d).sum()
            h = 1e-6
            for i in range(3):
                for j in range(9):
                    e = np.zeros((3, 9))
                    e[i, j] = h
                    diff = (f(l + e) - f(l - e)) / (2 * h)
                    assert abs(dl[i, j].item() - diff) <= 1e-6


def test_an_id_out_of_range_is_reported():
    from fp8_grouped_gemm_gb300 import mgq
    l = torch.randn(2, 4, device="cuda")
    idx = torch.tensor([[0, 9], [1, 2]], dtype=torch.int32, device="cuda")
    dl = torch.empty(2, 4, device="cuda")
    mgq.router_topk_bwd(l, idx, torch.ones(2, 2, device="cuda"), dl, renorm=False)
    assert mgq.get_error() == mgq.ERR_DEVICE_INDEX
    assert mgq.get_error() == mgq.OK
    assert torch.all(torch.isfinite(dl))


def test_refusals_of_the_binding():
    from fp8_grouped_gemm_gb300 import mgq
    l = torch.zeros(4, 16, device="cuda")
    idx = torch.empty(4, 2, dtype=torch.int32, device="cuda")
    p = torch.empty(4, 2, device="cuda")
    for bad in (dict(logits=l.t().contiguous().t()), dict(topk_idx=idx.long()), dict(probs=p[:3]),
                dict(logits=l[:, :1].contiguous())):
        a = dict(logits=l, topk_idx=idx, probs=p)
        a.update(bad)
        with pytest.raises(mgq.MGQError) as e:
            mgq.router_topk(**a)
        assert e.value.status == mgq.ERR_INVALID_ARG
    with pytest.raises(mgq.MGQError) as e:
        mgq.router_topk(l.half(), idx, p)
    assert e.value.status == mgq.ERR_UNSUPPORTED
    mgq.router_topk(l[:0], idx[:0], p[:0])                 # no rows


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_the_unpermute_reaches_the_logits(renorm):
    """out = sum_j p_j y_j through mgq_moe_unpermute; dprobs from mgq_moe_unpermute_bwd
    into the router's gradient, against the formula on the same y and dout."""
    from fp8_grouped_gemm_gb300 import mgq
    from tests.layer_check import bf16_np
    T, E, k, H = 40, 8, 2, 256
    g = torch.Generator().manual_seed(3)
    l = torch.randn(T, E, generator=g)
    ld = l.cuda()
    idx, p = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    mgq.router_topk(ld, idx, p, renorm=renorm)
    R = mgq.r_cap(T, k, E, 128)
    i32 = dict(dtype=torch.int32, device="cuda")
    rim, src, off, cnt = torch.empty(T, k, **i32), torch.empty(R, **i32), torch.empty(E + 1, **i32), torch.empty(E, **i32)
    ws = torch.empty(max(16, mgq.permute_workspace_size(T, k, E)), dtype=torch.uint8, device="cuda")
    mgq.moe_route(idx, E, 128, R, rim, src, off, cnt, ws)
    y = torch.randn(R, H, generator=g).bfloat16().cuda()
    dout = torch.randn(T, H, generator=g).bfloat16().cuda()
    codes, sc = torch.empty(R, H, dtype=torch.uint8, device="cuda"), torch.empty(mgq.mx_scale_bytes(R, H), dtype=torch.uint8,
                                                                               device="cuda")
    dp, dl = torch.empty(T, k, device="cuda"), torch.empty(T, E, device="cuda")
    mgq.moe_unpermute_bwd(dout, y, rim, src, p, R, off, E, mgq.qdesc(mgq.E5M2, mgq.MX32_E8M0, codes, sc), dp)
    mgq.router_topk_bwd(ld, idx, dp, dl, renorm=renorm)
    assert mgq.get_error() == mgq.OK
    y64, d64, rows = bf16_np(y), bf16_np(dout), rim.cpu().numpy()
    terms = y64[rows] * d64[:, None, :]
    ref, mag = terms.sum(-1), np.abs(terms).sum(-1)
    # 256 terms in float32, in any order
    assert np.all(np.abs(dp.double().cpu().numpy() - ref) <= 256 * U * mag)
    rl, m = OB.router_topk_bwd(l.double().numpy(), idx.cpu().numpy(), ref, "softmax", renorm, 1.0)
    _, m2 = OB.router_topk_bwd(l.double().numpy(), idx.cpu().numpy(), mag, "softmax", renorm, 1.0)
    assert np.all(np.abs(dl.double().cpu().numpy() - rl) <= 96 * U * m + 256 * U * m2 + 1e-37)
