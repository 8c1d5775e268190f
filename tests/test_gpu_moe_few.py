"""GPU parity of the expert layer for a few tokens with the float64 definition.

The oracle's and the kernel's g and u differ by float32 summation (about 1e-6
of their size), so a code of h lies on the other side of a rounding boundary
about once in 10^4 values (a step of 1/8 or less of the value for e4m3, 1/3 for
e2m1): 2e-3 of a row's norm at most for e4m3 and 5e-3 for e2m1. A bf16 output
adds 2^-9 relative. Per row the bound is 4e-3 (e2m1: 8e-3) of the row's norm.
Those are averages over a row's codes; a row whose largest value or block scale
sits on a rounding boundary is further off by that one step. The definition
leaves such a row two answers as far as float32 goes, so a row may match the
oracle for h as it is or for h changed by 4e-6 of itself either way."""
import numpy as np
import pytest
import torch

from oracle import block as OB
from oracle import quant as OQ
from tests.layer_check import bf16_np, tile_mx_scales

pytestmark = pytest.mark.gpu
RECIPES = ("mxfp8", "blockwise", "delayed", "nvfp4")
XS, HS = {"delayed": 3.0, "nvfp4": 11.03}, {"delayed": 7.0, "nvfp4": 6.7}
TOL = {"mxfp8": 4e-3, "blockwise": 4e-3, "delayed": 4e-3, "nvfp4": 8e-3}


def _weight(E, N, K, recipe, rng, ld=None):
    """(operand tensors, float64 values) of a random quantised weight [E, N, K]."""
    from fp8_grouped_gemm_gb300 import mgq
    w = rng.normal(size=(E, N, K)) * 0.1
    if recipe == "mxfp8":
        c, s = OQ.quantize_mx(w.reshape(E * N, K), "e4m3")
        v = OQ.dequantize_mx(c, s).reshape(E, N, K)
        t = dict(data=c, scale=tile_mx_scales(s))
    elif recipe == "nvfp4":
        cs, ss, sg, v = [], [], np.empty(E, np.float32), np.empty((E, N, K))
        for e in range(E):
            sg[e] = OQ.nvfp4_global_scale(np.abs(w[e]).max())
            c, s = OQ.quantize_nvfp4(w[e], sg[e])
            v[e] = OQ.dequantize_nvfp4(c, s, sg[e], K)
            cs.append(c)
            ss.append(s)
        t = dict(data=np.stack(cs), scale=tile_mx_scales(np.concatenate(ss)), global_scale=sg)
    elif recipe == "blockwise":
        cs, ss, v = [], [], np.empty((E, N, K))
        for e in range(E):
            c, s = OQ.quantize_block_128x128(w[e], "e4m3")
            v[e] = OQ.dequantize_block_128x128(c, s)
            cs.append(c)
            ss.append(s)
        t = dict(data=np.stack(cs), scale=np.stack(ss).astype(np.float32))
    else:
        s = (448.0 / np.abs(w).max((1, 2))).astype(np.float32)
        c = np.stack([OQ.quantize_tensor(w[e], s[e])[0] for e in range(E)])
        v = np.stack([OQ.dequantize_tensor(c[e], s[e]) for e in range(E)])
        t = dict(data=c, scale=s)
    t = {n: torch.from_numpy(np.ascontiguousarray(a)).cuda() for n, a in t.items()}
    dt = mgq.E2M1 if recipe == "nvfp4" else mgq.E4M3
    return t, mgq.operand(t["data"], t["scale"], K, dt, t.get("global_scale")), v


def _scaling(recipe):
    from fp8_grouped_gemm_gb300 import mgq
    return {"mxfp8": mgq.MX32_E8M0, "blockwise": mgq.BLK_1x128_F32, "delayed": mgq.TENSOR_F32,
            "nvfp4": mgq.NV16_UE4M3}[recipe]


def _call(x, idx, p, W1, W2, recipe, E, F, stream=None, ws=None, out=None):
    from fp8_grouped_gemm_gb300 import mgq
    T, H = x.shape
    k = idx.shape[1]
    if ws is None:
        ws = torch.full((mgq.moe_few_workspace_size(T, k, E, H, F, _scaling(recipe)),), 0xFF, dtype=torch.uint8,
                        device="cuda")
    if out is None:
        out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    sc = lambda d: torch.full((1,), d[recipe], device="cuda") if recipe in d else None
    xs, hs = sc(XS), sc(HS)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    mgq.moe_few_forward(x, idx, p, W1, W2, _scaling(recipe), E, F, out, ws, xs, hs, stream=stream)
    torch.cuda.synchronize()
    assert mgq.get_error() == mgq.OK
    return out


def _routing(T, E, k, rng, hot=None):
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    if hot is not None:                    # one expert in every token
        idx = np.where(idx == hot, idx[:, :1], idx)
        idx[:, 0] = hot
    p = rng.random((T, k)).astype(np.float32)
    return idx, p / p.sum(1, keepdims=True)


def _rows_close(out, x, idx, p, v1, v2, recipe, rows=slice(None), scales=None):
    xs, hs = scales or (XS.get(recipe), HS.get(recipe))
    got = bf16_np(out)[rows]
    least = None
    for nudge in (0.0, 4e-6, -4e-6):
        ref = OB.moe_few(bf16_np(x), idx, p, v1, v2, recipe, xs, hs, nudge)[rows]
        err = np.linalg.norm(got - ref, axis=1) / np.maximum(np.linalg.norm(ref, axis=1), 1e-30)
        least = err if least is None else np.minimum(least, err)
    assert np.all(least <= TOL[recipe]), (np.argmax(least), least.max())


SHAPES = [(8, 16, 8, 512, 1024), (8, 1, 1, 256, 512), (9, 16, 8, 512, 1024), (4, 64, 8, 2048, 768), (7, 8, 2, 1280, 256),
          (1, 4, 2, 256, 256), (1, 8, 1, 512, 768), (2, 3, 3, 768, 256), (5, 16, 4, 512, 512), (16, 4, 2, 1024, 256),
          (17, 8, 2, 256, 1536), (33, 5, 1, 512, 512), (64, 32, 8, 256, 256), (100, 2, 2, 256, 512),
          (128, 7, 3, 512, 256), (128, 64, 8, 256, 256)]


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("T,E,k,H,F", SHAPES)
def test_layer(recipe, T, E, k, H, F):
    rng = np.random.default_rng(T * E + H)
    x = torch.from_numpy(rng.normal(size=(T, H))).bfloat16()
    idx, p = _routing(T, E, k, rng)
    t1, W1, v1 = _weight(E, 2 * F, H, recipe, rng)
    t2, W2, v2 = _weight(E, H, F, recipe, rng)
    out = _call(x.cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(p).cuda(), W1, W2, recipe, E, F)
    _rows_close(out, x, idx, p, v1, v2, recipe)


@pytest.mark.parametrize("recipe", RECIPES[:3])
@pytest.mark.parametrize("T,E,k,H,F", [(3, 4, 2, 128, 128), (1, 2, 1, 384, 640), (9, 4, 2, 384, 640), (70, 3, 1, 640, 128)])
def test_odd_multiples_of_128(recipe, T, E, k, H, F):
    """The last tile of W2 has one half only."""
    test_layer(recipe, T, E, k, H, F)


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("T,E,k,H,F", [(2, 2, 2, 4096, 256), (1, 4, 2, 4352, 256), (3, 3, 3, 4352, 512), (8, 2, 1, 4608, 256),
                                       (8, 1, 1, 256, 9728), (1, 1, 1, 256, 9984), (2, 3, 2, 512, 7424)])
def test_few_tokens_with_long_rows(recipe, T, E, k, H, F):
    """Either side of the lengths at which few tokens change the form."""
    test_layer(recipe, T, E, k, H, F)


@pytest.mark.parametrize("recipe", RECIPES)
def test_every_token_on_one_expert(recipe):
    """128 tokens of one expert: two token blocks of the same weights."""
    rng = np.random.default_rng(11)
    T, E, k, H, F = 128, 6, 2, 256, 256
    x = torch.from_numpy(rng.normal(size=(T, H))).bfloat16()
    idx, p = _routing(T, E, k, rng, hot=3)
    t1, W1, v1 = _weight(E, 2 * F, H, recipe, rng)
    t2, W2, v2 = _weight(E, H, F, recipe, rng)
    out = _call(x.cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(p).cuda(), W1, W2, recipe, E, F)
    _rows_close(out, x, idx, p, v1, v2, recipe)


@pytest.mark.parametrize("recipe", RECIPES)
def test_same_bits_again_batch_neighbours_and_streams(recipe):
    """The same call gives the same bits, with a dirty or a used workspace, on a
    side stream and in a captured graph; zero and NaN rows stay their own."""
    from fp8_grouped_gemm_gb300 import mgq
    rng = np.random.default_rng(12)
    T, E, k, H, F = 20, 8, 2, 512, 512
    x = torch.from_numpy(rng.normal(size=(T, H))).bfloat16()
    x[3] = 0.0
    idx, p = _routing(T, E, k, rng)
    t1, W1, v1 = _weight(E, 2 * F, H, recipe, rng)
    t2, W2, v2 = _weight(E, H, F, recipe, rng)
    xd, di, dp = x.cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(p).cuda()
    ws = torch.zeros(mgq.moe_few_workspace_size(T, k, E, H, F, _scaling(recipe)), dtype=torch.uint8, device="cuda")
    a = _call(xd, di, dp, W1, W2, recipe, E, F, ws=ws)
    assert torch.all(a[3] == 0)
    for _ in range(3):
        assert torch.equal(a, _call(xd, di, dp, W1, W2, recipe, E, F, ws=ws))
    assert torch.equal(a, _call(xd, di, dp, W1, W2, recipe, E, F))
    assert torch.equal(a, _call(xd, di, dp, W1, W2, recipe, E, F, stream=torch.cuda.Stream()))
    xn = xd.clone()
    xn[5] = float("nan")
    b = _call(xn, di, dp, W1, W2, recipe, E, F)
    rest = [t for t in range(T) if t != 5]
    assert torch.equal(a[rest], b[rest])
    if recipe != "nvfp4":                       # (e2m1 has no NaN)
        assert torch.all(torch.isnan(b[5]))
    sc = lambda d: torch.full((1,), d[recipe], device="cuda") if recipe in d else None
    xs, hs, out = sc(XS), sc(HS), torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mgq.moe_few_forward(xd, di, dp, W1, W2, _scaling(recipe), E, F, out, ws, xs, hs)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, out)


@pytest.mark.parametrize("recipe", ["mxfp8", "nvfp4"])
def test_many_experts(recipe):
    """The largest expert count, nearly all of them empty."""
    rng = np.random.default_rng(13)
    T, E, k, H, F = 3, 1024, 8, 256, 256
    x = torch.from_numpy(rng.normal(size=(T, H))).bfloat16()
    idx, p = _routing(T, E, k, rng)
    used = np.unique(idx)
    t1, W1, v1 = _weight(used.size, 2 * F, H, recipe, rng)
    t2, W2, v2 = _weight(used.size, H, F, recipe, rng)

    def spread(t, per):     # the used experts' weights at their places in the full tensors
        out = {}
        for n, a in t.items():
            rows = a.reshape(used.size, -1)
            full = torch.zeros(E, rows.shape[1], dtype=a.dtype, device="cuda")
            full[torch.from_numpy(used).long().cuda()] = rows
            out[n] = full
        return out

    from fp8_grouped_gemm_gb300 import mgq
    f1, f2 = spread(t1, 2 * F), spread(t2, H)
    dt = mgq.E2M1 if recipe == "nvfp4" else mgq.E4M3
    O1 = mgq.operand(f1["data"], f1["scale"], H, dt, f1.get("global_scale"))
    O2 = mgq.operand(f2["data"], f2["scale"], F, dt, f2.get("global_scale"))
    out = _call(x.cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(p).cuda(), O1, O2, recipe, E, F)
    local = np.searchsorted(used, idx)
    _rows_close(out, x, local, p, v1, v2, recipe)


def test_ids_out_of_range_contribute_nothing_and_are_reported():
    from fp8_grouped_gemm_gb300 import mgq
    rng = np.random.default_rng(14)
    T, E, k, H, F = 4, 4, 2, 256, 256
    x = torch.from_numpy(rng.normal(size=(T, H))).bfloat16()
    idx, p = _routing(T, E, k, rng)
    idx[1, 0], idx[2] = 9, -1
    t1, W1, v1 = _weight(E, 2 * F, H, "mxfp8", rng)
    t2, W2, v2 = _weight(E, H, F, "mxfp8", rng)
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(mgq.moe_few_workspace_size(T, k, E, H, F, mgq.MX32_E8M0), dtype=torch.uint8, device="cuda")
    mgq.moe_few_forward(x.cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(p).cuda(), W1, W2, mgq.MX32_E8M0, E, F,
                        out, ws)
    assert mgq.get_error() == mgq.ERR_DEVICE_INDEX
    assert torch.all(out[2] == 0)
    _rows_close(out, x, idx, p, v1, v2, "mxfp8", [0, 1, 3])


def test_agrees_with_the_grouped_layer():
    """The same quantised weights through the many-token path: its h and y are
    rounded to bf16 on the way (2^-9 each, and the codes of h that this flips)."""
    from fp8_grouped_gemm_gb300 import layer as L
    from fp8_grouped_gemm_gb300 import mgq
    from fp8_grouped_gemm_gb300 import workloads as W
    w = W.WORKLOADS["tiny"].scaled(T=48)
    lay = L.ExpertLayer(w, "cuda:0")
    w1, w2 = W.make_weights(w)
    idx, probs = (torch.from_numpy(a).cuda() for a in W.make_routing(w))
    x = W.make_activations(w).cuda()
    lay.quantize_weights(w1.cuda(), w2.cuda())
    ref = bf16_np(lay.forward(x, idx, probs))
    out = torch.empty_like(x)
    ws = torch.empty(mgq.moe_few_workspace_size(w.T, w.k, w.E, w.H, w.F, lay.scaling), dtype=torch.uint8, device="cuda")
    mgq.moe_few_forward(x, idx, probs, mgq.operand(lay.w1q, lay.w1s, w.H, mgq.E4M3),
                        mgq.operand(lay.w2q, lay.w2s, w.F, mgq.E4M3), lay.scaling, w.E, w.F, out, ws)
    got = bf16_np(out)
    # a 2^-9 change of h moves one code in about 2^-9 / 2^-4 by 1/16..1/8: 0.03 * 0.1^2 -> 2e-2
    assert np.linalg.norm(got - ref) <= 2e-2 * np.linalg.norm(ref)


def test_refusals_of_the_binding():
    from fp8_grouped_gemm_gb300 import mgq
    T, E, k, H, F = 4, 4, 2, 256, 256
    rng = np.random.default_rng(15)
    t1, W1, _ = _weight(E, 2 * F, H, "mxfp8", rng)
    t2, W2, _ = _weight(E, H, F, "mxfp8", rng)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    a = dict(x=x, topk_idx=torch.zeros(T, k, dtype=torch.int32, device="cuda"), probs=torch.zeros(T, k, device="cuda"),
             W1=W1, W2=W2, scaling=mgq.MX32_E8M0, E=E, F=F, out=torch.empty_like(x),
             workspace=torch.empty(mgq.moe_few_workspace_size(T, k, E, H, F, mgq.MX32_E8M0), dtype=torch.uint8,
                                   device="cuda"))
    for bad in (dict(x=x.float()), dict(out=x[:2]), dict(probs=a["probs"].double()), dict(topk_idx=a["topk_idx"].long()),
                dict(workspace=a["workspace"][:-256]), dict(F=F + 1), dict(x=x.t().contiguous().t())):
        with pytest.raises(mgq.MGQError) as e:
            mgq.moe_few_forward(**{**a, **bad})
        assert e.value.status == mgq.ERR_INVALID_ARG, bad.keys()
    empty = dict(x=x[:0], out=x[:0], topk_idx=a["topk_idx"][:0], probs=a["probs"][:0])
    mgq.moe_few_forward(**{**a, **empty})


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("T,E,k,H,F", [(8, 8, 8, 256, 256), (3, 4, 2, 512, 512), (1, 16, 8, 256, 256), (16, 8, 8, 256, 512),
                                       (9, 8, 4, 512, 256), (40, 3, 3, 256, 256), (4, 8, 8, 1024, 1280)])
@pytest.mark.parametrize("rows", ["all", "some"])
def test_an_expert_named_twice_by_a_token(recipe, T, E, k, H, F, rows):
    """Padding of a batch names one expert k times (ids all 0): each mention
    counts with its probability, and nothing is written behind the workspace."""
    from fp8_grouped_gemm_gb300 import mgq
    rng = np.random.default_rng(T + k)
    x = torch.from_numpy(rng.normal(size=(T, H))).bfloat16()
    idx, p = _routing(T, E, k, rng)
    if rows == "all":
        idx[:] = 0
    else:
        idx[::2, 1] = idx[::2, 0]
        idx[T // 2] = E - 1
    t1, W1, v1 = _weight(E, 2 * F, H, recipe, rng)
    t2, W2, v2 = _weight(E, H, F, recipe, rng)
    n, guard = mgq.moe_few_workspace_size(T, k, E, H, F, _scaling(recipe)), 1 << 20
    ws = torch.full((n + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    args = (x.cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(p).cuda(), W1, W2, recipe, E, F)
    out = _call(*args, ws=ws[:n])
    assert torch.all(ws[n:] == 0xA5)
    _rows_close(out, x, idx, p, v1, v2, recipe)
    assert torch.equal(out, _call(*args, ws=ws[:n]))


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("H,F", [(512, 512), (1024, 768)])
def test_a_token_alone_and_in_batches(recipe, H, F):
    """The same rows in batches of 1, 8, 9 and 128 (both forms, other splits of the
    sums). The scales of x and the codes of x are the same; sums that differ by
    1e-6 of themselves move a code of h once in 10^4, and a row has 10^3: most rows
    differ by the bf16 rounding alone (2^-8 of a value), nine in ten by no more than
    two answers within the definition's bound can, and any by one step of an element
    or a block (1/8 of it, e2m1 1/3) that holds half of the row's norm."""
    rng = np.random.default_rng(H)
    T, E, k = 128, 8, 2
    x = torch.from_numpy(rng.normal(size=(T, H))).bfloat16().cuda()
    idx, p = (torch.from_numpy(a).cuda() for a in _routing(T, E, k, rng))
    t1, W1, _ = _weight(E, 2 * F, H, recipe, rng)
    t2, W2, _ = _weight(E, H, F, recipe, rng)
    run = lambda a, b: bf16_np(_call(x[a:b].contiguous(), idx[a:b].contiguous(), p[a:b].contiguous(), W1, W2, recipe, E, F))
    whole = run(0, T)
    for n in (1, 8, 9):
        part = np.concatenate([run(a, a + n) for a in range(0, 72, n)])
        err = np.linalg.norm(part - whole[:72], axis=1) / np.linalg.norm(whole[:72], axis=1)
        assert np.median(err) <= 2.0 ** -8, (n, np.median(err))
        assert np.quantile(err, 0.9) <= 2 * TOL[recipe], (n, np.quantile(err, 0.9))
        assert err.max() <= (1 / 6 if recipe == "nvfp4" else 1 / 16), (n, err.max())


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("T", [4, 12, 70])
def test_ids_out_of_range_in_both_forms(recipe, T):
    """Some ids out of range, then all of them: they contribute nothing and are reported."""
    from fp8_grouped_gemm_gb300 import mgq
    rng = np.random.default_rng(T)
    E, k, H, F = 6, 3, 256, 512
    x = torch.from_numpy(rng.normal(size=(T, H))).bfloat16()
    idx, p = _routing(T, E, k, rng)
    idx[1, 0], idx[2], idx[T - 1, 2] = E, -1, 2 ** 31 - 1
    t1, W1, v1 = _weight(E, 2 * F, H, recipe, rng)
    t2, W2, v2 = _weight(E, H, F, recipe, rng)
    sc = lambda d: torch.full((1,), d[recipe], device="cuda") if recipe in d else None
    xs, hs = sc(XS), sc(HS)
    ws = torch.full((mgq.moe_few_workspace_size(T, k, E, H, F, _scaling(recipe)),), 0xFF, dtype=torch.uint8, device="cuda")

    def run(ids):
        out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
        mgq.moe_few_forward(x.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(p).cuda(), W1, W2, _scaling(recipe), E,
                            F, out, ws, xs, hs)
        assert mgq.get_error() == mgq.ERR_DEVICE_INDEX and mgq.get_error() == mgq.OK
        return out

    out = run(idx)
    assert torch.all(out[2] == 0)
    _rows_close(out, x, idx, p, v1, v2, recipe, [t for t in range(T) if t != 2])
    assert torch.all(run(np.full_like(idx, -3)) == 0)


@pytest.mark.parametrize("recipe", ["mxfp8", "delayed", "nvfp4"])
@pytest.mark.parametrize("T", [3, 20])
def test_weights_with_a_longer_pitch(recipe, T):
    """The contraction is the first H (F) elements of longer weight rows (1x128: refused)."""
    rng = np.random.default_rng(T)
    E, k, H, F, more = 5, 2, 512, 768, 256
    x = torch.from_numpy(rng.normal(size=(T, H))).bfloat16()
    idx, p = _routing(T, E, k, rng)
    t1, W1, v1 = _weight(E, 2 * F, H + more, recipe, rng)
    t2, W2, v2 = _weight(E, H, F + 2 * more, recipe, rng)
    out = _call(x.cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(p).cuda(), W1, W2, recipe, E, F)
    _rows_close(out, x, idx, p, v1[:, :, :H], v2[:, :, :F], recipe)
