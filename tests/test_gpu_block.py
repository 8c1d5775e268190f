"""The MoE half of a decoder layer (block.py) on the GPU: its norm and router
and their gradients against the float64 definitions on the values that the step
itself produced, and decode batches on the same weights against the definition."""
import numpy as np
import pytest
import torch

from fp8_grouped_gemm_gb300 import mgq
from fp8_grouped_gemm_gb300 import workloads as W
from oracle import block as OB
from oracle import quant as OQ
from tests.layer_check import bf16_np, u8_np, ulp_bf16, untile_mx_scales
from tests.test_gpu_moe_few import _rows_close

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _block(recipe="mxfp8", T=64, train=True, **kw):
    from fp8_grouped_gemm_gb300 import block as B
    w = W.WORKLOADS["tiny"].scaled(T=T, E=8)
    b = B.MoEBlock(w, "cuda:0", recipe, train=train, **kw)
    g = torch.Generator().manual_seed(5)
    w1, w2 = W.make_weights(w)
    b.load(w1.cuda(), w2.cuda(), (1 + 0.1 * torch.randn(w.H, generator=g)).bfloat16().cuda(),
           (torch.randn(w.E, w.H, generator=g) * w.H ** -0.5).cuda())
    x = torch.randn(T, w.H, generator=g).bfloat16().cuda()
    r = torch.randn(T, w.H, generator=g).bfloat16().cuda()
    return b, x, r


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_steps_of_forward_and_backward(score, renorm):
    b, x, r = _block(score=mgq.SCORE_SOFTMAX if score == "softmax" else mgq.SCORE_SIGMOID, renorm=renorm, route_scale=1.5)
    out, s = b.forward(x, r)
    rs, rstd, ry = OB.rmsnorm(bf16_np(x), bf16_np(r), bf16_np(b.norm_w), b.eps)
    assert np.all(np.abs(bf16_np(s) - rs) <= 0.5 * ulp_bf16(rs) * (1 + 1e-9) + U * np.abs(rs))
    assert np.all(np.abs(bf16_np(b.y) - ry) <= 0.5 * ulp_bf16(ry) * (1 + 1e-9) + 72 * U * np.abs(ry))
    l = b.logits.double().cpu().numpy()
    idx, p = OB.router_topk(l, b.w.k, score, renorm, 1.5)
    assert np.array_equal(b.topk_idx.cpu().numpy(), idx)
    assert np.all(np.abs(b.probs.cpu().numpy() - p) <= 64 * U * p)
    g = torch.Generator().manual_seed(6)
    dout = torch.randn(x.shape, generator=g).bfloat16().cuda()
    dsum = torch.randn(x.shape, generator=g).bfloat16().cuda()
    dx = b.backward(dout, dsum)
    rl, mag = OB.router_topk_bwd(l, idx, b.experts.dprobs.double().cpu().numpy(), score, renorm, 1.5)
    assert np.all(np.abs(b.dlogits.double().cpu().numpy() - rl) <= 96 * U * mag + 1e-37)
    # the norm's gradient from the dy that reached it
    dy = (b.experts.dx.float() + b.dlogits @ b.router_w).bfloat16()
    rdx, rdw = OB.rmsnorm_bwd(bf16_np(dy), bf16_np(s), bf16_np(b.norm_w), b.rstd.double().cpu().numpy(), bf16_np(dsum))
    got = bf16_np(dx)
    # dy's bf16 rounding may fall the other way in an element (addmm against @): 2^-8 of it
    assert np.linalg.norm(got - rdx) <= 4e-3 * np.linalg.norm(rdx)
    assert np.linalg.norm(b.dnorm_w.cpu().numpy() - rdw) <= 1e-3 * np.linalg.norm(rdw)
    assert mgq.get_error() == mgq.OK


def _values(codes, scale, recipe, E, N, K, sg=None):
    """float64 values of the layer's quantised weight [E, N, K]."""
    c = u8_np(codes)
    if recipe == "mxfp8":
        return OQ.dequantize_mx(c.reshape(E * N, K), untile_mx_scales(u8_np(scale), E * N, K)).reshape(E, N, K)
    if recipe == "nvfp4":
        s = untile_mx_scales(u8_np(scale), E * N, K, block=16).reshape(E, N, K // 16)
        return np.stack([OQ.dequantize_nvfp4(c[e], s[e], np.float32(sg[e]), K) for e in range(E)])
    s = scale.cpu().numpy()
    if recipe == "blockwise":
        return np.stack([OQ.dequantize_block_128x128(c[e], s[e]) for e in range(E)])
    return np.stack([OQ.dequantize_tensor(c[e], s[e]) for e in range(E)])


@pytest.mark.parametrize("recipe", ["mxfp8", "blockwise", "nvfp4", "delayed"])
def test_decode(recipe):
    """Decode batches on the weights and scales that a many-token step left: the
    same sums and selections as that step, outputs as the definition has them."""
    b, x, r = _block(recipe, T=64, train=None)
    w, ex = b.w, b.experts
    if recipe == "delayed":                 # a first step sets the scales
        b.forward(x, r)
        ex.update_scaling()
        ex.quantize_weights(*(t.cuda() for t in W.make_weights(w)))
    _, s = b.forward(x, r)
    E, H, F = w.E, w.H, w.F
    sg = ex.nv_sg.cpu().numpy() if recipe == "nvfp4" else None
    fs = ex.fwd_scale if recipe == "delayed" else None
    v1 = _values(ex.w1q, fs[2:2 + E] if recipe == "delayed" else ex.w1s, recipe, E, 2 * F, H,
                 None if sg is None else sg[2:2 + E])
    v2 = _values(ex.w2q, fs[2 + E:2 + 2 * E] if recipe == "delayed" else ex.w2s, recipe, E, H, F,
                 None if sg is None else sg[2 + E:2 + 2 * E])
    xs, hs = (sg[0], sg[1]) if sg is not None else (fs[0].item(), fs[1].item()) if fs is not None else (None, None)
    at = 0
    for n in (1, 3, 8, 17, 35):
        out, s1 = b.decode(x[at:at + n].contiguous(), r[at:at + n].contiguous())
        assert torch.equal(s1, s[at:at + n])
        y, idx, probs = b.few
        assert torch.equal(y, b.y[at:at + n])
        _rows_close(out, y, idx.cpu().numpy(), probs.cpu().numpy(), v1, v2, recipe, scales=(xs, hs))
        at += n
    assert mgq.get_error() == mgq.OK


def _left(ex, recipe):
    """(W1, W2 values, x scale, h scale) that the layer's codes and scales stand for (delayed, NVFP4)."""
    E, H, F = ex.w.E, ex.w.H, ex.w.F
    if recipe == "nvfp4":
        sg = ex.nv_sg.cpu().numpy()
        return (_values(ex.w1q, ex.w1s, recipe, E, 2 * F, H, sg[2:2 + E]),
                _values(ex.w2q, ex.w2s, recipe, E, H, F, sg[2 + E:2 + 2 * E]), sg[0], sg[1])
    fs = ex.fwd_scale.clone()
    return (_values(ex.w1q, fs[2:2 + E], recipe, E, 2 * F, H), _values(ex.w2q, fs[2 + E:2 + 2 * E], recipe, E, H, F),
            fs[0].item(), fs[1].item())


def test_decode_after_update_scaling_on_the_same_weights():
    """A training step ends with update_scaling(), which sets the scales of the
    next step's weights; the codes are still those of the step's own."""
    b, x, r = _block("delayed", T=64, train=None)
    ex = b.experts
    b.forward(x, r)
    b.backward(torch.randn(x.shape, generator=torch.Generator().manual_seed(8)).bfloat16().cuda())
    v1, v2, _, _ = _left(ex, "delayed")
    old = ex.fwd_scale.clone()
    ex.update_scaling()
    assert not torch.equal(old, ex.fwd_scale)
    xs, hs = ex.fwd_scale[0].item(), ex.fwd_scale[1].item()
    for n in (5, 20):
        out, _ = b.decode(x[:n].contiguous(), r[:n].contiguous())
        y, idx, probs = b.few
        _rows_close(out, y, idx.cpu().numpy(), probs.cpu().numpy(), v1, v2, "delayed", scales=(xs, hs))
    # the many-token path on the same codes (bf16 g, u and h on the way: 2e-2, as for the grouped layer)
    many = bf16_np(b.forward(x, r)[0])[:20]
    assert np.linalg.norm(bf16_np(out) - many) <= 2e-2 * np.linalg.norm(many)
    assert mgq.get_error() == mgq.OK


@pytest.mark.parametrize("recipe", ["mxfp8", "nvfp4"])
def test_decode_batches_of_every_size_share_one_workspace(recipe):
    """Nothing is kept per batch size, and a captured step stays valid whatever sizes follow."""
    b, x, r = _block(recipe, T=128, train=None)
    b.forward(x, r)
    ex, y, idx, probs = b.experts, b.y, b.topk_idx, b.probs
    first = [ex.forward_few(y[:n], idx[:n], probs[:n]) for n in (3, 50)]
    out = torch.zeros_like(first[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ex.forward_few(y[:3], idx[:3], probs[:3], out)
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    for n in range(1, 129):
        ex.forward_few(y[:n], idx[:n], probs[:n])
        assert torch.cuda.memory_allocated() == held, n
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(ex.forward_few(y[:50], idx[:50], probs[:50]), first[1])
    assert mgq.get_error() == mgq.OK


def test_decode_on_another_stream_allocates_its_result_there():
    """Memory of the current stream's pool may still be in use there when the call runs on another."""
    b, x, r = _block("mxfp8", T=64, train=None)
    b.forward(x, r)
    args = (b.y[:9], b.topk_idx[:9], b.probs[:9])
    ref = b.experts.forward_few(*args)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = b.experts.forward_few(*args, stream=st)
    seg = [s for s in torch.cuda.memory_snapshot() if s["address"] <= out.data_ptr() < s["address"] + s["total_size"]]
    assert [s["stream"] for s in seg] == [st.cuda_stream]
    st.synchronize()
    assert torch.equal(out, ref)



def test_decode_refuses_rows_of_another_width():
    b, x, r = _block("mxfp8", T=64, train=None)
    b.forward(x, r)
    for H in (b.w.H // 2, 2 * b.w.H):
        with pytest.raises(mgq.MGQError) as e:
            b.experts.forward_few(torch.zeros(4, H, dtype=torch.bfloat16, device="cuda"), b.topk_idx[:4], b.probs[:4])
        assert e.value.status == mgq.ERR_INVALID_ARG



@pytest.mark.parametrize("recipe", ["nvfp4", "delayed"])
def test_decode_scales_of_its_own(recipe):
    """Scales of x and h that a program fixes stay, whatever forward runs between; without
    values they are the last step's."""
    b, x, r = _block(recipe, T=64, train=None)
    ex = b.experts

    def decode(xs, hs):
        out, _ = b.decode(x[:9].contiguous(), r[:9].contiguous())
        v1, v2, _, _ = _left(ex, recipe)
        y, idx, probs = b.few
        _rows_close(out, y, idx.cpu().numpy(), probs.cpu().numpy(), v1, v2, recipe, scales=(xs, hs))
        return out

    ex.set_decode_scales(11.5, torch.tensor([6.25], device="cuda"))      # no step has run
    a = decode(11.5, 6.25)
    b.forward(x * 8, r)
    assert torch.equal(decode(11.5, 6.25), a)
    ex.set_decode_scales()
    _, _, xs, hs = _left(ex, recipe)
    c = decode(xs, hs)
    b.forward(x, r * 8)
    assert torch.equal(decode(xs, hs), c)



def test_nvfp4_decode_without_scales_is_refused():
    """Before a step has run or scales were given there is no global scale of x and h."""
    b, x, r = _block("nvfp4", T=64, train=None)
    with pytest.raises(mgq.MGQError) as e:
        b.decode(x[:4].contiguous(), r[:4].contiguous())
    assert e.value.status == mgq.ERR_INVALID_ARG
    with pytest.raises(mgq.MGQError):
        b.experts.set_decode_scales()
    b.forward(x, r)
    b.decode(x[:4].contiguous(), r[:4].contiguous())
    with pytest.raises(mgq.MGQError) as e:
        _block("mxfp8", T=64, train=None)[0].experts.set_decode_scales(1.0, 1.0)
    assert e.value.status == mgq.ERR_UNSUPPORTED
