"""Pins of the float64 definitions around the expert layer (CPU only): the
gradients against central differences, the router against a brute-force
selection, the few-token layer against one token at a time."""
import numpy as np
import pytest

from oracle import block as OB


def _diff(f, x, h=1e-6):
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_rmsnorm_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(1)
    x, r, w = rng.normal(size=(3, 8)), rng.normal(size=(3, 8)), rng.normal(size=8)
    dy, dsum = rng.normal(size=(3, 8)), rng.normal(size=(3, 8))
    eps = 1e-2

    def loss(x_, w_):
        s, _, y = OB.rmsnorm(x_, r, w_, eps)
        return (y * dy).sum() + (s * dsum).sum()

    s, rstd, _ = OB.rmsnorm(x, r, w, eps)
    dx, dw = OB.rmsnorm_bwd(dy, s, w, rstd, dsum)
    # central differences with h = 1e-6: truncation ~h^2, rounding ~2^-52 / h
    assert np.allclose(dx, _diff(lambda v: loss(v, w), x), atol=1e-8)
    assert np.allclose(dw, _diff(lambda v: loss(x, v), w), atol=1e-8)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_router_gradient_is_the_difference_quotient(score, renorm):
    rng = np.random.default_rng(2)
    l, d = rng.normal(size=(4, 6)), rng.normal(size=(4, 3))
    idx, _ = OB.router_topk(l, 3, score, renorm, 1.7)

    def loss(v):   # the selection stays: differences of 1e-6 do not reorder these logits
        i, p = OB.router_topk(v, 3, score, renorm, 1.7)
        assert np.array_equal(i, idx)
        return (p * d).sum()

    g, bound = OB.router_topk_bwd(l, idx, d, score, renorm, 1.7)
    assert np.allclose(g, _diff(loss, l), atol=1e-8)
    assert np.all(np.abs(g) <= bound * (1 + 1e-12))


def test_router_ties_masks_and_nan():
    inf = np.inf
    l = np.array([[1.0, 2.0, 2.0, 0.0], [-inf, -inf, 3.0, -inf], [-inf] * 4, [np.nan, 1.0, np.nan, 2.0]])
    idx, p = OB.router_topk(l, 2)
    assert idx.tolist() == [[1, 2], [2, 0], [0, 1], [3, 1]]
    assert p[0].tolist() == [0.5, 0.5] and p[1].tolist() == [1.0, 0.0] and p[2].tolist() == [0.0, 0.0]
    g, _ = OB.router_topk_bwd(l, idx, np.ones((4, 2)))
    assert np.all(np.isfinite(g)) and np.all(g[2] == 0)


@pytest.mark.parametrize("recipe", ["mxfp8", "blockwise", "delayed", "nvfp4"])
def test_few_token_layer_is_the_sum_over_its_experts(recipe):
    rng = np.random.default_rng(3)
    T, E, k, H, F = 5, 4, 2, 128, 256
    x = rng.normal(size=(T, H))
    w1, w2 = rng.normal(size=(E, 2 * F, H)) * 0.1, rng.normal(size=(E, H, F)) * 0.1
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    p = rng.random((T, k))
    out = OB.moe_few(x, idx, p, w1, w2, recipe, 4.0, 2.0)
    for t in range(T):
        ref = np.zeros(H)
        xq = OB.quantize_rows(x[t:t + 1], recipe, 4.0)[0]
        for j in range(k):
            g, u = w1[idx[t, j], :F] @ xq, w1[idx[t, j], F:] @ xq
            h = OB.quantize_rows((g * u / (1 + np.exp(-g)))[None], recipe, 2.0)[0]
            ref += p[t, j] * (w2[idx[t, j]] @ h)
        # the same float64 sums in another order; a product at a rounding
        # boundary of h may flip one code (1/8 of a value among F)
        assert np.linalg.norm(out[t] - ref) <= 1e-2 * np.linalg.norm(ref)


def test_few_token_blockwise_rows():
    """Exact round trip of blocks whose scale is a power of two; the all-zero
    block; a value within half an e4m3 step of its block's scale otherwise."""
    rng = np.random.default_rng(7)
    v = rng.integers(-15, 16, size=(3, 256)).astype(np.float64)
    v[:, 0], v[:, 128] = 7 * 64.0, 3.5
    v[:, 129:] = np.clip(v[:, 129:], -3, 3)
    assert np.array_equal(OB.quantize_rows(v, "blockwise"), v)
    assert np.all(OB.quantize_rows(np.zeros((2, 128)), "blockwise") == 0)
    w = rng.normal(size=(4, 384))
    amax = np.abs(w).reshape(4, 3, 128).max(-1).repeat(128, 1)
    assert np.all(np.abs(OB.quantize_rows(w, "blockwise") - w) <= np.maximum(np.abs(w) / 16, amax / 448 * 2.0 ** -10) * 1.001)
