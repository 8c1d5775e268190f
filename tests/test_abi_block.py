"""Host-side argument validation of the entry points around the expert layer:
each refusal comes back before anything is launched (CPU only)."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def lib():
    from fp8_grouped_gemm_gb300 import _build, mgq
    if not os.path.exists(mgq.LIB_PATH):
        _build.build()
    return mgq.load()


P = 1024       # a well-aligned address that no refused call reads


def _norm(lib, q=None, **kw):
    a = dict(x=P, r=None, w=P, wd=0, T=4, H=256, eps=1e-5, sum=None, y=P, rstd=None)
    a.update(kw)
    return lib.mgq_add_rmsnorm_quantize(a["x"], a["r"], a["w"], a["wd"], a["T"], a["H"], a["eps"], a["sum"], a["y"],
                                        ctypes.byref(q) if q is not None else None, a["rstd"], None)


def test_norm_refusals(lib):
    from fp8_grouped_gemm_gb300 import mgq
    INV, UNS = mgq.ERR_INVALID_ARG, mgq.ERR_UNSUPPORTED
    assert _norm(lib, H=100) == INV and _norm(lib, H=0) == INV and _norm(lib, H=16392) == INV
    assert _norm(lib, T=-1) == INV and _norm(lib, eps=-1.0) == INV and _norm(lib, eps=float("nan")) == INV
    assert _norm(lib, x=None) == INV and _norm(lib, w=None) == INV and _norm(lib, wd=2) == INV
    assert _norm(lib, y=None) == INV                       # no output
    for name in ("x", "r", "w", "sum", "y"):
        assert _norm(lib, **{name: P + 8}) == INV          # alignment
    q = lambda **k: mgq.qdesc(k.pop("dtype", mgq.E4M3), k.pop("scaling", mgq.MX32_E8M0), P, P, **k)
    assert _norm(lib, q(), H=264) == INV                   # scaled outputs: whole 128-element blocks
    assert _norm(lib, q(scaling=mgq.NV16_UE4M3, dtype=mgq.E2M1)) == UNS
    assert _norm(lib, q(scaling=mgq.NV16_UE4M3)) == UNS
    assert _norm(lib, q(scaling=mgq.BLK_128x128_F32)) == UNS
    assert _norm(lib, q(col_data=P, col_scale=P)) == UNS
    assert _norm(lib, q(e8m0_mode=5)) == INV
    assert _norm(lib, mgq.qdesc(mgq.E4M3, mgq.MX32_E8M0, None, P)) == INV
    assert _norm(lib, mgq.qdesc(mgq.E4M3, mgq.MX32_E8M0, P, None)) == INV
    assert _norm(lib, mgq.qdesc(mgq.E4M3, mgq.TENSOR_F32, P)) == INV       # no scale
    assert _norm(lib, mgq.qdesc(mgq.E4M3, mgq.MX32_E8M0, P + 8, P)) == INV
    assert _norm(lib, T=0) == mgq.OK                       # nothing to do, nothing launched


def test_norm_backward_refusals(lib):
    from fp8_grouped_gemm_gb300 import mgq
    INV = mgq.ERR_INVALID_ARG
    ws = lib.mgq_add_rmsnorm_bwd_workspace_size(4, 256)
    assert ws >= 256 * 4 and lib.mgq_add_rmsnorm_bwd_workspace_size(4, 100) == 0

    def bwd(**kw):
        a = dict(dy=P, s=P, w=P, wd=0, rstd=P, dsum=None, T=4, H=256, dx=P, dw=P, beta=0.0, ws=P, n=ws)
        a.update(kw)
        return lib.mgq_add_rmsnorm_bwd(a["dy"], a["s"], a["w"], a["wd"], a["rstd"], a["dsum"], a["T"], a["H"],
                                       a["dx"], a["dw"], a["beta"], a["ws"], a["n"], None)

    for name in ("dy", "s", "w", "rstd", "dx", "dw", "ws"):
        assert bwd(**{name: None}) == INV, name
    for name in ("dy", "s", "w", "dsum", "dx", "ws"):
        assert bwd(**{name: P + 8}) == INV, name
    assert bwd(n=ws - 1) == INV and bwd(H=12) == INV and bwd(T=-1) == INV and bwd(wd=7) == INV


def test_router_refusals(lib):
    from fp8_grouped_gemm_gb300 import mgq
    INV = mgq.ERR_INVALID_ARG

    def fwd(**kw):
        a = dict(l=P, dt=1, T=4, E=16, k=2, score=0, renorm=1, idx=P, p=P)
        a.update(kw)
        return lib.mgq_router_topk(a["l"], a["dt"], a["T"], a["E"], a["k"], a["score"], a["renorm"], 1.0, a["idx"],
                                   a["p"], None)

    def bwd(**kw):
        a = dict(l=P, dt=1, T=4, E=16, k=2, score=0, renorm=1, idx=P, d=P, dl=P)
        a.update(kw)
        return lib.mgq_router_topk_bwd(a["l"], a["dt"], a["idx"], a["d"], a["T"], a["E"], a["k"], a["score"],
                                       a["renorm"], 1.0, a["dl"], None)

    for f in (fwd, bwd):
        for bad in (dict(l=None), dict(idx=None), dict(dt=2), dict(T=-1), dict(E=0), dict(E=1025), dict(k=0),
                    dict(k=9), dict(k=3, E=2), dict(score=2), dict(renorm=2), dict(l=P + 2)):
            assert f(**bad) == INV, (f.__name__, bad)
        assert f(T=0) == mgq.OK
    assert fwd(p=None) == INV and bwd(d=None) == INV and bwd(dl=None) == INV


def test_few_token_layer_refusals(lib):
    from fp8_grouped_gemm_gb300 import mgq
    INV, UNS = mgq.ERR_INVALID_ARG, mgq.ERR_UNSUPPORTED
    size = lib.mgq_moe_few_workspace_size
    ws = size(4, 2, 8, 512, 256, mgq.MX32_E8M0)
    assert ws > 0
    for bad in ((129, 2, 8, 512, 256), (4, 9, 16, 512, 256), (4, 3, 2, 512, 256), (4, 2, 1025, 512, 256),
                (4, 2, 8, 500, 256), (4, 2, 8, 512, 64), (-1, 2, 8, 512, 256), (4, 0, 8, 512, 256)):
        assert size(*bad, mgq.MX32_E8M0) == 0
    assert size(4, 2, 8, 384, 256, mgq.NV16_UE4M3) == 0       # NVFP4: multiples of 256
    assert size(4, 2, 8, 512, 256, mgq.BLK_128x128_F32) == 0
    op = lambda ld, dt=mgq.E4M3, **k: mgq.operand(k.pop("data", P), k.pop("scale", P), ld, dt, **k)

    def run(**kw):
        a = dict(x=P, T=4, H=512, F=256, idx=P, p=P, k=2, E=8, W1=op(512), W2=op(256), sc=mgq.MX32_E8M0, xs=None,
                 hs=None, out=P, ws=P, n=1 << 40)
        a.update(kw)
        r = lambda o: ctypes.byref(o) if o is not None else None
        return lib.mgq_moe_few_forward(a["x"], a["T"], a["H"], a["F"], a["idx"], a["p"], a["k"], a["E"], r(a["W1"]),
                                       r(a["W2"]), a["sc"], a["xs"], a["hs"], a["out"], a["ws"], a["n"], None)

    for name in ("x", "idx", "p", "out", "ws", "W1", "W2"):
        assert run(**{name: None}) == INV, name
    for name in ("x", "out"):
        assert run(**{name: P + 8}) == INV, name
    assert run(ws=P + 16) == INV and run(n=ws - 1) == INV
    assert run(T=129) == INV and run(H=520) == INV and run(F=100) == INV and run(k=9) == INV and run(E=1) == INV
    assert run(sc=mgq.BLK_128x128_F32) == UNS and run(W1=op(512, mgq.E5M2)) == UNS
    assert run(sc=mgq.NV16_UE4M3) == UNS                      # e4m3 codes
    assert run(W2=op(256, layout=mgq.LAYOUT_MN)) == UNS
    assert run(W1=op(256)) == INV and run(W1=op(520)) == INV  # row pitch
    assert run(W1=op(512, data=None)) == INV and run(W2=op(256, scale=None)) == INV and run(W1=op(512, data=P + 8)) == INV
    nv = dict(sc=mgq.NV16_UE4M3, W1=op(512, mgq.E2M1, global_scale=P), W2=op(256, mgq.E2M1, global_scale=P), xs=P, hs=P)
    assert run(**{**nv, "xs": None}) == INV and run(**{**nv, "hs": None}) == INV
    assert run(**{**nv, "W1": op(512, mgq.E2M1)}) == INV
    assert run(**{**nv, "H": 384}) == INV
    assert run(sc=mgq.TENSOR_F32) == INV                      # no scales of x and h
    assert run(sc=mgq.BLK_1x128_F32, W1=op(640)) == INV       # 128x128 scales: no padding of the rows
    assert run(T=0) == mgq.OK
