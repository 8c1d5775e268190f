"""Failure detection without a GPU fault: a grouped GEMM whose pipeline never
receives data (the producer is told to issue no loads) must come back with
MGQ_ERR_TIMEOUT after its bounded waits, leave the output untouched, and leave
the CUDA context usable for the next call. The stall and the short wait limit
are the library's test hooks (mgq_set_gemm_option); the test runs in a
subprocess so that its options cannot leak into other tests."""
import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = textwrap.dedent("""
    import os, sys, time
    import numpy as np, torch
    sys.path.insert(0, {root!r})
    from fp8_grouped_gemm_gb300 import mgq
    from tests.layer_check import tile_mx_scales
    mgq.load()
    dev = torch.device("cuda:0")
    rng = np.random.default_rng(0)
    E, N, K, R = 2, 256, 256, 512
    offs = torch.tensor([0, 256, 512], dtype=torch.int32, device=dev)
    a = torch.from_numpy(rng.integers(0, 0x7E, (R, K)).astype(np.uint8)).to(dev)
    w = torch.from_numpy(rng.integers(0, 0x7E, (E * N, K)).astype(np.uint8)).to(dev)
    sa = torch.tensor([1.0], device=dev)
    sw = torch.ones(E, device=dev)
    sca = torch.from_numpy(tile_mx_scales(np.full((R, K // 32), 127, np.uint8))).to(dev)
    scw = torch.from_numpy(tile_mx_scales(np.full((E * N, K // 32), 127, np.uint8))).to(dev)
    kinds = [("tensor", mgq.TENSOR_F32, (a, sa), (w, sw)), ("mx", mgq.MX32_E8M0, (a, sca), (w, scw))]
    for name, sc, (ad, asc), (wd, wsc) in kinds:
        A = mgq.operand(ad, asc, K, mgq.E4M3)
        W = mgq.operand(wd, wsc, K, mgq.E4M3)
        y = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=dev)
        mgq.set_gemm_option(mgq.GEMM_OPT_DEBUG_STALL, 1)
        mgq.set_gemm_option(mgq.GEMM_OPT_WAIT_MS, 50)
        t0 = time.time()
        mgq.grouped_gemm_fwd(A, W, sc, offs, E, R, N, K, y)
        torch.cuda.synchronize()
        dt = time.time() - t0
        st = mgq.get_error()
        assert st == mgq.ERR_TIMEOUT, (name, st)
        assert bool(torch.all(y == 7.0)), name            # nothing stored
        assert dt < 10.0, (name, dt)
        mgq.set_gemm_option(mgq.GEMM_OPT_DEBUG_STALL, 0)
        mgq.set_gemm_option(mgq.GEMM_OPT_WAIT_MS, 0)
        # the context is still usable: the same call without the stall is correct
        mgq.grouped_gemm_fwd(A, W, sc, offs, E, R, N, K, y)
        torch.cuda.synchronize()
        assert mgq.get_error() == mgq.OK
        assert not bool(torch.all(y == 7.0)), name
        print(name, "timeout reported in", round(dt, 3), "s; context usable")
    print("OK")
""")


def test_gemm_pipeline_timeout_is_reported_and_context_survives():
    code = SCRIPT.format(root=ROOT)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "OK" in r.stdout


NORM_SCRIPT = textwrap.dedent("""
    import sys, time
    import torch
    sys.path.insert(0, {root!r})
    from fp8_grouped_gemm_gb300 import mgq
    dev = torch.device("cuda:0")
    g = torch.Generator().manual_seed(1)
    # one warp a row, a few, the longest rows of the backward's ring
    for T, H in ((60000, 256), (6000, 2048), (1500, 8192)):
        x, dy = (torch.randn(T, H, generator=g).bfloat16().to(dev) for _ in range(2))
        w, rstd = torch.ones(H, device=dev), torch.ones(T, device=dev)
        ws = torch.empty(mgq.add_rmsnorm_bwd_workspace_size(T, H), dtype=torch.uint8, device=dev)
        def run():
            y, dx = (torch.full((T, H), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(2))
            codes = torch.full((T, H), 0xAB, dtype=torch.uint8, device=dev)
            sc = torch.empty(mgq.mx_scale_bytes(T, H), dtype=torch.uint8, device=dev)
            dw = torch.empty(H, device=dev)
            status = []
            t0 = time.time()
            mgq.add_rmsnorm_quantize(x, w, 1e-5, mgq.qdesc(mgq.E4M3, mgq.MX32_E8M0, codes, sc), residual=dy, y=y)
            torch.cuda.synchronize()
            status.append(mgq.get_error())
            mgq.add_rmsnorm_bwd(dy, x, w, rstd, dx, dw, ws, dsum=dy)
            torch.cuda.synchronize()
            status.append(mgq.get_error())
            return y, dx, codes, dw, status, time.time() - t0
        ref = run()
        assert ref[4] == [mgq.OK, mgq.OK] and not bool(torch.any(torch.all(ref[0] == 7.0, 1)))
        mgq.set_gemm_option(mgq.GEMM_OPT_DEBUG_STALL, 1)
        mgq.set_gemm_option(mgq.GEMM_OPT_WAIT_MS, 50)
        y, dx, codes, dw, status, dt = run()
        assert status == [mgq.ERR_TIMEOUT, mgq.ERR_TIMEOUT], status
        assert bool(torch.all(y == 7.0)) and bool(torch.all(dx == 7.0)) and bool(torch.all(codes == 0xAB))
        assert dt < 10.0, dt
        mgq.set_gemm_option(mgq.GEMM_OPT_DEBUG_STALL, 0)
        mgq.set_gemm_option(mgq.GEMM_OPT_WAIT_MS, 0)
        again = run()
        assert again[4] == [mgq.OK, mgq.OK] and all(torch.equal(a, b) for a, b in zip(ref[:4], again[:4]))
    print("OK")
""")


def test_norm_ring_timeout_is_reported_and_context_survives():
    r = subprocess.run([sys.executable, "-c", NORM_SCRIPT.format(root=ROOT)], capture_output=True, text=True, timeout=300,
                       cwd=ROOT)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "OK" in r.stdout


FEW_SCRIPT = textwrap.dedent("""
    import sys, time
    import numpy as np, torch
    sys.path.insert(0, {root!r})
    from fp8_grouped_gemm_gb300 import mgq
    from tests.test_gpu_moe_few import RECIPES, XS, HS, _routing, _scaling, _weight
    rng = np.random.default_rng(3)
    # more than eight tokens: the form with a ring; several tiles a CTA, and fewer tiles than CTAs
    for T, E, k, H, F in ((20, 8, 2, 256, 512), (12, 16, 4, 256, 1024)):
        for recipe in RECIPES:
            x = torch.from_numpy(rng.normal(size=(T, H))).bfloat16().cuda()
            idx, p = (torch.from_numpy(a).cuda() for a in _routing(T, E, k, rng))
            t1, W1, _ = _weight(E, 2 * F, H, recipe, rng)
            t2, W2, _ = _weight(E, H, F, recipe, rng)
            ws = torch.zeros(mgq.moe_few_workspace_size(T, k, E, H, F, _scaling(recipe)), dtype=torch.uint8, device="cuda")
            sc = lambda d: torch.full((1,), d[recipe], device="cuda") if recipe in d else None
            xs, hs = sc(XS), sc(HS)
            def run():
                out = torch.empty_like(x)
                t0 = time.time()
                mgq.moe_few_forward(x, idx, p, W1, W2, _scaling(recipe), E, F, out, ws, xs, hs)
                torch.cuda.synchronize()
                return out, mgq.get_error(), time.time() - t0
            ref, status, _ = run()
            assert status == mgq.OK
            mgq.set_gemm_option(mgq.GEMM_OPT_DEBUG_STALL, 1)
            mgq.set_gemm_option(mgq.GEMM_OPT_WAIT_MS, 20)
            _, status, dt = run()
            assert status == mgq.ERR_TIMEOUT, (recipe, status)
            assert dt < 10.0, dt
            mgq.set_gemm_option(mgq.GEMM_OPT_DEBUG_STALL, 0)
            mgq.set_gemm_option(mgq.GEMM_OPT_WAIT_MS, 0)
            out, status, _ = run()
            assert status == mgq.OK and torch.equal(out, ref), recipe
    print("OK")
""")


def test_few_token_pipeline_timeout_is_reported_and_context_survives():
    r = subprocess.run([sys.executable, "-c", FEW_SCRIPT.format(root=ROOT)], capture_output=True, text=True, timeout=300,
                       cwd=ROOT)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "OK" in r.stdout
