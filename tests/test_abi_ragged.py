"""Host-side argument validation of the products over ragged groups and of the
int8 row quantiser: each refusal comes back before anything is launched (CPU only)."""
import os
import subprocess
import sys

import pytest
import torch

P = 1024       # a well-aligned address that no refused call reads
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from fp8_grouped_gemm_gb300 import _build, mgq
    if not os.path.exists(mgq.LIB_PATH):
        _build.build()
    return mgq.load()


def _call(fn, order, base, **kw):
    a = dict(base)
    a.update(kw)
    return fn(*[a[n] for n in order], None)


ROWS = dict(x=P, ldx=64, w=P, off=P, E=4, R=10, N=32, K=64, y=P, ldy=32, dt=0)
ROWS_ORDER = ("x", "ldx", "w", "off", "E", "R", "N", "K", "y", "ldy", "dt")
SIZES = (dict(E=0), dict(E=1025), dict(R=-1), dict(R=1 << 31), dict(N=0), dict(N=12), dict(K=0), dict(K=20),
         dict(N=1 << 31), dict(K=1 << 31), dict(off=None), dict(off=P + 2), dict(dt=2), dict(dt=-1))


@pytest.mark.parametrize("name", ["mgq_ragged_gemm_fwd", "mgq_ragged_gemm_dgrad"])
def test_row_products_refusals(lib, name):
    from fp8_grouped_gemm_gb300 import mgq
    INV = mgq.ERR_INVALID_ARG
    base = dict(ROWS) if name.endswith("fwd") else dict(ROWS, ldx=32, ldy=64)
    run = lambda **kw: _call(getattr(lib, name), ROWS_ORDER, base, **kw)
    for bad in SIZES + (dict(x=None), dict(w=None), dict(y=None), dict(x=P + 8), dict(w=P + 8), dict(y=P + 8),
                        dict(ldx=base["ldx"] - 8), dict(ldx=base["ldx"] + 4), dict(ldy=base["ldy"] - 8),
                        dict(ldy=base["ldy"] + 2)):
        assert run(**bad) == INV, bad
    assert run(R=0) == mgq.OK and run(R=0, x=None, w=None) == mgq.OK      # nothing to do, nothing launched


def test_wgrad_refusals(lib):
    from fp8_grouped_gemm_gb300 import mgq
    INV = mgq.ERR_INVALID_ARG
    order = ("dy", "lddy", "x", "ldx", "off", "E", "R", "N", "K", "beta", "dw", "dt")
    base = dict(dy=P, lddy=32, x=P, ldx=64, off=P, E=4, R=10, N=32, K=64, beta=0.0, dw=P, dt=1)
    run = lambda **kw: _call(lib.mgq_ragged_gemm_wgrad, order, base, **kw)
    for bad in SIZES + (dict(dy=None), dict(x=None), dict(dw=None), dict(dy=P + 8), dict(x=P + 8), dict(dw=P + 8),
                        dict(lddy=24), dict(ldx=56), dict(lddy=36), dict(beta=float("nan")), dict(beta=1.0, dt=0)):
        assert run(**bad) == INV, bad
    assert run(R=0, beta=1.0) == mgq.OK


def test_int8_refusals(lib):
    from fp8_grouped_gemm_gb300 import mgq
    INV = mgq.ERR_INVALID_ARG
    order = ("x", "ldx", "xs", "w", "ws", "off", "E", "R", "N", "K", "y", "ldy", "dt")
    base = dict(ROWS, xs=P, ws=P)
    run = lambda **kw: _call(lib.mgq_ragged_gemm_int8, order, base, **kw)
    for bad in SIZES + (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None), dict(x=P + 8),
                        dict(xs=P + 2), dict(w=P + 8), dict(ws=P + 4), dict(y=P + 8), dict(ldx=48), dict(ldx=72),
                        dict(K=56, ldx=64), dict(ldy=24), dict(ldy=36)):
        assert run(**bad) == INV, bad
    assert run(R=0) == mgq.OK


def test_quantiser_refusals(lib):
    from fp8_grouped_gemm_gb300 import mgq
    INV = mgq.ERR_INVALID_ARG
    order = ("x", "ldx", "T", "K", "codes", "scale")
    base = dict(x=P, ldx=64, T=4, K=64, codes=P, scale=P)
    run = lambda **kw: _call(lib.mgq_rows_quantize_int8, order, base, **kw)
    for bad in (dict(x=None), dict(codes=None), dict(scale=None), dict(x=P + 8), dict(codes=P + 8), dict(scale=P + 2),
                dict(ldx=56), dict(ldx=68), dict(T=-1), dict(T=1 << 31), dict(K=0), dict(K=56), dict(K=1 << 31)):
        assert run(**bad) == INV, bad
    assert run(T=0) == mgq.OK


def test_binding_refuses_other_tensors():
    """What the C entry points cannot see: types, shapes, strides and place (host tensors here)."""
    from fp8_grouped_gemm_gb300 import mgq
    bf, f32, i8 = torch.bfloat16, torch.float32, torch.int8
    z = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype)
    off = torch.zeros(3, dtype=torch.int32)
    calls = [
        (lambda: mgq.ragged_gemm_fwd(z(4, 16, dtype=f32), z(2, 8, 16), off, z(4, 8)), mgq.ERR_UNSUPPORTED),
        (lambda: mgq.ragged_gemm_fwd(z(4, 16), z(2, 8, 16), off, z(4, 8, dtype=torch.float16)), mgq.ERR_UNSUPPORTED),
        (lambda: mgq.ragged_gemm_dgrad(z(4, 8), z(2, 8, 16, dtype=i8), off, z(4, 16)), mgq.ERR_UNSUPPORTED),
        (lambda: mgq.ragged_gemm_wgrad(z(4, 8), z(4, 16, dtype=i8), off, z(2, 8, 16)), mgq.ERR_UNSUPPORTED),
        (lambda: mgq.ragged_gemm_int8(z(4, 16), z(4, dtype=f32), z(2, 8, 16, dtype=i8), z(2, 8, dtype=f32), off, z(4, 8)),
         mgq.ERR_UNSUPPORTED),
        (lambda: mgq.rows_quantize_int8(z(4, 16, dtype=f32), z(4, 16, dtype=i8), z(4, dtype=f32)), mgq.ERR_UNSUPPORTED),
        (lambda: mgq.ragged_gemm_fwd(z(4, 16), z(8, 16), off, z(4, 8)), mgq.ERR_INVALID_ARG),
        (lambda: mgq.rows_quantize_int8(z(4, 2, 16), z(4, 2, 16, dtype=i8), z(4, dtype=f32)), mgq.ERR_INVALID_ARG),
    ]
    if not torch.cuda.is_available():      # (host tensors of the right shapes: the place is refused)
        torch_device, mgq._device = mgq._device, lambda: 0
        try:
            calls += [
                (lambda: mgq.ragged_gemm_fwd(z(4, 16), z(2, 8, 16), off, z(4, 8)), mgq.ERR_INVALID_ARG),
                (lambda: mgq.rows_quantize_int8(z(4, 16), z(4, 16, dtype=i8), z(4, dtype=f32)), mgq.ERR_INVALID_ARG),
            ]
            _expect(calls, mgq)
        finally:
            mgq._device = torch_device
    else:
        _expect(calls, mgq)


def _expect(calls, mgq):
    for i, (call, status) in enumerate(calls):
        with pytest.raises(mgq.MGQError) as e:
            call()
        assert e.value.status == status, i


@pytest.mark.parametrize("name", ["ragged.cu", "ragged_int8.cu", "ragged_few.cu"])
def test_programmatic_launches_read_with_plain_loads(name):
    """They may start before the launch in front of them has finished: each kernel waits before its first
    load, and takes nothing through the read-only path."""
    csrc = os.path.join(ROOT, "fp8_grouped_gemm_gb300", "csrc")
    text, shared = (open(os.path.join(csrc, n)).read() for n in (name, "ragged.cuh"))
    kernels = text.split("__global__")[1:]
    assert kernels and "launch_after(" in text and "<<<" not in text
    for k in kernels:
        assert "grid_wait()" in k
        wait = k.index("grid_wait()")
        assert all(wait < k.index(w) for w in ("load_groups", "p.offsets[", "tma_load_3d", "x[2 * u]") if w in k)
    for word in ("__ldg(", ".nc.", "__restrict__"):
        assert word not in text and word not in shared


def test_split_parts_are_read_by_lanes_that_use_them():
    """The few-row form's last cluster barrier lets the peers leave and waits for no load by itself. So every
    load from a peer's shared memory has its value stored before it: a lane that stores nothing reads nothing."""
    text = open(os.path.join(ROOT, "fp8_grouped_gemm_gb300", "csrc", "ragged_few.cu")).read()
    body = text[text.index("const bool in = "):text.index("ptx::cluster_sync_relaxed()")]
    assert body.count("ld_cluster_f32x4(") == 1 and "continue" not in body and "break" not in body
    assert "; in && j < n; " in body[:body.index("ld_cluster_f32x4(")]


@pytest.mark.parametrize("name", ["ragged.cu", "ragged_int8.cu", "ragged_few.cu"])
def test_first_calls_prepare_their_kernel_once(name):
    """What a launcher keeps per device is filled by one host thread, and read after it is whole: no flag or table
    that a second first caller could read or write meanwhile."""
    text = open(os.path.join(ROOT, "fp8_grouped_gemm_gb300", "csrc", name)).read()
    launchers = text.count("launch_after(kern")
    assert launchers and text.count("static OncePerDevice once;") == text.count("once.run(") == launchers
    assert "attr_set" not in text and "static bool" not in text


def test_binding_imports_without_cuda_in_torch():
    """A PyTorch built without CUDA lacks the bindings that the calls use: the module and the library load, and what
    needs no device (versions, sizes, refusals by type) works."""
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
from fp8_grouped_gemm_gb300 import mgq
assert mgq.load().mgq_version() == mgq.INTERFACE_VERSION and mgq.permute_workspace_size(64, 2, 8) > 0
try:
    mgq.ragged_gemm_fwd(torch.zeros(4, 16), torch.zeros(2, 8, 16), None, torch.zeros(4, 8))
except mgq.MGQError as e:
    assert e.status == mgq.ERR_UNSUPPORTED
else:
    raise AssertionError("not refused")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
