"""The operators around the routed-expert layer, as cases to time and to compare.

Three operators: the residual addition + RMSNorm with an 8-bit output (forward
"norm" and backward "norm_bwd"), the top-k router ("router", with its gradient
where the case trains) and the whole expert layer for a few tokens ("few").
Each case runs either the plain form below (elementary torch operations in
float32) or, with `own` set, the library's entry points; `exact` restates the
definitions in float64.

8-bit outputs are returned as float8 tensors (e4m3 codes, E8M0 scales), i.e. as
the values they stand for.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
ALL_SCALINGS = ("mxfp8", "blockwise", "delayed", "nvfp4")


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # one new token of a 4096-wide model: latency of a single row
        dict(name="norm_decode_1x4096", op="norm", T=1, H=4096, scaling="mxfp8", residual=True),
        # the training batch of the Mixtral-shaped layer
        dict(name="norm_train_16384x4096", op="norm", T=16384, H=4096, scaling="mxfp8", residual=True),
        # a ragged prefill of the Scout-shaped layer, blockwise FP8, the layer's first norm (no residual)
        dict(name="norm_prefill_1003x5120", op="norm", T=1003, H=5120, scaling="blockwise", residual=False),
        # gradients of the two training shapes: the large batch, and a short ragged micro-batch
        dict(name="norm_bwd_16384x4096", op="norm_bwd", T=16384, H=4096, residual=True),
        dict(name="norm_bwd_333x2048", op="norm_bwd", T=333, H=2048, residual=False),
        # a decode batch routed over the fine-grained layer's experts
        dict(name="router_decode_16x128", op="router", T=16, E=128, k=8, score="softmax", renorm=True, train=False),
        # the fine-grained layer's training batch, with the logits' gradient
        dict(name="router_train_32768x128", op="router", T=32768, E=128, k=8, score="softmax", renorm=True,
             train=True),
        # single-token decode of the Mixtral-shaped experts (two experts read)
        dict(name="few_mixtral_T1_mxfp8", op="few", T=1, E=8, k=2, H=4096, F=14336, scaling="mxfp8"),
        # a decode batch that reaches all eight experts: the largest weight read
        dict(name="few_mixtral_T16_delayed", op="few", T=16, E=8, k=2, H=4096, F=14336, scaling="delayed"),
        # single-token decode of the fine-grained experts: the smallest weight read
        dict(name="few_finegrained_T1_nvfp4", op="few", T=1, E=128, k=8, H=2048, F=768, scaling="nvfp4"),
        # a decode batch over nearly all fine-grained experts, a few rows each
        dict(name="few_finegrained_T64_nvfp4", op="few", T=64, E=128, k=8, H=2048, F=768, scaling="nvfp4"),
        # an odd batch on the Scout-shaped top-1 experts, blockwise FP8
        dict(name="few_scout_T33_blockwise", op="few", T=33, E=16, k=1, H=5120, F=8192, scaling="blockwise"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "router", "few", "few", "few"])
    if op == "norm":
        c = dict(op=op, T=_log_int(rng, 1, 16384), H=128 * _log_int(rng, 2, 64),
                 scaling=rng.choice(["mxfp8", "blockwise", "delayed"]), residual=rng.random() < 0.7)
        c["T"] = max(1, min(c["T"], 16384 * 4096 // c["H"]))
        return c
    if op == "norm_bwd":
        c = dict(op=op, T=_log_int(rng, 1, 16384), H=128 * _log_int(rng, 2, 64), residual=rng.random() < 0.5)
        c["T"] = max(1, min(c["T"], 16384 * 4096 // c["H"]))
        return c
    if op == "router":
        return dict(op=op, T=_log_int(rng, 1, 32768), E=_log_int(rng, 8, 256), k=rng.randint(1, 8),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.6, train=rng.random() < 0.6)
    E, scaling = _log_int(rng, 4, 128), rng.choice(ALL_SCALINGS)
    unit = 256 if scaling == "nvfp4" else 128      # NVFP4 contractions are multiples of 256
    H, F = unit * _log_int(rng, 2, 5120 // unit), unit * _log_int(rng, 2, 14336 // unit)
    while E * H * F > 8 * 4096 * 14336:
        E = E // 2
    E = max(2, E)
    return dict(op=op, T=_log_int(rng, 1, 128), E=E, k=rng.randint(1, min(8, E)), H=H, F=F, scaling=scaling)


# bytes of one weight element, scales included
_WEIGHT_BYTES = {"mxfp8": 1 + 1 / 32, "blockwise": 1 + 4 / 16384, "delayed": 1.0, "nvfp4": 0.5 + 1 / 16}


def work(case):
    T, op = case["T"], case["op"]
    if op == "norm":
        H = case["H"]
        scale = {"mxfp8": 1 / 32, "blockwise": 4 / 128, "delayed": 0.0}[case["scaling"]]
        r = 4 if case["residual"] else 0          # the residual read and the sum written
        return {"bytes": T * H * (2 + r + 2 + 1 + scale) + 2 * H + 4 * T, "flops": 6 * T * H}
    if op == "norm_bwd":
        H = case["H"]
        return {"bytes": T * H * (6 + (2 if case["residual"] else 0)) + 2 * H + 4 * H + 4 * T, "flops": 10 * T * H}
    if op == "router":
        E, k = case["E"], case["k"]
        b = T * E * 4 + T * k * 8
        if case["train"]:
            b += T * k * 4 + T * E * 4            # dprobs read, dlogits written
        return {"bytes": b, "flops": T * E * 4}
    E, k, H, F = case["E"], case["k"], case["H"], case["F"]
    # experts that at least one of the T tokens picked (k distinct ones each), on average
    active = E * (1 - (1 - k / E) ** T)
    return {"bytes": active * 3 * H * F * _WEIGHT_BYTES[case["scaling"]] + T * H * 4 + T * k * 8,
            "flops": 6 * T * k * H * F}


# ---------------------------------------------------------------------------
# inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, std=1.0):
    return torch.randn(shape, device="cuda", generator=g) * std


def _activations(T, H, g):
    """Hidden states with a few large channels, as the training shapes have them."""
    x = _randn((T, H), g)
    ch = torch.randperm(H, device="cuda", generator=g)[: max(1, H // 1000)]
    x[:, ch] *= 50.0
    return x.to(torch.bfloat16)


def _tile_scales(s):
    """[..., rows, blocks] scale bytes -> the 128x4-tiled layout (rows and blocks padded to whole tiles)."""
    rows, nb = s.shape
    rp = (rows + 127) // 128 * 128
    full = torch.zeros(rp, nb, dtype=s.dtype, device=s.device)
    full[:rows] = s
    return full.view(rp // 128, 4, 32, nb // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile_scales(t, rows, nb):
    return t.view(-1, nb // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, nb)[:rows]


def _mx_exponent(amax):
    """Smallest e with amax <= 448 * 2^e, in [-127, 127] (-127 for 0); works in the dtype given."""
    m, e = torch.frexp(amax)                       # amax = m 2^e, m in [0.5, 1)
    e = e.to(torch.int32) - 9 + (m > 0.875).to(torch.int32)
    return torch.where(amax == 0, torch.full_like(e, -127), e.clamp(-127, 127))


def _pow2(e):
    """2^e as float32, for integers e in [-127, 127]."""
    return torch.where(e > -127, ((e + 127) << 23).view(torch.float32), 2.0 ** -127)


def _weight(E, N, K, scaling, g):
    """Quantised weights [E, N, K] of N(0, 0.02) in the framework's layouts."""
    d = {}
    nv = scaling == "nvfp4"
    codes = torch.empty(E, N, K // 2 if nv else K, dtype=torch.uint8, device="cuda")
    if scaling == "mxfp8":
        d["scale"] = torch.empty(E, N * (K // 32), dtype=torch.uint8, device="cuda")
    elif nv:
        d["scale"] = torch.empty(E, N * (K // 16), dtype=torch.uint8, device="cuda")
        d["global"] = torch.empty(E, device="cuda")
    elif scaling == "blockwise":
        d["scale"] = torch.empty(E, N // 128, K // 128, device="cuda")
    else:
        d["scale"] = torch.empty(E, device="cuda")
    for e in range(E):
        w = _randn((N, K), g, 0.02)
        if scaling == "mxfp8":
            wb = w.view(N, K // 32, 32)
            ex = _mx_exponent(wb.abs().amax(-1))
            codes[e] = (wb * _pow2(-ex)[..., None]).view(N, K).to(torch.float8_e4m3fn).view(torch.uint8)
            d["scale"][e] = _tile_scales((ex + 127).to(torch.uint8))
        elif nv:
            wb = w.view(N, K // 16, 16)
            sg = 2688.0 / w.abs().amax()
            sc = (wb.abs().amax(-1) / 6.0 * sg).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn)
            v = wb * torch.where(sc.float() == 0, 0.0, sg / sc.float())[..., None]
            codes[e] = _pack_e2m1(_round_e2m1(v)).view(N, K // 2)
            d["scale"][e] = _tile_scales(sc.view(torch.uint8))
            d["global"][e] = sg
        elif scaling == "blockwise":
            wb = w.view(N // 128, 128, K // 128, 128)
            s = E4M3_MAX / wb.abs().amax((1, 3))
            codes[e] = (wb * s[:, None, :, None]).view(N, K).clamp(-E4M3_MAX, E4M3_MAX).to(
                torch.float8_e4m3fn).view(torch.uint8)
            d["scale"][e] = 1.0 / s
        else:
            s = E4M3_MAX / w.abs().amax()
            codes[e] = (w * s).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
            d["scale"][e] = s
    d["codes"] = codes
    return d


def prepare(case, seed):
    g = _gen(seed)
    T, op = case["T"], case["op"]
    st = dict(case)
    if op in ("norm", "norm_bwd"):
        H = case["H"]
        st["x"] = _activations(T, H, g)
        st["w"] = (1.0 + _randn((H,), g, 0.1)).to(torch.bfloat16)
        st["eps"] = 1e-5
        r = _randn((T, H), g, 2.0).to(torch.bfloat16)
        if op == "norm":
            if case["residual"]:
                st["res"] = r
            if case["scaling"] == "delayed":
                st["scale"] = torch.full((1,), 8.0, device="cuda")
                st["amax"] = torch.zeros(1, device="cuda")
        else:
            st["dy"] = _randn((T, H), g, 1e-3).to(torch.bfloat16)
            if case["residual"]:
                st["dsum"] = _randn((T, H), g, 1e-3).to(torch.bfloat16)
            st["rstd"] = torch.rsqrt(st["x"].float().square().mean(-1) + st["eps"])
    elif op == "router":
        st["logits"] = _randn((T, case["E"]), g)
        st["dprobs"] = _randn((T, case["k"]), g, 1e-2)
    else:
        E, k, H, F = case["E"], case["k"], case["H"], case["F"]
        st["x"] = _activations(T, H, g)
        top = torch.topk(_randn((T, E), g), k, dim=-1)
        st["idx"] = top.indices.to(torch.int32)
        st["probs"] = torch.softmax(top.values, -1)
        st["w1"] = _weight(E, 2 * F, H, case["scaling"], g)
        st["w2"] = _weight(E, H, F, case["scaling"], g)
        if case["scaling"] == "delayed":            # calibrated scales of the activations
            st["xs"] = torch.full((1,), 2.0, device="cuda")
            st["hs"] = torch.full((1,), 4.0, device="cuda")
        elif case["scaling"] == "nvfp4":
            st["xs"] = torch.full((1,), 2688.0 / 243.7, device="cuda")
            st["hs"] = torch.full((1,), 2688.0 / 400.0, device="cuda")
    if own:
        _plan(st)
    return st


# ---------------------------------------------------------------------------
# the framework's own operators

def _plan(st):
    """Output buffers, workspace and operand descriptors, as a program keeps them."""
    from fp8_grouped_gemm_gb300 import mgq
    st["mgq"] = mgq
    op, T = st["op"], st["T"]
    u8 = dict(dtype=torch.uint8, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    if op == "norm":
        H = st["H"]
        st["y"], st["codes"] = torch.empty(T, H, **bf), torch.empty(T, H, **u8)
        st["rstd"] = torch.empty(T, device="cuda")
        st["sum"] = torch.empty(T, H, **bf) if st["residual"] else None
        if st["scaling"] == "mxfp8":
            st["sc"] = torch.empty(mgq.mx_scale_bytes(T, H), **u8)
            st["q"] = mgq.qdesc(mgq.E4M3, mgq.MX32_E8M0, st["codes"], st["sc"])
        elif st["scaling"] == "blockwise":
            st["sc"] = torch.empty(H // 128, T, device="cuda")
            st["q"] = mgq.qdesc(mgq.E4M3, mgq.BLK_1x128_F32, st["codes"], st["sc"])
        else:
            st["q"] = mgq.qdesc(mgq.E4M3, mgq.TENSOR_F32, st["codes"], tensor_scale=st["scale"], amax_out=st["amax"])
    elif op == "norm_bwd":
        H = st["H"]
        st["dx"], st["dw"] = torch.empty(T, H, **bf), torch.empty(H, device="cuda")
        st["ws"] = torch.empty(max(16, mgq.add_rmsnorm_bwd_workspace_size(T, H)), **u8)
    elif op == "router":
        st["idx"] = torch.empty(T, st["k"], dtype=torch.int32, device="cuda")
        st["probs"] = torch.empty(T, st["k"], device="cuda")
        st["dlogits"] = torch.empty_like(st["logits"])
        st["mode"] = mgq.SCORE_SOFTMAX if st["score"] == "softmax" else mgq.SCORE_SIGMOID
    else:
        E, k, H, F = st["E"], st["k"], st["H"], st["F"]
        st["sc"] = {"mxfp8": mgq.MX32_E8M0, "blockwise": mgq.BLK_1x128_F32, "delayed": mgq.TENSOR_F32,
                    "nvfp4": mgq.NV16_UE4M3}[st["scaling"]]
        dt = mgq.E2M1 if st["scaling"] == "nvfp4" else mgq.E4M3
        st["W1"] = mgq.operand(st["w1"]["codes"], st["w1"]["scale"], H, dt, st["w1"].get("global"))
        st["W2"] = mgq.operand(st["w2"]["codes"], st["w2"]["scale"], F, dt, st["w2"].get("global"))
        st["out"] = torch.empty(T, H, **bf)
        st["ws"] = torch.empty(mgq.moe_few_workspace_size(T, k, E, H, F, st["sc"]), **u8)


def _own_run(st):
    mgq, op = st["mgq"], st["op"]
    if op == "norm":
        mgq.add_rmsnorm_quantize(st["x"], st["w"], st["eps"], st["q"], residual=st.get("res"), sum_out=st["sum"],
                                 y=st["y"], rstd=st["rstd"])
        out = [st["y"], st["codes"].view(torch.float8_e4m3fn), st["rstd"]]
        if st["residual"]:
            out.append(st["sum"])
        if st["scaling"] == "mxfp8":
            out.append(st["sc"].view(torch.float8_e8m0fnu))
        elif st["scaling"] == "blockwise":
            out.append(st["sc"])
        else:
            out.append(st["amax"])
        return out
    if op == "norm_bwd":
        mgq.add_rmsnorm_bwd(st["dy"], st["x"], st["w"], st["rstd"], st["dx"], st["dw"], st["ws"],
                            dsum=st.get("dsum"))
        return [st["dx"], st["dw"]]
    if op == "router":
        mgq.router_topk(st["logits"], st["idx"], st["probs"], st["mode"], st["renorm"])
        if not st["train"]:
            return [st["idx"], st["probs"]]
        mgq.router_topk_bwd(st["logits"], st["idx"], st["dprobs"], st["dlogits"], st["mode"], st["renorm"])
        return [st["idx"], st["probs"], st["dlogits"]]
    mgq.moe_few_forward(st["x"], st["idx"], st["probs"], st["W1"], st["W2"], st["sc"], st["E"], st["F"], st["out"],
                        st["ws"], x_scale=st.get("xs"), h_scale=st.get("hs"))
    return [st["out"]]


# ---------------------------------------------------------------------------
# the plain forms

def _round_e2m1(v):
    """Nearest e2m1 value (ties to the even code), saturating at 6."""
    a = v.abs()
    q = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
    return torch.copysign(q.clamp(max=6.0), v)


def _pack_e2m1(v):
    """e2m1 values [..., 2n] -> bytes [..., n], element 2i in the low nibble."""
    a = v.abs()
    c = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c = c | (torch.signbit(v).to(torch.uint8) << 3)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _unpack_e2m1(b):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=b.device)
    return torch.stack([table[(b & 15).long()], table[(b >> 4).long()]], -1).flatten(-2)


def _cast_e4m3(v):
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _quant_rows(v, scaling, scale=None):
    """Row-wise quantisation of [..., K] values: (e4m3 codes, scales)."""
    if scaling == "mxfp8":
        b = v.unflatten(-1, (-1, 32))
        ex = _mx_exponent(b.abs().amax(-1))
        return _cast_e4m3(b * _pow2(-ex)[..., None]).flatten(-2), ex
    if scaling == "blockwise":
        b = v.unflatten(-1, (-1, 128))
        amax = b.abs().amax(-1)
        s = torch.where(amax == 0, 1.0, E4M3_MAX / amax)
        return _cast_e4m3(b * s[..., None]).flatten(-2), 1.0 / s
    return _cast_e4m3(v * scale), None


def _fake_quant(v, scaling, scale=None):
    """The values the quantised [..., K] rows stand for (NVFP4: times the global scale)."""
    if scaling == "nvfp4":
        b = v.unflatten(-1, (-1, 16))
        sc = (b.abs().amax(-1) / 6.0 * scale).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn).to(v.dtype)
        q = _round_e2m1(b * torch.where(sc == 0, 0.0, scale / sc)[..., None])
        return (q * sc[..., None]).flatten(-2) / scale
    c, s = _quant_rows(v, scaling, scale)
    c = c.to(v.dtype)
    if scaling == "mxfp8":
        return (c.unflatten(-1, (-1, 32)) * _pow2(s)[..., None]).flatten(-2)
    if scaling == "blockwise":
        return (c.unflatten(-1, (-1, 128)) * s[..., None]).flatten(-2)
    return c / scale


def _dequant(w, scaling, N, K, ids=None):
    """The values of the quantised weights of experts `ids` (all of them if None): [n, N, K]."""
    pick = (lambda t: t) if ids is None else (lambda t: t[ids])
    codes, scale = pick(w["codes"]), pick(w["scale"])
    n = codes.shape[0]
    if scaling in ("mxfp8", "nvfp4"):
        nb = K // (32 if scaling == "mxfp8" else 16)
        s = scale.view(n, N // 128, nb // 4, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(n, N, nb, 1)
    if scaling == "nvfp4":
        v = _unpack_e2m1(codes).view(n, N, nb, 16) * s.view(torch.float8_e4m3fn).float()
        return v.view(n, N, K) / pick(w["global"]).view(n, 1, 1)
    v = codes.view(torch.float8_e4m3fn).float()
    if scaling == "mxfp8":
        return (v.view(n, N, nb, 32) * _pow2(s.to(torch.int32) - 127)).view(n, N, K)
    if scaling == "blockwise":
        return (v.view(n, N // 128, 128, K // 128, 128) * scale[:, :, None, :, None]).view(n, N, K)
    return v / scale.view(n, 1, 1)


def _norm_plain(st):
    s = st["x"].float()
    if st["residual"]:
        s = s + st["res"].float()
    rstd = torch.rsqrt(s.square().mean(-1) + st["eps"])
    y = s * rstd[:, None] * st["w"].float()
    c, sc = _quant_rows(y, st["scaling"], st.get("scale"))
    out = [y.to(torch.bfloat16), c, rstd]
    if st["residual"]:
        out.append(s.to(torch.bfloat16))
    if st["scaling"] == "mxfp8":
        out.append(_tile_scales((sc + 127).to(torch.uint8)).view(torch.float8_e8m0fnu))
    elif st["scaling"] == "blockwise":
        out.append(sc.t().contiguous())
    else:
        out.append(y.abs().amax().reshape(1))
    return out


def _norm_bwd_plain(st):
    dy, s, r = st["dy"].float(), st["x"].float(), st["rstd"][:, None]
    xh = s * r
    g = dy * st["w"].float()
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    if st["residual"]:
        dx = dx + st["dsum"].float()
    return [dx.to(torch.bfloat16), (dy * xh).sum(0)]


def _router_plain(logits, dprobs, k, score, renorm, train):
    val, idx = torch.sort(logits, dim=-1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    if score == "softmax":
        sc = torch.softmax(logits, -1)
    else:
        sc = torch.sigmoid(logits)
    sel = torch.gather(sc, 1, idx)
    S = sel.sum(-1, keepdim=True)
    p = sel / S if renorm else sel
    if not train:
        return [idx.to(torch.int32), p]
    dsel = (dprobs - (dprobs * p).sum(-1, keepdim=True)) / S if renorm else dprobs
    d = torch.zeros_like(logits).scatter(1, idx, dsel)
    if score == "softmax":
        d = sc * (d - (d * sc).sum(-1, keepdim=True))
    else:
        d = d * sc * (1 - sc)
    return [idx.to(torch.int32), p, d]


def _few_plain(st):
    T, E, k, H, F, scaling = (st[n] for n in ("T", "E", "k", "H", "F", "scaling"))
    xq = _fake_quant(st["x"].float(), scaling, st.get("xs"))
    idx = st["idx"].long()
    if T * k <= E:
        # a weight gathered for every routed row
        ids = idx.reshape(-1)
        rows = xq[:, None, :].expand(T, k, H).reshape(T * k, H, 1)
        gu = torch.matmul(_dequant(st["w1"], scaling, 2 * F, H, ids), rows)[..., 0]
        h = _fake_quant(gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:], scaling, st.get("hs"))
        y = torch.matmul(_dequant(st["w2"], scaling, H, F, ids), h[..., None])[..., 0]
        out = (y.view(T, k, H) * st["probs"][..., None]).sum(1)
    else:
        # every expert on every token, weighted by its probability (0 where not chosen)
        gu = torch.matmul(xq, _dequant(st["w1"], scaling, 2 * F, H).transpose(1, 2))
        h = _fake_quant(gu[..., :F] * torch.sigmoid(gu[..., :F]) * gu[..., F:], scaling, st.get("hs"))
        y = torch.matmul(h, _dequant(st["w2"], scaling, H, F).transpose(1, 2))          # [E, T, H]
        p = torch.zeros(T, E, device="cuda").scatter(1, idx, st["probs"])
        out = (y * p.t()[..., None]).sum(0)
    return [out.to(torch.bfloat16)]


def run(state):
    if own:
        return _own_run(state)
    op = state["op"]
    if op == "norm":
        return _norm_plain(state)
    if op == "norm_bwd":
        return _norm_bwd_plain(state)
    if op == "router":
        return _router_plain(state["logits"], state["dprobs"], state["k"], state["score"], state["renorm"],
                             state["train"])
    return _few_plain(state)


# ---------------------------------------------------------------------------
# the definitions in float64, written apart from the plain forms

def _pow2_f64(e):
    """2^e as float64 from its bits, for integers e in the normal range."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3_f64(v):
    """Nearest e4m3 value of float64 values: the spacing is 2^(e-3) in [2^e, 2^(e+1)), 2^-9 below 2^-6."""
    a = v.abs().clamp(max=E4M3_MAX)
    _, e = torch.frexp(a)
    step = _pow2_f64((e - 1).clamp(min=-6) - 3)
    return torch.copysign(torch.round(a / step) * step, v)


def _e2m1_f64(v):
    a = v.abs().clamp(max=6.0)
    _, e = torch.frexp(a)
    step = _pow2_f64((e - 1).clamp(min=0) - 1)
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), v)


def _blocks_f64(v, scaling, scale):
    """Element values and block scales (value = element * scale)."""
    n = {"mxfp8": 32, "blockwise": 128, "nvfp4": 16, "delayed": v.shape[-1]}[scaling]
    b = v.reshape(*v.shape[:-1], -1, n)
    amax = b.abs().amax(-1, keepdim=True)
    if scaling == "mxfp8":
        m = _pow2_f64(torch.ceil(torch.log2(amax / E4M3_MAX)).clamp(-127, 127))
        return _e4m3_f64(b / m), m
    if scaling == "blockwise":
        m = torch.where(amax == 0, 1.0, amax / E4M3_MAX)
        return _e4m3_f64(b / m), m
    if scaling == "nvfp4":
        m = _e4m3_f64(amax / 6.0 * scale.double()) / scale.double()
        return _e2m1_f64(torch.where(m == 0, 0.0, b / m)), m
    return _e4m3_f64(b * scale.double()), (1.0 / scale.double()).expand_as(amax)


def _exact_norm(st):
    s = st["x"].double() + (st["res"].double() if st["residual"] else 0.0)
    rms = ((s * s).sum(-1) / st["H"] + st["eps"]).sqrt()
    y = s / rms[:, None] * st["w"].double()
    c, m = _blocks_f64(y, st["scaling"], st.get("scale"))
    out = [y, c.reshape(y.shape), 1.0 / rms]
    if st["residual"]:
        out.append(s)
    if st["scaling"] == "mxfp8":
        rp = (st["T"] + 127) // 128 * 128
        full = torch.full((rp, st["H"] // 32), 2.0 ** -127, dtype=torch.float64, device="cuda")
        full[: st["T"]] = m[..., 0]
        out.append(full.view(rp // 128, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).reshape(-1))
    elif st["scaling"] == "blockwise":
        out.append(m[..., 0].t().contiguous())
    else:
        out.append(y.abs().max().reshape(1))
    return out


def _exact_norm_bwd(st):
    s = st["x"].double().requires_grad_()
    w = st["w"].double().requires_grad_()
    xh = s * st["rstd"].double()[:, None]
    # rstd^-2 = mean(s^2) + eps: its gradient carried by an equal-valued expression
    ms = (s * s).sum(-1, keepdim=True) / st["H"]
    xh = s * st["rstd"].double()[:, None] * (1.0 - 0.5 * st["rstd"].double()[:, None] ** 2 * (ms - ms.detach()))
    total = (xh * w * st["dy"].double()).sum()
    if st["residual"]:
        total = total + (s * st["dsum"].double()).sum()
    dx, dw = torch.autograd.grad(total, (s, w))
    return [dx, dw]


def _exact_router(st):
    z = st["logits"].double().requires_grad_()
    k = st["k"]
    idx = torch.argsort(-z.detach(), dim=-1, stable=True)[:, :k]
    e = torch.exp(z - z.detach().amax(-1, keepdim=True)) if st["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-z))
    sel = e.gather(1, idx)
    if st["renorm"]:
        p = sel / sel.sum(-1, keepdim=True)
    else:
        p = sel / e.sum(-1, keepdim=True) if st["score"] == "softmax" else sel
    if not st["train"]:
        return [None, p.detach()]
    d, = torch.autograd.grad((p * st["dprobs"].double()).sum(), z)
    return [None, p.detach(), d]


def _weight_f64(w, scaling, e, N, K):
    """Expert e's weight [N, K] from the bits of its codes and the documented place of each scale."""
    c = w["codes"][e].to(torch.int64)
    r = torch.arange(N, device="cuda")[:, None]
    if scaling == "nvfp4":
        c = torch.stack([c & 15, c >> 4], -1).view(N, K)
        ef, mf = (c >> 1) & 3, (c & 1).double()
        v = torch.where(ef == 0, mf * 0.5, _pow2_f64(ef - 1) * (1 + mf / 2))
        v = torch.where(c >= 8, -v, v)
        b = torch.arange(K // 16, device="cuda")[None, :]
    else:
        ef, mf = (c >> 3) & 15, (c & 7).double()
        v = torch.where(ef == 0, mf * 2.0 ** -9, _pow2_f64(ef - 7) * (1 + mf / 8))
        v = torch.where(c >= 128, -v, v)
        b = torch.arange(K // 32, device="cuda")[None, :]
    sc = w["scale"][e]
    if scaling == "delayed":
        return v / sc.double()
    if scaling == "blockwise":
        return v * sc.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    nb = b.shape[1]
    s = sc[((r // 128) * (nb // 4) + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4].to(torch.int64)
    if scaling == "mxfp8":
        s = _pow2_f64(s - 127)
        return (v.view(N, nb, 32) * s[..., None]).view(N, K)
    es, ms = s >> 3, (s & 7).double()
    s = torch.where(es == 0, ms * 2.0 ** -9, _pow2_f64(es - 7) * (1 + ms / 8))
    return (v.view(N, nb, 16) * s[..., None]).view(N, K) / w["global"][e].double()


def _exact_few(st):
    T, E, k, H, F, scaling = (st[n] for n in ("T", "E", "k", "H", "F", "scaling"))
    idx, out = st["idx"].long(), torch.zeros(T, H, dtype=torch.float64, device="cuda")
    c, m = _blocks_f64(st["x"].double(), scaling, st.get("xs"))
    xq = (c * m).reshape(T, H)
    for e in idx.unique().tolist():
        t, j = (idx == e).nonzero(as_tuple=True)
        gu = xq[t] @ _weight_f64(st["w1"], scaling, e, 2 * F, H).t()
        h = gu[:, :F] / (1.0 + torch.exp(-gu[:, :F])) * gu[:, F:]
        c, m = _blocks_f64(h, scaling, st.get("hs"))
        y = (c * m).reshape(h.shape) @ _weight_f64(st["w2"], scaling, e, H, F).t()
        out.index_add_(0, t, y * st["probs"][t, j].double()[:, None])
    return [out]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    with torch.enable_grad():
        if op == "norm":
            return _exact_norm(st)
        if op == "norm_bwd":
            return _exact_norm_bwd(st)
        if op == "router":
            return _exact_router(st)
        return _exact_few(st)
