"""The unpadded products of the routed experts, as cases to time and to compare.

Operators: the bf16 products grouped by expert over ragged groups (forward
"fwd", the gradient of the rows "dgrad", of the weights "wgrad"), the same
forward product over 8-bit integers with a scale for each token and each output
channel ("int8"; one group: a plain matrix product) and the row quantiser that
makes such codes ("quant8").

Each case runs either the plain form below (elementary torch operations in
float32) or, with `own` set, the library's entry points; `exact` restates the
definitions in float64.
"""
import math

import torch

own = False

# ---------------------------------------------------------------------------
# cases: T tokens, k experts a token, E experts (k = E = 1: a plain product); N outputs and K inputs of
# every expert's weight; skew: the experts' popularity (0 even, 1 Zipf)


def listed():
    return [
        # one new token through eight of the fine-grained experts' gate/up weights: the smallest weight read
        dict(name="fwd_finegrained_T1", op="fwd", T=1, k=8, E=128, N=1536, K=2048, skew=0.0, out="bf16"),
        # a ragged prompt of the Mixtral-shaped layer, gate/up
        dict(name="fwd_mixtral_T1003", op="fwd", T=1003, k=2, E=8, N=28672, K=4096, skew=1.0, out="bf16"),
        # the training batch of the Mixtral-shaped layer, gate/up: the largest product
        dict(name="fwd_mixtral_T16384", op="fwd", T=16384, k=2, E=8, N=28672, K=4096, skew=0.0, out="bf16"),
        # gradient of the rows: a short micro-batch spread over all fine-grained experts (about 60 rows each)
        dict(name="dgrad_finegrained_T1003", op="dgrad", T=1003, k=8, E=128, N=1536, K=2048, skew=0.0, out="bf16"),
        # and the Mixtral-shaped down projection's training batch
        dict(name="dgrad_mixtral_T16384", op="dgrad", T=16384, k=2, E=8, N=4096, K=14336, skew=0.0, out="bf16"),
        # gradient of the weights: the fine-grained down projection over uneven groups of odd sizes
        dict(name="wgrad_finegrained_T1003", op="wgrad", T=1003, k=8, E=128, N=2048, K=768, skew=1.0, out="f32"),
        # and the Mixtral-shaped down projection's training batch, float32 gradients
        dict(name="wgrad_mixtral_T16384", op="wgrad", T=16384, k=2, E=8, N=4096, K=14336, skew=0.0, out="f32"),
        # a decode batch of 16 tokens on the Mixtral-shaped gate/up weights in int8
        dict(name="int8_mixtral_T16", op="int8", T=16, k=2, E=8, N=28672, K=4096, skew=0.0, out="bf16"),
        # a plain int8 product (one group) of a ragged prompt, the Scout-shaped gate/up
        dict(name="int8_plain_1003", op="int8", T=1003, k=1, E=1, N=16384, K=5120, skew=0.0, out="bf16"),
        # the Mixtral-shaped down projection of a long prompt in int8, float32 result
        dict(name="int8_mixtral_T16384", op="int8", T=16384, k=2, E=8, N=4096, K=14336, skew=0.0, out="f32"),
        # token scales of one new token, and of a long prompt
        dict(name="quant8_1x4096", op="quant8", T=1, K=4096),
        dict(name="quant8_16384x4096", op="quant8", T=16384, K=4096),
    ]


_LARGEST_WEIGHT = 8 * 28672 * 4096          # elements
_LARGEST_MACS = 32768 * 28672 * 4096


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "dgrad", "wgrad", "int8", "int8", "quant8"])
    if op == "quant8":
        K = 16 * _log_int(rng, 4, 1024)
        return dict(op=op, T=max(1, min(_log_int(rng, 1, 32768), 16384 * 4096 // K)), K=K)
    E = _log_int(rng, 1, 128)
    k = rng.randint(1, min(8, E))
    unit = 16 if op == "int8" else 8
    N, K = 8 * _log_int(rng, 16, 3584), unit * _log_int(rng, 128 // unit, 14336 // unit)
    T = _log_int(rng, 1, 32768 // k)
    while E * N * K > _LARGEST_WEIGHT // 2:
        E = max(1, E // 2)
        k = min(k, E)
        if E == 1:
            break
    while T * k * N * K > _LARGEST_MACS // 2:
        T = max(1, T // 2)
    out = rng.choice(["f32", "f32", "bf16"] if op == "wgrad" else ["bf16", "bf16", "f32"])
    return dict(op=op, T=T, k=k, E=E, N=N, K=K, skew=rng.choice([0.0, 1.0]), out=out)


def work(case):
    T, K = case["T"], case["K"]
    if case["op"] == "quant8":
        return {"bytes": 3 * T * K + 4 * T, "flops": 3 * T * K}
    E, k, N, op = case["E"], case["k"], case["N"], case["op"]
    R = T * k
    ob = 2 if case["out"] == "bf16" else 4
    active = min(E, R) if case["skew"] else E * (1 - (1 - k / E) ** T)     # experts with a row, on average
    if op == "wgrad":
        b = 2 * R * (N + K) + ob * E * N * K
    elif op == "int8":
        b = R * K + active * N * K + ob * R * N + 4 * R + 4 * active * N
    else:
        rows_in, rows_out = (K, N) if op == "fwd" else (N, K)
        b = 2 * R * rows_in + 2 * active * N * K + ob * R * rows_out
    return {"bytes": int(b), "flops": 2 * R * N * K}


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


def _weights(E, N, K, g):
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        w[e] = _randn((N, K), g, 0.02)
    return w


def _codes(x):
    """int8 codes and scale of every row of a float32 matrix."""
    amax = x.abs().amax(-1, keepdim=True)
    return torch.round(x * (127.0 / amax)).to(torch.int8), (amax / 127.0)[..., 0]


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    T, K, op = case["T"], case["K"], case["op"]
    if op == "quant8":
        st["x"] = _activations(T, K, g)
    else:
        E, k, N = case["E"], case["k"], case["N"]
        R = T * k
        # every token takes its k best experts
        logits = _randn((T, E), g)
        if case["skew"]:
            logits -= case["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
        ids = torch.topk(logits, k, dim=-1).indices.reshape(-1)
        counts = torch.bincount(ids, minlength=E)
        st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        st["bounds"] = st["offsets"].tolist()               # the plain form's loop
        if op in ("dgrad", "wgrad"):
            st["dy"] = _randn((R, N), g, 1e-3).to(torch.bfloat16)
        if op in ("fwd", "wgrad"):
            st["x"] = _activations(R, K, g)
        if op in ("fwd", "dgrad"):
            st["w"] = _weights(E, N, K, g)
        if op == "int8":
            st["xq"], st["xs"] = _codes(_activations(R, K, g).float())
            st["wq"] = torch.empty(E, N, K, dtype=torch.int8, device="cuda")
            st["ws"] = torch.empty(E, N, device="cuda")
            for e in range(E):
                st["wq"][e], st["ws"][e] = _codes(_randn((N, K), g, 0.02))
    if own:
        _plan(st)
    return st


# ---------------------------------------------------------------------------
# the framework's own operators

def _plan(st):
    """Result buffers, as a program keeps them."""
    from fp8_grouped_gemm_gb300 import mgq
    st["mgq"] = mgq
    op, T, K = st["op"], st["T"], st["K"]
    if op == "quant8":
        st["codes"] = torch.empty(T, K, dtype=torch.int8, device="cuda")
        st["scale"] = torch.empty(T, device="cuda")
        return
    E, N, R = st["E"], st["N"], T * st["k"]
    shape = {"fwd": (R, N), "int8": (R, N), "dgrad": (R, K), "wgrad": (E, N, K)}[op]
    st["out_buf"] = torch.empty(shape, dtype=torch.bfloat16 if st["out"] == "bf16" else torch.float32, device="cuda")


def _own_run(st):
    mgq, op = st["mgq"], st["op"]
    if op == "quant8":
        mgq.rows_quantize_int8(st["x"], st["codes"], st["scale"])
        return [st["codes"], st["scale"]]
    off = None if st["E"] == 1 else st["offsets"]
    if op == "fwd":
        mgq.ragged_gemm_fwd(st["x"], st["w"], off, st["out_buf"])
    elif op == "dgrad":
        mgq.ragged_gemm_dgrad(st["dy"], st["w"], off, st["out_buf"])
    elif op == "wgrad":
        mgq.ragged_gemm_wgrad(st["dy"], st["x"], off, st["out_buf"])
    else:
        mgq.ragged_gemm_int8(st["xq"], st["xs"], st["wq"], st["ws"], off, st["out_buf"])
    return [st["out_buf"]]


# ---------------------------------------------------------------------------
# the plain forms

def _plain_run(st):
    op = st["op"]
    if op == "quant8":
        x = st["x"].double()                     # (quotients that end in a half are ties: exact in 64 bits)
        amax = x.abs().amax(-1, keepdim=True)
        codes = torch.round(x * 127.0 / torch.where(amax == 0, 1.0, amax))
        return [codes.to(torch.int8), (amax[:, 0] / 127.0).float()]
    dt = torch.bfloat16 if st["out"] == "bf16" else torch.float32
    b, E, N, K = st["bounds"], st["E"], st["N"], st["K"]
    R = b[-1]
    if op == "wgrad":
        out = torch.zeros(E, N, K, dtype=dt, device="cuda")
        dy, x = st["dy"].float(), st["x"].float()
        for e in range(E):
            if b[e + 1] > b[e]:
                out[e] = torch.matmul(dy[b[e]:b[e + 1]].t(), x[b[e]:b[e + 1]])
        return [out]
    out = torch.empty(R, K if op == "dgrad" else N, dtype=dt, device="cuda")
    for e in range(E):
        lo, hi = b[e], b[e + 1]
        if lo == hi:
            continue
        if op == "fwd":
            out[lo:hi] = torch.matmul(st["x"][lo:hi].float(), st["w"][e].float().t())
        elif op == "dgrad":
            out[lo:hi] = torch.matmul(st["dy"][lo:hi].float(), st["w"][e].float())
        else:
            acc = torch.matmul(st["xq"][lo:hi].float(), st["wq"][e].float().t())
            out[lo:hi] = acc * st["xs"][lo:hi, None] * st["ws"][e]
    return [out]


def run(state):
    return _own_run(state) if own else _plain_run(state)


# ---------------------------------------------------------------------------
# the definitions in float64, written apart from the plain forms

def _half_even(q):
    """Nearest integer of float64 values, a half to the even neighbour."""
    lo = torch.floor(q)
    d = q - lo
    up = (d > 0.5) | ((d == 0.5) & (torch.remainder(lo, 2.0) == 1.0))
    return lo + up.double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quant8":
        x = st["x"].double()
        amax = torch.maximum(x.amax(1), -x.amin(1))
        q = _half_even(127.0 * x / amax.clamp(min=1e-300)[:, None])
        return [q.to(torch.int8), amax / 127.0]
    E, N, K = case["E"], case["N"], case["K"]
    off = st["offsets"].long()
    group = torch.bucketize(torch.arange(int(off[-1]), device="cuda"), off[1:], right=True)
    if op == "wgrad":
        out = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
    else:
        out = torch.zeros(len(group), K if op == "dgrad" else N, dtype=torch.float64, device="cuda")
    for e in range(E):
        r = (group == e).nonzero()[:, 0]
        if not len(r):
            continue
        if op == "fwd":
            out[r] = torch.einsum("rk,nk->rn", st["x"][r].double(), st["w"][e].double())
        elif op == "dgrad":
            out[r] = torch.einsum("rn,nk->rk", st["dy"][r].double(), st["w"][e].double())
        elif op == "wgrad":
            out[e] = torch.einsum("rn,rk->nk", st["dy"][r].double(), st["x"][r].double())
        else:
            x = st["xq"][r].double() * st["xs"][r].double()[:, None]
            out[r] = torch.einsum("rk,nk->rn", x, st["wq"][e].double() * st["ws"][e].double()[:, None])
    return [out]
