"""The 8-bit linear layer's operators: what is measured of them, and in which sizes.

Three operators that a transformer layer with 8-bit weights and activations chains:

``gemm``      C = act(sA_i sB_j (A B^T)_ij + beta C_ij + bias_j): a product of 8-bit integers with a scale
              for each token (row of A) and each channel (row of B, the weight stored N x K)
``quantize``  a float matrix to 8-bit integers with a scale for each row (activations), or for each
              column of a weight stored K x N, which it stores transposed ("columns")
``rmsnorm``   h = x + r, the residual stream's addition, and rmsnorm(h) * w in 8 bits with a scale for each row

``run`` computes them in elementary torch operations where ``own`` is false and calls the library where it
is true.  ``exact`` states their definitions in 64 bits.  8-bit results are returned as the values they
stand for, code times scale.

The scale of a quantised row is fl32(max |v| / 127), and the code is v / scale rounded to the nearest
integer, halves to even, with the quotient not rounded first.  A quotient rounded to 32 bits can fall on
a half that the quotient itself is next to, so the plain form divides in 64.  The normalised row is
quantised before its division by the root mean square, which is one number for the whole row: v = fl32(h w)
has the same codes, and its scale is multiplied by that number.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5


def _gemm(name, M, N, K, type, bias=False, relu=False, beta=0.0, packed=False):
    return dict(name=name, op="gemm", M=M, N=N, K=K, type=type, bias=bias, relu=relu, beta=beta,
                packed=packed)


def _quantize(name, M, K, type, columns=False):
    return dict(name=name, op="quantize", M=M, K=K, type=type, columns=columns)


def _rmsnorm(name, M, K, type, residual=True):
    return dict(name=name, op="rmsnorm", M=M, K=K, type=type, residual=residual)


def listed():
    return [
        # one sequence's next token through a square projection
        _gemm("gemm 1x4096x4096 bf16", 1, 4096, 4096, "bf16"),
        # sixteen sequences' next tokens through the feed-forward block's first product
        _gemm("gemm 16x11008x4096 bf16", 16, 11008, 4096, "bf16", bias=True, relu=True),
        # a ragged batch of 100 tokens through its second product, added to the residual stream
        _gemm("gemm 100x4096x11008 f16", 100, 4096, 11008, "f16", beta=1.0),
        # sizes that no tile divides, rows stored back to back and so without alignment
        _gemm("gemm 777x1234x4099 f32", 777, 1234, 4099, "f32", bias=True, packed=True),
        # the square product
        _gemm("gemm 4096x4096x4096 f32", 4096, 4096, 4096, "f32"),
        # a prompt of 2048 tokens through the feed-forward block's first product
        _gemm("gemm 2048x11008x4096 bf16", 2048, 11008, 4096, "bf16", bias=True, relu=True),
        # one token's hidden state
        _rmsnorm("rmsnorm 1x4096 bf16", 1, 4096, "bf16"),
        # a ragged batch with an odd width, and no residual, as before the first layer
        _rmsnorm("rmsnorm 777x5003 f32", 777, 5003, "f32", residual=False),
        # a long prompt
        _rmsnorm("rmsnorm 8192x4096 bf16", 8192, 4096, "bf16"),
        # a few sequences' activations before the feed-forward block's second product
        _quantize("quantize 16x11008 f16", 16, 11008, "f16"),
        # a prompt's
        _quantize("quantize 2048x11008 bf16", 2048, 11008, "bf16"),
        # a weight stored K x N in 32 bits, once when a model is loaded
        _quantize("quantize columns 11008x4096 f32", 11008, 4096, "f32", columns=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm; every other one a multiple of 16 where there is one."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 16:
        v -= v % 16
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "rmsnorm", "quantize"])
    type = rng.choice(["f32", "f16", "bf16"])
    if op == "gemm":
        while True:
            M, N, K = _spread(rng, 1, 4096), _spread(rng, 64, 11008), _spread(rng, 64, 11008)
            if M * N * K <= 2048 * 11008 * 4096:
                break
        c = _gemm("", M, N, K, type, rng.random() < 0.5, rng.random() < 0.5,
                  rng.choice([0.0, 0.0, 1.0, 0.5]), rng.random() < 0.3)
    else:
        while True:
            M, K = _spread(rng, 1, 8192), _spread(rng, 64, 16384)
            if M * K <= 8192 * 4096:
                break
        if op == "rmsnorm":
            c = _rmsnorm("", M, K, type, rng.random() < 0.7)
        else:
            c = _quantize("", M, K, type, rng.random() < 0.3)
    del c["name"]
    return c


def _codes(g, rows, cols, spread, packed):
    """8-bit codes with their scales, as quantising normal values with a few wide columns gives them; rows
    stored back to back, or each from a multiple of 16 bytes."""
    v = torch.randn(rows, cols, generator=g, device="cuda") * spread
    v[:, :: 97] *= 4.0
    s = v.abs().amax(1) / 127.0
    q = (v / s[:, None]).round_().clamp_(-127, 127)
    ld = cols if packed else -(-cols // 16) * 16
    out = torch.zeros(rows, ld, dtype=torch.int8, device="cuda")[:, :cols]
    out.copy_(q)
    return out, s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = _TYPES[case["type"]]
    M, K = case["M"], case["K"]
    st = dict(case)

    def normal(*shape, spread=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * spread

    def codes_out():
        # what the library writes: rows of codes from multiples of 16 bytes, and their scales
        st["Q"] = torch.empty(M, -(-K // 16) * 16, dtype=torch.int8, device="cuda")[:, :K]
        st["scales"] = torch.empty(M, device="cuda")

    if case["op"] == "gemm":
        N = case["N"]
        st["A"], st["sA"] = _codes(g, M, K, 1.0, case["packed"])
        st["B"], st["sB"] = _codes(g, N, K, 0.02, case["packed"])
        st["bias"] = normal(N, spread=0.1) if case["bias"] else None
        st["C0"] = normal(M, N).to(t) if case["beta"] else None
        st["C"] = torch.empty(M, N, dtype=t, device="cuda")
    elif case["op"] == "quantize":
        X = normal(K, M, spread=0.02) if case["columns"] else normal(M, K)
        X[3 if X.shape[0] > 3 else 0, :] *= 8.0
        st["X"] = X.to(t)
        codes_out()
    else:
        X = normal(M, K)
        X[:, :: 97] *= 10.0
        st["X"] = X.to(t)
        st["R"] = normal(M, K, spread=2.0).to(t) if case["residual"] else None
        st["W"] = (1.0 + normal(K, spread=0.1)).to(t)
        st["H"] = torch.empty(M, K, dtype=t, device="cuda") if case["residual"] else None
        codes_out()
    return st


def _own(st):
    import fp32_gemm_06_amd as fg
    M, K = st["M"], st["K"]
    type = {"f32": fg.TYPE_F32, "f16": fg.TYPE_F16, "bf16": fg.TYPE_BF16}[st["type"]]
    if st["op"] == "gemm":
        C = st["C"]
        if st["beta"]:
            C.copy_(st["C0"])  # the call updates C
        rc = fg.s8gemm(M, st["N"], K, st["A"], st["A"].stride(0), st["sA"], st["B"],
                       st["B"].stride(0), st["sB"], st["beta"], type, C, st["N"], st["bias"],
                       fg.ACT_RELU if st["relu"] else fg.ACT_NONE)
        out = C
    else:
        Q, scales = st["Q"], st["scales"]
        if st["op"] == "quantize":
            rc = fg.s8_quantize(fg.OP_T if st["columns"] else fg.OP_N, M, K, type, st["X"],
                                st["X"].stride(0), Q, Q.stride(0), scales)
            out = [Q * scales[:, None], scales]
        else:
            rc = fg.s8_rmsnorm(M, K, type, st["X"], K, st["R"], K, st["H"], K, st["W"], EPS, Q,
                               Q.stride(0), scales)
            out = [Q * scales[:, None], scales] + ([st["H"]] if st["residual"] else [])
    if rc:
        raise fg.Fp32GemmError(rc)
    return out


def _plain_codes(v):
    """(codes, scales) of the rows of a float32 matrix."""
    s = v.abs().amax(1).double()
    s = (s / torch.full_like(s, 127.0)).float()  # rounded once: torch divides by a number through its reciprocal
    q = (v.double() / s.double()[:, None]).round_().clamp_(-127.0, 127.0)
    return torch.where(s[:, None] > 0, q, 0.0).float(), s


def _plain(st):
    t = _TYPES[st["type"]]
    if st["op"] == "gemm":
        v = st["A"].float() @ st["B"].float().t()
        v = v * st["sA"][:, None] * st["sB"][None, :]
        if st["beta"]:
            v = v + st["beta"] * st["C0"].float()
        if st["bias"] is not None:
            v = v + st["bias"]
        if st["relu"]:
            v = torch.where(v < 0, 0.0, v)
        return v.to(t)
    if st["op"] == "quantize":
        X = st["X"].float()
        q, s = _plain_codes(X.t().contiguous() if st["columns"] else X)
        return [q * s[:, None], s]
    h = st["X"]
    if st["residual"]:
        h = (h.float() + st["R"].float()).to(t)
    f = h.float()
    rstd = 1.0 / torch.sqrt((f * f).mean(1) + EPS)
    q, s = _plain_codes(f * st["W"].float())
    s = s * rstd
    return [q * s[:, None], s] + ([h] if st["residual"] else [])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    M, K, b = case["M"], case["K"], _BYTES[case["type"]]
    if case["op"] == "gemm":
        N = case["N"]
        by = M * K + N * K + 4 * (M + N) + M * N * b * (2 if case["beta"] else 1)
        return {"bytes": by + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    codes = M * K + 4 * M
    if case["op"] == "quantize":
        return {"bytes": M * K * b + codes, "flops": 3 * M * K}
    return {"bytes": M * K * b * (3 if case["residual"] else 1) + K * b + codes, "flops": 7 * M * K}


def exact(case, seed):
    st = prepare(case, seed)
    t = _TYPES[case["type"]]
    d = torch.float64
    if case["op"] == "gemm":
        z = torch.mm(st["A"].to(d), st["B"].to(d).t().contiguous())
        z *= torch.outer(st["sA"].to(d), st["sB"].to(d))
        if st["C0"] is not None:
            z += case["beta"] * st["C0"].to(d)
        if st["bias"] is not None:
            z += st["bias"].to(d)[None, :]
        return z.clamp_min(0.0) if case["relu"] else z
    h = None
    if case["op"] == "quantize":
        v = st["X"].to(d)
        v = v.t() if case["columns"] else v
        factor = torch.ones(case["M"], dtype=d, device="cuda")
    else:
        h = st["X"].to(d)
        if st["R"] is not None:
            h = (h + st["R"].to(d)).to(t).to(d)  # the residual stream is kept in its type
        factor = torch.rsqrt((h ** 2).sum(1) / case["K"] + EPS)
        v = (h * st["W"].to(d)).to(torch.float32).to(d)
    top = torch.maximum(v.amax(1), -v.amin(1))
    step = (top / torch.tensor(127.0, dtype=d, device="cuda").expand_as(top)).to(torch.float32).to(d)
    code = torch.round(v / step.clamp_min(1e-300)[:, None])
    scale = step * factor
    out = [code * scale[:, None], scale]
    return out + [h] if case["op"] == "rmsnorm" and case["residual"] else out
