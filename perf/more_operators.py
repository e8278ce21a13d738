"""What stands between a decode step's QKV projection and its output projection: what is measured of it.

``rope``    norms of the queries and the keys, head by head, and the position rotation, in one pass
``store``   the same for a chunk of tokens whose keys and values go into a paged cache, in 8-bit codes with a
            scale for each token and head or in a float type, and the cache's rows of these tokens read back
            as floats (what the next products over the chunk read); without norm and rotation where the
            model has them elsewhere
``attend``  attention of one new token of each sequence over the paged cache

``run`` computes them in elementary torch operations where ``own`` is false and calls the library where it
is true.  ``exact`` states their definitions in 64 bits.

A cache is K and V, pages x heads x page size x head size, packed, with scales pages x heads x page size for
codes.  A token's slot is page * page size + offset.  Codes are those of a row of 32-bit values:
scale = max |v| / 127 rounded to 32 bits, code = v / scale to the nearest integer, halves to even, the quotient
not rounded first.  The row that is coded is the rotated key, computed in 64 bits and rounded once to 32, so
that no rounding on the way can move a value across a half; the angles are 64-bit products of position and
frequency, since far positions times 32-bit frequencies would lose whole turns' digits.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2, "s8": 1}
EPS = 1e-6


def _rope(name, T, Hq, Hk, D, type, R=None, pairs=False, norm=True, far=0):
    """R of the D values of a head turn (all by default), as halves or as neighbouring pairs; positions from ``far``."""
    return dict(name=name, op="rope", T=T, Hq=Hq, Hk=Hk, D=D, type=type, R=D if R is None else R, pairs=pairs,
                norm=norm, far=far)


def _store(name, T, Hq, Hk, D, type, cache, page, R=None, pairs=False, norm=True, far=0, rotate=True):
    return dict(_rope(name, T, Hq, Hk, D, type, R, pairs, norm, far), op="store", cache=cache, page=page, rotate=rotate)


def _attend(name, B, L, Hq, Hk, D, type, cache, page, window=0):
    """B sequences of L tokens and fewer (a lone one has L)."""
    return dict(name=name, op="attend", B=B, L=L, Hq=Hq, Hk=Hk, D=D, type=type, cache=cache, page=page, window=window)


def listed():
    return [
        # one sequence's next token, far into its text
        _rope("rope 1 x 32+8 x 128 bf16", 1, 32, 8, 128, "bf16", far=100000),
        # a ragged batch of tokens, a part of each head turning, in neighbouring pairs
        _rope("rope 777 x 12+4 x 80 f32", 777, 12, 4, 80, "f32", R=32, pairs=True),
        # a long prompt
        _rope("rope 8192 x 32+8 x 128 bf16", 8192, 32, 8, 128, "bf16"),
        # the next tokens of 64 sequences, into the 8-bit cache
        _store("store 64 x 32+8 x 128 bf16 s8", 64, 32, 8, 128, "bf16", "s8", 64, far=4000),
        # an odd chunk whose keys are ready as they are, into a cache of their own type
        _store("store 1001 x 0+16 x 64 f16 f16", 1001, 0, 16, 64, "f16", "f16", 16, rotate=False, norm=False),
        # a long prompt, into the 8-bit cache
        _store("store 8192 x 32+8 x 128 bf16 s8", 8192, 32, 8, 128, "bf16", "s8", 64),
        # one sequence: latency, and the split over its length
        _attend("attend 1 x 4096, 32/8 x 128 bf16 s8", 1, 4096, 32, 8, 128, "bf16", "s8", 64),
        # the same length with a key head for each query head, all in 32 bits
        _attend("attend 1 x 4096, 32/32 x 128 f32 f32", 1, 4096, 32, 32, 128, "f32", "f32", 128),
        # a few ragged sequences, odd heads, small odd pages
        _attend("attend 7 x 1000, 28/4 x 80 f32 s8", 7, 1000, 28, 4, 80, "f32", "s8", 24),
        # a sliding window over long sequences, one key head for all queries
        _attend("attend 16 x 16384, 16/1 x 256 f16 f16", 16, 16384, 16, 1, 256, "f16", "f16", 16, window=4096),
        # many sequences of all lengths
        _attend("attend 64 x 8192, 32/8 x 128 bf16 s8", 64, 8192, 32, 8, 128, "bf16", "s8", 64),
        # the same in 16 bits
        _attend("attend 64 x 8192, 32/8 x 128 bf16 bf16", 64, 8192, 32, 8, 128, "bf16", "bf16", 64),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "store", "attend", "attend"])
    type = rng.choice(["f32", "f16", "bf16"])
    while True:
        D = rng.choice([64, 80, 96, 128, 128, 192, 256])
        Hk = rng.choice([1, 2, 4, 5, 8, 16])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        page = rng.choice([16, 32, 64, 128, 24, 7])
        cache = rng.choice(["s8", "s8", type])
        Hq = Hk * group
        if op == "attend":
            L, B = _spread(rng, 1, 32768), _spread(rng, 1, 64)
            window = rng.choice([0, 0, _spread(rng, 1, L)])
            c = _attend("", B, L, Hq, Hk, D, type, cache, page, window)
            if Hq <= 64 and sum(_lengths(c)) * Hk * D * _BYTES[cache] <= 64 * 2900 * 8 * 128 * 2:
                break
        else:
            T = _spread(rng, 1, 8192)
            R = rng.choice([D, D, D // 2, 16])
            pairs, norm, far = rng.random() < 0.4, rng.random() < 0.7, rng.choice([0, 1000, 1000000])
            if T * (Hq + 2 * Hk) * D * _BYTES[type] > 8192 * 48 * 128 * 2:
                continue
            if op == "rope":
                c = _rope("", T, Hq, Hk, D, type, R, pairs, norm, far)
            else:
                rotate = rng.random() < 0.7
                c = _store("", T, Hq if rotate else 0, Hk, D, type, cache, page, R, pairs, norm and rotate, far, rotate)
            break
    del c["name"]
    return c


def _lengths(case):
    """The sequences' lengths: from a few tokens to L, more short than long."""
    B, L = case["B"], case["L"]
    return [max(1, round(L * ((i + 1) / B) ** 1.5)) for i in range(B)]


def _seen(case):
    """How many tokens each sequence's attention sees."""
    return [min(n, case["window"]) if case["window"] else n for n in _lengths(case)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = _TYPES[case["type"]]
    st = dict(case)
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]

    def normal(*shape, spread=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * spread

    def shuffled(n):
        return torch.randperm(n, generator=g, device="cuda")

    def cache_of(pages, fill):
        ps, kind = case["page"], case["cache"]
        for name in ("k", "v"):
            if kind == "s8":
                codes = torch.zeros(pages, Hk, ps, D, dtype=torch.int8, device="cuda")
                scales = torch.zeros(pages, Hk, ps, device="cuda")
                if fill:
                    for p0 in range(0, pages, 4096):
                        x = normal(*codes[p0:p0 + 4096].shape)
                        s = x.abs().amax(-1) / 127.0
                        codes[p0:p0 + 4096] = (x / s[..., None]).round_().clamp_(-127, 127)
                        scales[p0:p0 + 4096] = s
                st[name], st[name + "_scale"] = codes, scales
            else:
                x = torch.zeros(pages, Hk, ps, D, dtype=t, device="cuda")
                if fill:
                    for p0 in range(0, pages, 4096):
                        x[p0:p0 + 4096] = normal(*x[p0:p0 + 4096].shape)
                st[name], st[name + "_scale"] = x, None

    if case["op"] == "attend":
        B, ps = case["B"], case["page"]
        lengths = torch.tensor(_lengths(case), device="cuda")[shuffled(B)]
        width = -(-case["L"] // ps)
        used = torch.arange(width, device="cuda")[None, :] < ((lengths + ps - 1) // ps)[:, None]
        pages = int(used.sum())
        table = torch.zeros(B, width, dtype=torch.int64, device="cuda")
        table[used] = shuffled(pages)  # a sequence's pages lie anywhere
        st["table"], st["lengths"] = table.int(), lengths.int()
        cache_of(pages, True)
        # queries about three times a unit vector's spread: a softmax that is neither flat nor a single token
        st["q"] = normal(B, Hq * D, spread=3.0).to(t)
        st["out"] = torch.empty(B, Hq * D, dtype=t, device="cuda")
        st["lse"] = torch.empty(B, Hq, device="cuda")
        return st
    T = case["T"]
    # queries, keys and values as the projection leaves them: one row a token, some features large
    x = normal(T, (Hq + 2 * Hk) * D)
    x[:, :: 61] *= 6.0
    st["x"] = x.to(t)
    st["wq"], st["wk"] = ((1.0 + normal(D, spread=0.2)).to(t) if case["norm"] else None for _ in range(2))
    R = case["R"]
    st["freq"] = 10000.0 ** (torch.arange(R // 2, dtype=torch.float64, device="cuda") * (-2.0 / R))
    st["pos"] = (case["far"] + torch.arange(T, device="cuda")).int()
    st["yq"] = torch.empty(T, Hq * D, dtype=t, device="cuda")
    if case["op"] == "rope":
        st["yk"] = torch.empty(T, Hk * D, dtype=t, device="cuda")
        return st
    pages = -(-T // case["page"]) + 3
    cache_of(pages, False)
    st["slots"] = shuffled(pages * case["page"])[:T].int()
    if T > 64:  # a prompt's tokens follow each other
        st["slots"] = (case["page"] + torch.arange(T, device="cuda")).int()
    st["kr"], st["vr"] = (torch.empty(T, Hk * D, dtype=t, device="cuda") for _ in range(2))
    return st


def _handle(st, fg):
    """The cache as the library takes it; a program makes it once."""
    if "handle" not in st:
        st["handle"] = fg.KVCache(st["k"], st["v"], st["k_scale"], st["v_scale"])
    return st["handle"]


def _own(st):
    import fp32_gemm_06_amd as fg
    type = {"f32": fg.TYPE_F32, "f16": fg.TYPE_F16, "bf16": fg.TYPE_BF16}[st["type"]]
    Hq, Hk, D = st["Hq"], st["Hk"], st["D"]
    if st["op"] == "attend":
        cache, B = _handle(st, fg), st["B"]
        if "workspace" not in st:
            size = fg.kv_attention_workspace_size(B, Hq, cache)
            st["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
        rc = fg.kv_attention(B, type, Hq, st["q"], Hq * D, cache, st["table"], st["table"].shape[1], st["lengths"],
                             st["window"], D ** -0.5, st["out"], Hq * D, st["lse"], st["workspace"],
                             st["workspace"].numel())
        if rc:
            raise fg.Fp32GemmError(rc)
        return [st["out"], st["lse"]]
    x, T, ld = st["x"], st["T"], st["x"].stride(0)
    q = x.data_ptr()
    k = q + Hq * D * x.element_size()
    v = k + Hk * D * x.element_size()
    style = fg.ROPE_PAIRS if st["pairs"] else fg.ROPE_HALVES
    if st["op"] == "rope":
        rc = fg.qk_norm_rope(T, D, type, Hq, q, ld, st["yq"], Hq * D, st["wq"], Hk, k, ld, st["yk"], Hk * D, st["wk"],
                             EPS, st["R"], style, st["freq"], st["pos"])
        out = [st["yq"], st["yk"]]
    else:
        cache = _handle(st, fg)
        if st["rotate"]:
            rc = fg.qkv_rope_write(T, type, Hq, q, ld, st["yq"], Hq * D, st["wq"], k, ld, st["wk"], v, ld, EPS,
                                   st["R"], style, st["freq"], st["pos"], st["slots"], cache)
        else:
            rc = fg.kv_write(T, type, k, ld, v, ld, st["slots"], cache)
        rc = rc or fg.kv_read(T, st["slots"], cache, type, st["kr"], Hk * D, st["vr"], Hk * D)
        out = [st["kr"], st["vr"]] + ([st["yq"]] if st["rotate"] else [])
    if rc:
        raise fg.Fp32GemmError(rc)
    return out


def _plain_rope(x, w, st, t):
    """(T, H, D) values, normalised and turned, as float64 or (t given) rounded to t."""
    d = x.double() if t is None else x.float()
    if w is not None:
        d = d * (1.0 / torch.sqrt((d * d).mean(-1, keepdim=True) + EPS)) * w.to(d.dtype)
    R = st["R"]
    angle = st["pos"].double()[:, None] * st["freq"][None, :]
    c, s = torch.cos(angle).to(d.dtype)[:, None, :], torch.sin(angle).to(d.dtype)[:, None, :]
    y = d.clone()
    if st["pairs"]:
        a, b = d[..., 0:R:2], d[..., 1:R:2]
        y[..., 0:R:2], y[..., 1:R:2] = a * c - b * s, b * c + a * s
    else:
        a, b = d[..., :R // 2], d[..., R // 2:R]
        y[..., :R // 2], y[..., R // 2:R] = a * c - b * s, b * c + a * s
    return y if t is None else y.to(t)


def _plain_stored(rows, st, name):
    """Rows (T, Hk, D) put into the cache, and read back."""
    t, ps = _TYPES[st["type"]], st["page"]
    slots = st["slots"].long()
    page, at = slots // ps, slots % ps
    if st["cache"] != "s8":
        st[name][page, :, at] = rows.to(t)
        return st[name][page, :, at].reshape(rows.shape[0], -1)
    v = rows.float()
    top = v.abs().amax(-1).double()
    scale = (top / torch.full_like(top, 127.0)).float()
    code = (v.double() / scale.double()[..., None]).round_().clamp_(-127.0, 127.0)
    code = torch.where(scale[..., None] > 0, code, 0.0)
    st[name][page, :, at], st[name + "_scale"][page, :, at] = code.to(torch.int8), scale
    got = st[name][page, :, at].float() * st[name + "_scale"][page, :, at][..., None]
    return got.to(t).reshape(rows.shape[0], -1)


def _plain_attend(st):
    t = _TYPES[st["type"]]
    B, Hq, Hk, D, ps = st["B"], st["Hq"], st["Hk"], st["D"], st["page"]
    n = st["lengths"].long()
    table = st["table"].long()
    width = table.shape[1]
    token = torch.arange(width * ps, device="cuda")[None, :]
    seen = token < n[:, None]
    if st["window"]:
        seen = seen & (token >= n[:, None] - st["window"])

    def rows(name):
        x = st[name][table].float()  # B, width, Hk, ps, D
        if st[name + "_scale"] is not None:
            x *= st[name + "_scale"][table][..., None]
        return x.transpose(1, 2).reshape(B, Hk, width * ps, D)

    q = st["q"].float().view(B, Hk, Hq // Hk, D)
    s = torch.matmul(q, rows("k").transpose(2, 3).contiguous()) * D ** -0.5
    s = torch.where(seen[:, None, None, :], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, rows("v")) / total
    return [o.reshape(B, Hq * D).to(t), (m + torch.log(total)).reshape(B, Hq)]


def _plain(st):
    if st["op"] == "attend":
        return _plain_attend(st)
    t, T, Hq, Hk, D = _TYPES[st["type"]], st["T"], st["Hq"], st["Hk"], st["D"]
    q, k, v = st["x"].view(T, -1, D).split([Hq, Hk, Hk], 1)
    if st["op"] == "rope":
        return [_plain_rope(q, st["wq"], st, t).reshape(T, -1), _plain_rope(k, st["wk"], st, t).reshape(T, -1)]
    if st["rotate"]:
        out = [_plain_stored(_plain_rope(k, st["wk"], st, None), st, "k"), _plain_stored(v, st, "v")]
        return out + [_plain_rope(q, st["wq"], st, t).reshape(T, -1)]
    return [_plain_stored(k, st, "k"), _plain_stored(v, st, "v")]


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    Hq, Hk, D, b = case["Hq"], case["Hk"], case["D"], _BYTES[case["type"]]
    if case["op"] == "attend":
        n = sum(_seen(case))
        row = 2 * D * _BYTES[case["cache"]] + (8 if case["cache"] == "s8" else 0)
        return {"bytes": n * Hk * row + case["B"] * Hq * (2 * D * b + 4), "flops": 4 * n * Hq * D}
    T = case["T"]
    if case["op"] == "rope":
        return {"bytes": 2 * T * (Hq + Hk) * D * b + 4 * T, "flops": 8 * T * (Hq + Hk) * D}
    stored = 2 * Hk * (D * _BYTES[case["cache"]] + (4 if case["cache"] == "s8" else 0))
    return {"bytes": T * (Hq * 2 + Hk * 2 + Hk * 2) * D * b + 2 * T * stored + 4 * T,
            "flops": T * (8 * (Hq + Hk) + 4 * Hk) * D}


def exact(case, seed):
    st = prepare(case, seed)
    f8 = torch.float64
    t, Hq, Hk, D = _TYPES[case["type"]], case["Hq"], case["Hk"], case["D"]
    if case["op"] == "attend":
        ps, out, lses = case["page"], [], []
        for b, n in enumerate(st["lengths"].tolist()):
            lo = max(0, n - case["window"]) if case["window"] else 0
            at = torch.arange(lo, n, device="cuda")
            page, off = st["table"][b].long()[at // ps], at % ps
            k, v = (st[x][page, :, off].to(f8).permute(1, 0, 2).contiguous() for x in ("k", "v"))  # Hk, n, D
            if case["cache"] == "s8":
                k *= st["k_scale"][page, :, off].to(f8).t()[..., None]
                v *= st["v_scale"][page, :, off].to(f8).t()[..., None]
            q = st["q"][b].to(f8).view(Hk, Hq // Hk, D)
            s = torch.bmm(k, q.transpose(1, 2).contiguous()).transpose(1, 2).contiguous() / math.sqrt(D)
            lse = torch.logsumexp(s, -1)
            out.append(torch.bmm(torch.exp(s - lse[..., None]), v).reshape(Hq * D))
            lses.append(lse.reshape(Hq))
        return [torch.stack(out), torch.stack(lses)]

    def turned(x, w):
        x = x.to(f8)
        if w is not None:
            x = x * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS) * w.to(f8)
        R = case["R"]
        turn = torch.polar(torch.ones_like(st["freq"]), torch.zeros_like(st["freq"]))
        turn = torch.polar(turn.real.expand(case["T"], -1), torch.outer(st["pos"].to(f8), st["freq"]))[:, None, :]
        if case["pairs"]:
            z = torch.view_as_complex(x[..., :R].reshape(*x.shape[:2], R // 2, 2).contiguous()) * turn
            z = torch.view_as_real(z).reshape(*x.shape[:2], R)
        else:
            z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * turn
            z = torch.cat([z.real, z.imag], -1)
        return torch.cat([z, x[..., R:]], -1)

    def kept(x):
        if case["cache"] != "s8":
            return x.to(t).to(f8).flatten(1)
        x = x.to(torch.float32).to(f8)
        top = torch.maximum(x.amax(-1), -x.amin(-1))
        step = (top / torch.tensor(127.0, dtype=f8, device="cuda").expand_as(top)).to(torch.float32).to(f8)
        return (torch.round(x / step.clamp_min(1e-300)[..., None]) * step[..., None]).flatten(1)

    x = st["x"].view(case["T"], -1, D)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    if case["op"] == "rope":
        return [turned(q, st["wq"]).flatten(1), turned(k, st["wk"]).flatten(1)]
    if not case["rotate"]:
        return [kept(k), kept(v)]
    return [kept(turned(k, st["wk"])), kept(v), turned(q, st["wq"]).flatten(1)]
