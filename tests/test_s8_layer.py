"""The 8-bit operators together, as a transformer's feed-forward block uses them, through the torch
wrappers; under graph capture, on other streams, and with calls the wrappers refuse."""
import pytest
import torch

import fp32_gemm_06_amd as fg
import s8_reference as ref
from gpu_util import require_gpu

gpu = pytest.mark.gpu
TYPE_OF = {d: t for t, d in ref.TYPES.items()}


def weights(D, F, dtype, seed=0):
    """Norm weight, two projections stored N x K and K x N in fp32, and the first one's bias."""
    g = torch.Generator().manual_seed(seed)
    return ((1 + 0.1 * torch.randn(D, generator=g)).to(dtype), torch.randn(F, D, generator=g) * D ** -0.5,
            torch.randn(F, D, generator=g) * F ** -0.5, 0.1 * torch.randn(F, generator=g))


def block(x, r, w, q1, s1, b1, q2, s2, stream=None):
    """h = x + r; h + relu(rmsnorm(h) W1 + b1) W2, products in 8 bits."""
    cx, sx, h = fg.rmsnorm_s8(x, w, 1e-5, residual=r, stream=stream)
    u = fg.gemm_s8(cx, sx, q1.t(), s1, dtype=x.dtype, bias=b1, act="relu", stream=stream)
    cu, su = fg.quantize_s8(u, stream=stream)
    y = h.clone() if stream is None else None
    if y is None:
        with torch.cuda.stream(stream):
            y = h.clone()
    fg.gemm_s8(cu, su, q2.t(), s2, C=y, beta=1.0, stream=stream)
    return dict(cx=cx, sx=sx, h=h, u=u, cu=cu, su=su, y=y)


@gpu
@pytest.mark.parametrize("dtype", list(ref.TYPES.values()), ids=str)
@pytest.mark.parametrize("M,D,F", [(1, 512, 1376), (7, 333, 1001), (130, 1024, 2752)])
def test_block_step_by_step(M, D, F, dtype):
    """Each step against its 64-bit reference on the inputs the step got, and the first product against
    the layer without codes, within what half a step of both operands' codes can add up to."""
    require_gpu()
    type = TYPE_OF[dtype]
    g = torch.Generator().manual_seed(M)
    x, r = (torch.randn(M, D, generator=g).to(dtype) for _ in range(2))
    w, W1, W2, b1 = weights(D, F, dtype)
    q1, s1 = fg.quantize_s8(W1.cuda())
    q2, s2 = fg.quantize_s8(W2.cuda().t())  # stored K x N = F x D: the codes are D x F
    assert q1.shape == (F, D) and q2.shape == (D, F) and q2.stride(0) % 16 == 0
    for W, q, s in ((W1, q1, s1), (W2.t(), q2, s2)):
        wq, ws = ref.codes(W.double())
        assert torch.equal(q.cpu().long(), wq) and torch.equal(s.cpu(), ws)
    o = {k: v.cpu() for k, v in block(x.cuda(), r.cuda(), w.cuda(), q1, s1, b1.cuda(), q2, s2).items()}
    h, cx, _, sx = ref.rmsnorm(x, r, w, 1e-5)
    assert torch.equal(o["h"], h) and torch.equal(o["cx"].long(), cx)
    assert bool(((o["sx"].double() - sx).abs() <= sx * (ref.U32 + 1e-11)).all())
    z, bound = ref.gemm(o["cx"], o["sx"], q1.cpu(), s1.cpu(), 0.0, None, b1, True, type)
    assert bool(((o["u"].double() - z).abs() <= bound).all())
    cu, su = ref.codes(o["u"].double())
    assert torch.equal(o["cu"].long(), cu) and torch.equal(o["su"], su)
    z2, bound2 = ref.gemm(o["cu"], o["su"], q2.cpu(), s2.cpu(), 1.0, o["h"], None, False, type)
    assert bool(((o["y"].double() - z2).abs() <= bound2).all())
    # the first product without codes
    a = h.double() / torch.sqrt((h.double() ** 2).mean(1, keepdim=True) + 1e-5) * w.double()
    b = W1.double()
    full = torch.clamp(a @ b.t() + b1.double(), min=0.0)
    da, db = sx[:, None] * 0.5001, s1.cpu().double()[None, :] * 0.5001
    codes_bound = a.abs().sum(1)[:, None] * db + da * b.abs().sum(1)[None, :] + D * da * db
    assert bool(((o["u"].double() - full).abs() <= codes_bound + bound).all())


@gpu
def test_block_captured_in_two_graphs_replays_with_eager_work_between():
    """Two graphs of the block, replayed in turn and together with eager calls; every replay equals the
    eager result bit for bit (the operators share no scratch)."""
    require_gpu()
    dtype, D, F = torch.bfloat16, 512, 1376
    w, W1, W2, b1 = weights(D, F, dtype)
    q1, s1 = fg.quantize_s8(W1.cuda())
    q2, s2 = fg.quantize_s8(W2.cuda().t())
    args = (w.cuda(), q1, s1, b1.cuda(), q2, s2)
    made = []
    for M in (3, 70):
        x, r = torch.empty(M, D, dtype=dtype, device="cuda"), torch.empty(M, D, dtype=dtype, device="cuda")
        x.normal_()
        r.normal_()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            block(x, r, *args)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = block(x, r, *args)
        made.append((x, r, graph, out))
    other = torch.cuda.Stream()
    for turn in range(4):
        for x, r, _, _ in made:
            x.normal_()
            r.normal_()
        torch.cuda.synchronize()
        made[0][2].replay()
        with torch.cuda.stream(other):
            made[1][2].replay()
        eager = [block(x, r, *args) for x, r, _, _ in made]
        torch.cuda.synchronize()
        for (x, r, graph, out), want in zip(made, eager):
            for k in want:
                assert torch.equal(out[k], want[k]), (turn, k)


@gpu
def test_calls_on_other_streams_at_once():
    """Eight streams at once, through the wrappers' stream argument and as handles."""
    require_gpu()
    dtype, D, F = torch.float16, 640, 1024
    w, W1, W2, b1 = weights(D, F, dtype)
    q1, s1 = fg.quantize_s8(W1.cuda())
    q2, s2 = fg.quantize_s8(W2.cuda().t())
    args = (w.cuda(), q1, s1, b1.cuda(), q2, s2)
    xs = [torch.randn(M, D, device="cuda").to(dtype) for M in (1, 5, 17, 64, 129, 300, 2, 40)]
    rs = [torch.randn_like(x) for x in xs]
    want = [block(x, r, *args) for x, r in zip(xs, rs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [block(x, r, *args, stream=s) for x, r, s in zip(xs, rs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for k in a:
            assert torch.equal(a[k], b[k]), k
    c, s = fg.quantize_s8(xs[3], stream=streams[0].cuda_stream)
    c0, s0 = fg.quantize_s8(xs[3], stream=0)
    torch.cuda.synchronize()
    assert torch.equal(c, c0) and torch.equal(s, s0)


@gpu
def test_wrappers_take_given_outputs_and_keep_what_lies_around_them():
    require_gpu()
    X = torch.randn(9, 50, device="cuda")
    buf = torch.full((9, 64), 77, dtype=torch.int8, device="cuda")
    scales = torch.full((9,), 5.0, device="cuda")
    q, s = fg.quantize_s8(X, out=buf[:, :50], scales=scales)
    assert q.data_ptr() == buf.data_ptr() and s is scales and bool((buf[:, 50:] == 77).all())
    h = X.clone()
    q2, s2, h2 = fg.rmsnorm_s8(X, torch.ones(50, device="cuda"), residual=h, residual_out=h)
    assert h2 is h and torch.equal(h, X + X)
    q3, s3, h3 = fg.rmsnorm_s8(X, torch.ones(50, device="cuda"))
    assert h3 is X
    C = torch.full((9, 20), 3.0, device="cuda")
    same = fg.gemm_s8(q, s, q.t(), s, C=C[:, :9], beta=0.5)
    assert same.data_ptr() == C.data_ptr() and bool((C[:, 9:] == 3.0).all())
    want = (q.double() @ q.double().t()) * s.double()[:, None] * s.double()[None, :] + 1.5
    assert bool(((same.double() - want).abs() <= 6.001 * ref.U32 * (want.abs() + 3.0)).all())
    for cfg in range(fg.fp32gemm_num_configs(fg.KIND_S8GEMM)):
        C.fill_(3.0)
        assert torch.equal(fg.gemm_s8(q, s, q.t(), s, C=C[:, :9], beta=0.5, config=cfg), same)


@gpu
def test_wrappers_of_nothing():
    require_gpu()
    for M, K in ((0, 8), (3, 0), (0, 0)):
        q, s = fg.quantize_s8(torch.empty(M, K, device="cuda"))
        assert q.shape == (M, K) and s.shape == (M,) and bool((s == 0).all())
        q, s, h = fg.rmsnorm_s8(torch.empty(M, K, device="cuda"), torch.empty(K, device="cuda"))
        assert q.shape == (M, K) and bool((s == 0).all())
        C = fg.gemm_s8(q, s, torch.empty(5, K, dtype=torch.int8, device="cuda").t(),
                       torch.ones(5, device="cuda"), bias=torch.arange(5.0, device="cuda"))
        assert C.shape == (M, 5) and torch.equal(C, torch.arange(5.0, device="cuda").expand(M, 5))


@gpu
def test_wrappers_refuse():
    require_gpu()
    dev = "cuda"
    X = torch.randn(4, 32, device=dev)
    q, s = fg.quantize_s8(X)
    w = torch.ones(32, device=dev)
    with pytest.raises(TypeError):
        fg.quantize_s8(X.double())
    with pytest.raises(ValueError):
        fg.quantize_s8(X[:, ::2])
    with pytest.raises(ValueError):
        fg.quantize_s8(X[0])
    with pytest.raises(ValueError):
        fg.quantize_s8(X, out=q[:3])
    with pytest.raises(ValueError):
        fg.quantize_s8(X, scales=s[:3])
    with pytest.raises(TypeError):
        fg.quantize_s8(X, out=X)
    with pytest.raises(ValueError):
        fg.quantize_s8(X, out=q.cpu())
    with pytest.raises(ValueError):
        fg.quantize_s8(X[:1].expand(4, 32))          # rows on top of each other
    with pytest.raises(ValueError):
        fg.rmsnorm_s8(X, w[:31])
    with pytest.raises(ValueError):
        fg.rmsnorm_s8(X, w.half())
    with pytest.raises(ValueError):
        fg.rmsnorm_s8(X, w, residual=X[:3])
    with pytest.raises(TypeError):
        fg.rmsnorm_s8(X, w, residual=X.half())
    with pytest.raises(fg.Fp32GemmError):
        fg.rmsnorm_s8(X, w, eps=-1.0)
    with pytest.raises(ValueError):
        fg.gemm_s8(q, s, q, s)                       # inner dimensions
    sq = torch.zeros(4, 4, dtype=torch.int8, device=dev)
    with pytest.raises(ValueError):
        fg.gemm_s8(sq, s, sq, s)                     # a K x N weight has to be quantised to N x K
    with pytest.raises(ValueError):
        fg.gemm_s8(q, s[:3], q.t(), s)
    with pytest.raises(ValueError):
        fg.gemm_s8(q, s, q.t(), s, beta=1.0)
    with pytest.raises(ValueError):
        fg.gemm_s8(q, s, q.t(), s, bias=s.half())
    with pytest.raises(TypeError):
        fg.gemm_s8(q, s, q.t(), s, C=torch.zeros(4, 4, dtype=torch.float64, device=dev))
    with pytest.raises(TypeError):
        fg.gemm_s8(q, s, q.t(), s, C=torch.zeros(4, 4, device=dev), dtype=torch.float16)
    with pytest.raises(ValueError):
        fg.gemm_s8(q, s, q.t(), s, C=torch.zeros(4, 5, device=dev))
    with pytest.raises(fg.Fp32GemmError) as e:
        fg.gemm_s8(q, s, q.t(), s, config=99)
    assert e.value.code == fg.ERR_CONFIG
    with pytest.raises(fg.Fp32GemmError) as e:
        fg.gemm_s8(q, s, q.t(), s, act=7)
    assert e.value.code == -15


def test_wrappers_refuse_host_tensors():
    X = torch.randn(4, 32)
    with pytest.raises(ValueError):
        fg.quantize_s8(X)
    with pytest.raises(ValueError):
        fg.rmsnorm_s8(X, torch.ones(32))
    c = torch.zeros(4, 32, dtype=torch.int8)
    with pytest.raises(ValueError):
        fg.gemm_s8(c, torch.ones(4), c.t(), torch.ones(4))


@gpu
def test_gemm_keeps_the_leading_dimension_of_one_row(monkeypatch):
    """One token's codes (or a weight of one channel) come in a padded row: the call has to say so, or
    a K that is no multiple of 16 takes the loads for rows without alignment."""
    require_gpu()
    seen = []
    call = fg.fp32gemm_s8gemm_with_config

    def spy(*args):
        seen.append((args[5], args[8]))
        return call(*args)

    monkeypatch.setattr(fg, "fp32gemm_s8gemm_with_config", spy)
    g = torch.Generator().manual_seed(6)
    one, more = torch.randn(1, 1001, generator=g).cuda(), torch.randn(70, 1001, generator=g).cuda()
    (c1, s1), (c2, s2) = fg.quantize_s8(one), fg.quantize_s8(more)
    tile = fg.config_names(fg.KIND_S8GEMM).index("64x64_k1_s4")
    for a, sa, b, sb in ((c1, s1, c2, s2), (c2, s2, c1, s1), (c2[9:10], s2[9:10], c2, s2)):
        z, bound = ref.gemm(a.cpu(), sa.cpu(), b.cpu(), sb.cpu(), 0.0, None, None, False, 0)
        for cfg in (-1, tile):
            y = fg.gemm_s8(a, sa, b.t(), sb, config=cfg)
            assert seen[-1] == (1024, 1024)
            assert bool(((y.cpu().double() - z).abs() <= bound).all())
    # a row that is stored by itself, a step that is less than a row, and one past the library's limit
    for row in (c1.as_strided((1, 1001), (1001, 1)), c1.as_strided((1, 1001), (7, 1)),
                torch.zeros(1, 1, dtype=torch.int8, device="cuda").as_strided((1, 1), (1 << 21, 1))):
        w = torch.zeros(3, row.shape[1], dtype=torch.int8, device="cuda")
        fg.gemm_s8(row, s1, w.t(), torch.ones(3, device="cuda"))
        assert seen[-1][0] == row.shape[1]


@gpu
def test_wrappers_tell_autograd_what_they_overwrite():
    """A tensor that a backward pass still needs, given as an output: that pass has to refuse, as after
    any in-place operation, and not to use the new values."""
    require_gpu()
    dev = "cuda"
    w = torch.ones(32, device=dev)

    def saved():
        leaf = torch.randn(4, 32, device=dev, requires_grad=True)
        h = leaf * 2
        return h, (h * h).sum()

    h, loss = saved()
    fg.rmsnorm_s8(h, w, residual=torch.ones(4, 32, device=dev), residual_out=h)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    h, loss = saved()
    fg.rmsnorm_s8(torch.ones(4, 32, device=dev), w, residual=h, residual_out=h)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    h, loss = saved()
    q, s = fg.quantize_s8(torch.randn(4, 32, device=dev))
    fg.gemm_s8(q, s, torch.zeros(32, 32, dtype=torch.int8, device=dev).t(), torch.ones(32, device=dev), C=h, beta=1.0)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    # inputs are read only, and outputs made under no_grad or inference mode work as well
    h, loss = saved()
    fg.quantize_s8(h)
    fg.rmsnorm_s8(h, w)
    loss.backward()
    before = (q._version, s._version)
    fg.quantize_s8(torch.randn(4, 32, device=dev), out=q, scales=s)
    assert q._version > before[0] and s._version > before[1]
    before = q._version
    with pytest.raises(fg.Fp32GemmError):
        fg.rmsnorm_s8(torch.randn(4, 32, device=dev), w, eps=-1.0, out=q)
    assert q._version == before  # nothing was written
    with torch.inference_mode():
        x = torch.randn(4, 32, device=dev)
        fg.rmsnorm_s8(x, w, residual=x.clone(), residual_out=x)
        fg.gemm_s8(q, s, q.t(), s, C=torch.zeros(4, 4, device=dev))
