"""The cache's operators together, as a decoder's attention block uses them, through the torch wrappers: a
prompt's chunk and decode steps; under graph capture, on other streams, and with calls the wrappers refuse."""
import pytest
import torch

import fp32_gemm_06_amd as fg
import kv_reference as ref
import s8_reference
from gpu_util import require_gpu

gpu = pytest.mark.gpu
FREQ = 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)


class Block:
    """h + Wo attend(rope(norm(Wqkv rmsnorm(h)))), all projections in 8 bits."""

    def __init__(self, D, Hq, Hk, dim, dtype, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.Hq, self.Hk, self.dim, self.dtype = Hq, Hk, dim, dtype
        rows = (Hq + 2 * Hk) * dim
        self.norm = (1 + 0.1 * torch.randn(D, generator=g)).to(dtype).cuda()
        self.wq, self.wk = ((1 + 0.1 * torch.randn(dim, generator=g)).to(dtype).cuda() for _ in range(2))
        self.qkv = fg.quantize_s8((torch.randn(rows, D, generator=g) * D ** -0.5).cuda())
        self.out = fg.quantize_s8((torch.randn(D, Hq * dim, generator=g) * (Hq * dim) ** -0.5).cuda())
        self.freq = FREQ[:dim // 2].cuda()

    def project(self, h):
        c, s, _ = fg.rmsnorm_s8(h, self.norm)
        x = fg.gemm_s8(c, s, self.qkv[0].t(), self.qkv[1], dtype=self.dtype).view(h.shape[0], -1, self.dim)
        return x.split([self.Hq, self.Hk, self.Hk], 1)

    def step(self, h, cache, slots, positions, table, lengths, workspace=None, window=0, stream=None):
        """One new token of each sequence."""
        q, k, v = self.project(h)
        q = fg.rope_write(cache, q, k, v, slots, positions, self.freq, self.wq, self.wk)
        o = fg.attention(q, cache, table, lengths, window=window, workspace=workspace)
        c, s = fg.quantize_s8(o.view(h.shape[0], -1))
        y = h.clone()
        fg.gemm_s8(c, s, self.out[0].t(), self.out[1], C=y, beta=1.0)
        return dict(q=q, o=o, y=y)


def setup(lengths, ps, spare=3, room=8, seed=0):
    """(table, pages) with room for `room` more tokens each."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-(n + room) // ps) for n in lengths]
    perm = torch.randperm(sum(need) + spare, generator=g)
    table, at = torch.full((len(lengths), max(need)), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n].int()
        at += n
    return table, sum(need) + spare


def slots_of(table, ps, b, t):
    t = torch.as_tensor(t)
    return (table[b].long()[t // ps] * ps + t % ps).int()


@gpu
@pytest.mark.parametrize("dtype,kind", [(d, k) for d in ref.TYPES.values() for k in (torch.int8, d)], ids=str)
@pytest.mark.parametrize("Hq,Hk,dim,ps,window", [(8, 2, 64, 16, 0), (3, 3, 48, 10, 40)])
def test_prompt_and_steps(Hq, Hk, dim, ps, window, dtype, kind):
    """Prompts written in one call, then decode steps; each step's attention against the 64-bit reference on
    what the cache holds, and the cache against the reference's rows of the projections."""
    require_gpu()
    lengths = [1, 37, 150]
    table, pages = setup(lengths, ps)
    cache = fg.KVCache.empty(pages, ps, Hk, dim, kind)
    block = Block(256, Hq, Hk, dim, dtype)
    g = torch.Generator().manual_seed(1)
    dtable = table.cuda()
    for b, n in enumerate(lengths):
        h = torch.randn(n, 256, generator=g).to(dtype).cuda()
        q, k, v = block.project(h)
        t = torch.arange(n)
        fg.rope_write(cache, q, k, v, slots_of(table, ps, b, t).cuda(), t.int().cuda(), block.freq, block.wq, block.wk)
        kr, vr = fg.cache_read(cache, slots_of(table, ps, b, t).cuda(), dtype=dtype)
        want, bound, exact = ref.norm_rope(k.cpu(), block.wk.cpu(), 1e-6, t, FREQ[:dim // 2], False)
        if kind == torch.int8:
            # half a step of the code, and the reading's two roundings
            step = (want.abs().amax(-1, keepdim=True) / 127) * 1.001
            bound = 0.5001 * step + exact + ref.half_step(want.abs() + step, dtype) + 2 * ref.U32 * (want.abs() + step)
        assert bool(((kr.cpu().double() - want).abs() <= bound).all())
        if kind != torch.int8:
            assert torch.equal(vr, v)
    ws = fg.attention_workspace(cache, Hq)
    for step in range(3):
        n = torch.tensor(lengths) + step
        slots = torch.stack([slots_of(table, ps, b, int(n[b])) for b in range(3)])
        h = torch.randn(3, 256, generator=g).to(dtype).cuda()
        o = block.step(h, cache, slots.cuda(), n.int().cuda(), dtable, (n + 1).int().cuda(),
                       ws if step else None, window)
        kv = [None if t is None else t.cpu() for t in cache._tensors()]
        wo, _, bo, _ = ref.attention(o["q"].cpu(), *kv, table, n + 1, window, dim ** -0.5)
        assert bool(((o["o"].cpu().double() - wo).abs() <= bo).all())
        assert bool(torch.isfinite(o["y"]).all())


@gpu
def test_steps_captured_in_two_graphs_follow_the_lengths():
    """Two graphs with workspaces of their own, replayed in turn and together with eager calls, while the
    lengths, the positions and the table that they read change; every replay equals the eager result."""
    require_gpu()
    dtype, Hq, Hk, dim, ps = torch.bfloat16, 8, 2, 64, 16
    block = Block(256, Hq, Hk, dim, dtype)
    made = []
    for seed, lengths in ((0, [5, 700, 40]), (1, [64])):
        table, pages = setup(lengths, ps, seed=seed)
        caches = [fg.KVCache.empty(pages, ps, Hk, dim) for _ in range(2)]
        for t in zip(*(c._tensors() for c in caches)):
            x = torch.randint(-127, 128, t[0].shape, device="cuda") if t[0].dtype == torch.int8 else torch.rand_like(t[0])
            for y in t:
                y.copy_(x)
        B = len(lengths)
        st = dict(h=torch.randn(B, 256, device="cuda").to(dtype), slots=torch.full((B,), -1, dtype=torch.int32, device="cuda"),  # the call before writes none
                  positions=torch.zeros(B, dtype=torch.int32, device="cuda"), table=table.cuda(),
                  lengths=torch.ones(B, dtype=torch.int32, device="cuda"))
        ws = [fg.attention_workspace(c, Hq) for c in caches]

        def args(i, st=st, caches=caches, ws=ws):
            return dict(st, cache=caches[i], workspace=ws[i])

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            block.step(**args(0))
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = block.step(**args(0))
        made.append((lengths, table, st, caches, args, graph, out))
    other = torch.cuda.Stream()
    for turn in range(5):
        for lengths, table, st, caches, args, graph, out in made:
            n = torch.tensor(lengths) + turn
            st["h"].normal_()
            st["positions"].copy_(n.int())
            st["lengths"].copy_((n + 1).int())
            st["slots"].copy_(torch.stack([slots_of(table, ps, b, int(n[b])) for b in range(len(lengths))]))
        torch.cuda.synchronize()
        made[0][5].replay()
        with torch.cuda.stream(other):
            made[1][5].replay()
        want = [block.step(**m[4](1)) for m in made]
        torch.cuda.synchronize()
        for m, w in zip(made, want):
            for k in w:
                assert torch.equal(m[6][k], w[k]), (turn, k)
            for x, y in zip(*(c._tensors() for c in m[3])):
                assert torch.equal(x, y)


@gpu
def test_workspace_of_a_capture_without_one():
    """A captured call that makes its own workspace clears it in the graph: replays stay right."""
    require_gpu()
    kv = [torch.randn(40, 1, 16, 64, device="cuda") for _ in range(2)]
    cache = fg.KVCache(*kv)
    table = torch.arange(40, dtype=torch.int32, device="cuda")[None]
    lengths = torch.tensor([640], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 2, 64, device="cuda")
    want = fg.attention(q, cache, table, lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fg.attention(q, cache, table, lengths)
    for _ in range(4):
        got.zero_()
        torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@gpu
def test_calls_on_other_streams_at_once():
    require_gpu()
    dtype, Hq, Hk, dim, ps = torch.float16, 6, 3, 64, 32
    g = torch.Generator().manual_seed(2)
    cache = fg.KVCache(*((torch.randn(64, Hk, ps, dim, generator=g)).to(dtype).cuda() for _ in range(2)))
    qs = [torch.randn(B, Hq, dim, generator=g).to(dtype).cuda() for B in (1, 3, 7, 2, 30, 1, 5, 9)]
    tables = [torch.randint(0, 64, (len(q), 40), generator=g).int().cuda() for q in qs]
    lengths = [torch.randint(0, 1281, (len(q),), generator=g).int().cuda() for q in qs]
    want = [fg.attention(*a) for a in zip(qs, [cache] * 8, tables, lengths)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    spaces = [fg.attention_workspace(cache, Hq) for _ in qs]
    torch.cuda.synchronize()
    for turn in range(3):
        got = [fg.attention(q, cache, t, n, workspace=w, stream=s)
               for q, t, n, w, s in zip(qs, tables, lengths, spaces, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
    slots = torch.arange(9, dtype=torch.int32, device="cuda")
    x = torch.randn(9, Hk, dim, device="cuda").to(dtype)
    torch.cuda.synchronize()
    fg.cache_write(cache, x, x, slots, stream=streams[0])
    k, v = fg.cache_read(cache, slots, stream=streams[0].cuda_stream)
    y, _ = fg.norm_rope(x, None, slots, FREQ.cuda(), stream=0)
    torch.cuda.synchronize()
    assert torch.equal(k, x) and torch.equal(v, x)
    assert torch.equal(y, fg.norm_rope(x, None, slots, FREQ.cuda())[0])


@gpu
def test_wrappers_take_given_outputs():
    require_gpu()
    x = torch.randn(5, 6, 32, device="cuda")
    q, k, v = x.split([4, 1, 1], 1)
    pos, freq = torch.arange(5, dtype=torch.int32, device="cuda"), FREQ[:16].cuda()
    yq, yk = fg.norm_rope(q, k, pos, freq)
    big = torch.full((5, 9, 32), 3.0, device="cuda")
    a, b = fg.norm_rope(q, k, pos, freq, out_q=big[:, :4], out_k=big[:, 5:6])
    assert torch.equal(a, yq) and torch.equal(b, yk) and a.data_ptr() == big.data_ptr()
    assert bool((big[:, 4] == 3).all()) and bool((big[:, 6:] == 3).all())
    c = x.clone()
    fg.norm_rope(c[:, :4], c[:, 4:5], pos, freq, out_q=c[:, :4], out_k=c[:, 4:5])   # in place
    assert torch.equal(c[:, :4], yq) and torch.equal(c[:, 4:5], yk) and torch.equal(c[:, 5:], v)
    cache = fg.KVCache.empty(2, 8, 1, 32, torch.float32)
    slots = torch.tensor([3, -1, 12, 99, 0], dtype=torch.int32, device="cuda")
    out = torch.empty(5, 4, 32, device="cuda")
    assert fg.rope_write(cache, q, k, v, slots, pos, freq, out_q=out) is out and torch.equal(out, yq)
    kr, vr = (torch.full((5, 1, 32), 9.0, device="cuda") for _ in range(2))
    k2, v2 = fg.cache_read(cache, slots, out_k=kr, out_v=vr)
    live = [0, 2, 4]
    assert k2 is kr and torch.equal(kr[live], yk[live]) and torch.equal(vr[live], v[live])
    assert bool((kr[[1, 3]] == 9).all())
    k3, _ = fg.cache_read(cache, slots)
    assert torch.equal(k3[live], yk[live]) and bool((k3[[1, 3]] == 0).all())
    table, n = torch.zeros(5, 1, dtype=torch.int32, device="cuda"), torch.full((5,), 4, dtype=torch.int32, device="cuda")
    o, lse = torch.empty(5, 4, 32, device="cuda"), torch.empty(5, 4, device="cuda")
    assert fg.attention(yq, cache, table, n, out=o, lse=lse) is o
    assert torch.equal(o, fg.attention(yq, cache, table, n)) and bool(torch.isfinite(lse).all())
    # nothing
    e = fg.attention(yq[:0], cache, table[:0], n[:0])
    assert e.shape == (0, 4, 32)
    fg.cache_write(cache, k[:0], v[:0], slots[:0])
    assert fg.cache_read(cache, slots[:0])[0].shape == (0, 1, 32)
    assert fg.norm_rope(q[:0], k[:0], pos[:0], freq)[0].shape == (0, 4, 32)


@gpu
def test_wrappers_refuse():
    require_gpu()
    dev = "cuda"
    x = torch.randn(4, 3, 32, device=dev)
    pos, freq, w = torch.arange(4, dtype=torch.int32, device=dev), FREQ[:16].cuda(), torch.ones(32, device=dev)
    slots = pos.clone()
    cache = fg.KVCache.empty(2, 16, 3, 32)
    table, n = torch.zeros(4, 2, dtype=torch.int32, device=dev), torch.ones(4, dtype=torch.int32, device=dev)
    bad = [
        (TypeError, lambda: fg.norm_rope(x.double(), None)),
        (ValueError, lambda: fg.norm_rope(None, None)),
        (ValueError, lambda: fg.norm_rope(x[0], None)),
        (ValueError, lambda: fg.norm_rope(x.transpose(0, 1), None)),
        (ValueError, lambda: fg.norm_rope(x[:, ::2], None)),
        (ValueError, lambda: fg.norm_rope(x[:1].expand(4, 3, 32), None)),
        (ValueError, lambda: fg.norm_rope(x, x[:3])),
        (TypeError, lambda: fg.norm_rope(x, x.half())),
        (ValueError, lambda: fg.norm_rope(x, None, pos)),
        (ValueError, lambda: fg.norm_rope(x, None, None, freq)),
        (ValueError, lambda: fg.norm_rope(x, None, pos.long(), freq)),
        (ValueError, lambda: fg.norm_rope(x, None, pos, freq.float())),
        (ValueError, lambda: fg.norm_rope(x, None, pos, FREQ[:17].cuda())),
        (ValueError, lambda: fg.norm_rope(x, None, pos, freq, style="other")),
        (ValueError, lambda: fg.norm_rope(x, None, q_weight=w[:31])),
        (ValueError, lambda: fg.norm_rope(x, None, k_weight=w)),
        (ValueError, lambda: fg.norm_rope(x, None, out_q=x[:3])),
        (fg.Fp32GemmError, lambda: fg.norm_rope(x, None, eps=-1.0)),
        (fg.Fp32GemmError, lambda: fg.norm_rope(torch.randn(4, 3, 24, device=dev), None)),
        (ValueError, lambda: fg.cache_write(cache, x[:, :2], x, slots)),
        (ValueError, lambda: fg.cache_write(cache, x, x, slots[:3])),
        (ValueError, lambda: fg.cache_write(cache, x, x, slots.long())),
        (TypeError, lambda: fg.cache_write(cache, x, x.half(), slots)),
        (TypeError, lambda: fg.cache_write(fg.KVCache.empty(2, 16, 3, 32, torch.half), x, x, slots)),
        (ValueError, lambda: fg.rope_write(cache, x[:3], x, x, slots)),
        (ValueError, lambda: fg.rope_write(cache, x, x, x, slots, q_weight=w.half())),
        (ValueError, lambda: fg.cache_read(cache, slots, out_k=x[:3])),
        (TypeError, lambda: fg.cache_read(fg.KVCache.empty(2, 16, 3, 32, torch.half), slots, dtype=torch.float32)),
        (ValueError, lambda: fg.attention(x[0], cache, table, n)),
        (ValueError, lambda: fg.attention(x, cache, table[:3], n)),
        (ValueError, lambda: fg.attention(x, cache, table.long(), n)),
        (ValueError, lambda: fg.attention(x, cache, table.t().contiguous().t(), n)),
        (ValueError, lambda: fg.attention(x, cache, table, n[:3])),
        (ValueError, lambda: fg.attention(x, cache, table, n, out=x[:3])),
        (ValueError, lambda: fg.attention(x, cache, table, n, lse=w)),
        (ValueError, lambda: fg.attention(x, cache, table, n, workspace=w)),
        (fg.Fp32GemmError, lambda: fg.attention(x, cache, table, n, window=-1)),
        (fg.Fp32GemmError, lambda: fg.attention(x, cache, table, n, scale=float("nan"))),
        (fg.Fp32GemmError, lambda: fg.attention(x, cache, table, n, workspace=torch.zeros(64, dtype=torch.uint8, device=dev))),
        (ValueError, lambda: fg.attention(x[:, :2], cache, table, n)),
        (TypeError, lambda: fg.KVCache(x.double(), x.double())),
        (ValueError, lambda: fg.KVCache(x, x)),
        (ValueError, lambda: fg.KVCache(cache.k, cache.v)),
        (ValueError, lambda: fg.KVCache(cache.k, cache.v, cache.k_scale, cache.v_scale[:, :, :8])),
        (ValueError, lambda: fg.KVCache(cache.k[:, :, ::2], cache.v[:, :, ::2], cache.k_scale, cache.v_scale)),
        (ValueError, lambda: fg.KVCache(cache.k.cpu(), cache.v.cpu(), cache.k_scale.cpu(), cache.v_scale.cpu())),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            print(i)
    torch.cuda.synchronize()


@gpu
def test_wrappers_tell_autograd_what_they_overwrite():
    require_gpu()
    leaf = torch.randn(4, 2, 32, device="cuda", requires_grad=True)
    h = leaf * 2
    loss = (h * h).sum()
    fg.norm_rope(h, None, q_weight=torch.ones(32, device="cuda"), out_q=h)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    cache = fg.KVCache.empty(1, 16, 2, 32, torch.float32)
    before = cache.k._version
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    fg.cache_write(cache, leaf, leaf, slots)
    assert cache.k._version > before
    with torch.inference_mode():
        c = fg.KVCache.empty(1, 16, 2, 32)
        fg.cache_write(c, leaf, leaf, slots)
        fg.cache_read(c, slots)


def test_wrappers_refuse_host_tensors():
    x = torch.randn(4, 2, 32)
    with pytest.raises(ValueError):
        fg.norm_rope(x, None)
    with pytest.raises(ValueError):
        fg.KVCache(torch.zeros(1, 2, 16, 32), torch.zeros(1, 2, 16, 32))
