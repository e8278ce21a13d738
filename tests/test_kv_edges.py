"""Corners of the cache's operators: digits of the fixed-point products, bounds of a call's size, the order of
loads that a kernel's waits count on, and values at the ends."""
import os
import re
import shutil
import struct
import subprocess

import pytest
import torch

import fp32_gemm_06_amd as fg
import kv_reference as ref
from gpu_util import require_gpu
from test_kv import ATTEND, attend, cache_struct, refused

gpu = pytest.mark.gpu
TYPES = list(ref.TYPES.values())


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("D,ps", [(64, 16), (128, 64), (192, 16), (256, 24)])
def test_a_token_with_large_values_leaves_the_others_their_digits(D, ps, dtype):
    """64 tokens of weight 1, one of which has 512 times the others' scale, and codes 0 in every other column.

    There the other tokens' sums come out to half a step of the fixed-point weights for each token, which is
    512 / 8355000 / 2 of the others' scale; the fp32 operations on the way (quotient, factor, products, sum,
    division) take 16 roundings at most; the output has its own."""
    require_gpu()
    n, big, step = 64, 7, 2.0 ** -10
    g = torch.Generator().manual_seed(D)
    pages = -(-n // ps)
    k = torch.randint(-127, 128, (pages, 1, ps, D), generator=g).to(torch.int8)
    v = torch.randint(90, 128, (pages, 1, ps, D), generator=g).to(torch.int8)
    v[big // ps, 0, big % ps, ::2] = 0
    ks, vs = torch.full((pages, 1, ps), 0.01), torch.full((pages, 1, ps), step)
    vs[big // ps, 0, big % ps] = 512 * step
    table, lengths = torch.arange(pages)[None], torch.tensor([n])
    o, lse = attend(torch.zeros(1, 2, D, dtype=dtype), (k, v, ks, vs), table, lengths)
    t = torch.arange(n)
    want = (v[t // ps, 0, t % ps].double() * vs[t // ps, 0, t % ps].double()[:, None]).mean(0)
    size = (v[t // ps, 0, t % ps].double().abs().sum(0) * 512 * step / ref.TOP[3] / 2) / n
    bound = size + 16 * ref.U32 * (want + size)
    bound = bound + ref.half_step(want + bound, dtype)
    assert bool(((o[0].double() - want).abs() <= bound)[:, ::2].all()), float(((o[0].double() - want).abs() / bound)[:, ::2].max())
    assert bool(((o[0].double() - want).abs() <= bound).all())


@gpu
@pytest.mark.parametrize("at", [40000.3125, 39999.6875, 40000.4375, 300000.3125, 3000000.25])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_query_values_are_rounded_to_the_nearest_step(at, sign):
    """A query whose largest value is 8355000 steps of 2^-22, by which the others come out as fractions of a step.

    The largest meets codes 0, so the score is the others' sum: off by half a step each, and 16 roundings of the
    fp32 operations behind it.  One token's log-sum-exp is its score."""
    require_gpu()
    D, step = 64, 2.0 ** -22
    q = torch.full((1, 1, D), sign * at * step)
    q[0, 0, 0] = ref.TOP[3] * step
    k = torch.full((1, 1, 16, D), 127, dtype=torch.int8)
    k[..., 0] = 0
    v, s = torch.zeros_like(k), torch.ones(1, 1, 16)
    _, lse = attend(q, (k, v, s, s), torch.zeros(1, 1), torch.tensor([1]), scale=1.0)
    want = sign * at * step * 127 * (D - 1)
    assert abs(float(lse) - want) <= 127 * (D - 1) * step / 2 + 16 * ref.U32 * abs(want)


def attention_loads(tmp):
    """{kernel: [order of the tile's loads between two branches]} of the built library's attention kernels: K for a
    load of keys into LDS, V for one of values, which are those past the caches."""
    objdump = shutil.which("llvm-objdump", path=os.pathsep.join(["/opt/rocm/llvm/bin", os.environ.get("PATH", "")]))
    path = os.path.join(os.path.dirname(fg.__file__), "libfp32gemm.so")
    if objdump is None or not os.path.exists(path):
        pytest.skip("no llvm-objdump, or the library is not built")
    with open(path, "rb") as f:
        data = f.read()
    found = {}
    for m in re.finditer(b"__CLANG_OFFLOAD_BUNDLE__", data):
        at = m.start() + 24
        count, = struct.unpack_from("<Q", data, at)
        at += 8
        for _ in range(count):
            offset, size, name = struct.unpack_from("<QQQ", data, at)
            image = data[m.start() + offset:m.start() + offset + size]
            at += 24 + name
            if b"attend_kernel" not in image:
                continue
            (tmp / "image").write_bytes(image)
            text = subprocess.run([objdump, "-d", "--no-show-raw-insn", str(tmp / "image")], capture_output=True, text=True,
                                  check=True).stdout
            for kernel, body in re.findall(r"<(\w*attend_kernel\w*)>:\n(.*?)(?=\n\n|\Z)", text, re.S):
                runs = [""]
                for line in body.splitlines():
                    op = line.split("//")[0].split()
                    if not op:
                        continue
                    if re.match(r"s_(cbranch|branch|endpgm|setpc)", op[0]):
                        runs.append("")
                    elif "_load_lds_" in op[0] or "_load_" in op[0] and "lds" in op:
                        runs[-1] += "K"
                    elif op[0].startswith("global_load") and "nt" in op:
                        runs[-1] += "V"
                found[kernel] = [r for r in runs if r]
    return found


def test_a_tile_s_keys_are_asked_for_before_its_values(tmp_path):
    """The wait for a tile's keys lets as many loads be on the way as its values have, so all of those have to be
    asked for behind all of these, in every kernel and wherever a tile is asked for."""
    found = attention_loads(tmp_path)
    assert len(found) == 84
    for kernel, runs in found.items():
        assert any("K" in r for r in runs) and any("V" in r for r in runs), kernel
        assert all(re.fullmatch("K*V*", r) for r in runs), (kernel, runs)
        values = {r.count("V") for r in runs if "V" in r}
        assert len(values) == 1, (kernel, runs)


@pytest.mark.parametrize("type,step,heads,Hq,B", [(fg.TYPE_F32, 64, 4, 4, 32), (fg.TYPE_F32, 64, 1, 2, 128),
                                                  (fg.TYPE_BF16, 128, 1, 17, 200), (fg.TYPE_S8, 256, 8, 8, 90)])
def test_a_call_whose_runs_pass_32_bits_is_refused(type, step, heads, Hq, B):
    """The count of all units is rounded up to whole runs in 32 bits, which leaves it 2^31 - 1024.  The longest
    table below that is taken, which the next argument's refusal shows; one more page is not."""
    groups = -(-Hq // heads // 16)
    steps = (2 ** 31 - 1024 - 1) // (B * heads * groups) - 3        # of a table, the most
    pages = steps * step // 64                                      # of 64 tokens
    assert (pages + step // 64) * 64 <= 2 ** 30
    c = cache_struct(type=type, heads=heads, page_size=64)
    floats = type if type != fg.TYPE_S8 else fg.TYPE_F32
    kw = dict(type=floats, Hq=Hq, ldq=4096, ldo=4096, B=B, cache=c, lengths=0)
    for ldt, code in ((pages, -9), (pages + step // 64, -8)):
        refused(fg.kv_attention, ATTEND, dict(kw, ldt=ldt), code)


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("style", ["halves", "pairs"])
def test_an_infinity_under_the_norm_leaves_zeros_beside_it(style, dtype):
    """x / sqrt(mean x^2 + eps) of a row with an infinity is NaN there and 0 elsewhere; a rotation spreads the NaN to
    the other value of its pair.  A row with a NaN is NaN throughout."""
    require_gpu()
    D, R = 80, 32
    x = torch.randn(3, 4, D, generator=torch.Generator().manual_seed(2)).to(dtype)
    x[0, 1, 6], x[1, 2, 70], x[2, 0, 50] = float("inf"), float("-inf"), float("nan")
    pos, freq = torch.arange(3).int(), 10000.0 ** (-torch.arange(R // 2, dtype=torch.float64) / 16)
    w = torch.full((D,), 1.5, dtype=dtype)
    y, _ = fg.norm_rope(x.cuda(), None, pos.cuda(), freq.cuda(), w.cuda(), style=style)
    want = torch.zeros(3, 4, D, dtype=torch.bool)
    want[0, 1, [6, 7 if style == "pairs" else 22]] = True
    want[1, 2, 70] = want[2, 0] = True
    y = y.cpu()
    assert torch.equal(torch.isnan(y), want)
    assert bool((y[0, 1] == 0)[~want[0, 1]].all()) and bool((y[1, 2] == 0)[~want[1, 2]].all())
    clean, bound, _ = ref.norm_rope(x, w, 1e-6, pos, freq, style == "pairs")
    rows = torch.isfinite(x).all(-1)
    assert bool(((y.double() - clean).abs() <= bound)[rows].all())


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("D,R,style", [(128, 128, "halves"), (128, 64, "halves"), (64, 64, "pairs"), (256, 64, "halves"),
                                       (80, 20, "halves")])
def test_a_large_prompt_into_a_float_cache_is_that_of_small_calls(D, R, style, dtype):
    """From 32 and from 75 MB of outputs on, rows take one or another way to memory, by their layout; a token's
    queries, and its rows of the cache, do not depend on it."""
    require_gpu()
    for mb in (40, 88):
        Hq, Hk = 2048 // D, 512 // D or 1
        T = int(mb * 2 ** 20 / ((Hq + 2 * Hk) * D * dtype.itemsize))
        g = torch.Generator(device="cuda").manual_seed(R)
        x = torch.randn(T, Hq + 2 * Hk, D, generator=g, device="cuda").to(dtype)
        q, k, v = x.split([Hq, Hk, Hk], 1)
        w = torch.randn(D, generator=g, device="cuda").to(dtype)
        freq = torch.rand(R // 2, generator=g, device="cuda", dtype=torch.float64)
        pos = torch.arange(T, device="cuda", dtype=torch.int32)
        slots = torch.randperm(T + 100, generator=g, device="cuda")[:T].int()
        a, b = (fg.KVCache.empty(-(-(T + 100) // 16), 16, Hk, D, dtype) for _ in range(2))
        y = fg.rope_write(a, q, k, v, slots, pos, freq, w, w, style=style)
        for t0 in range(0, T, 2500):
            s = slice(t0, t0 + 2500)
            z = fg.rope_write(b, q[s], k[s], v[s], slots[s], pos[s], freq, w, w, style=style)
            assert torch.equal(y[s], z)
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


@gpu
def test_a_window_of_any_size():
    """A window longer than the sequence, also one past 32 bits, is no window; others that are none are refused."""
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(3)
    cache = fg.KVCache(*(torch.randn(4, 2, 16, 32, generator=g, device="cuda") for _ in range(2)))
    q = torch.randn(1, 4, 32, generator=g, device="cuda")
    table, n = torch.arange(4, device="cuda").int()[None].contiguous(), torch.tensor([50], device="cuda").int()
    want = fg.attention(q, cache, table, n)
    for window in (50, 64, 50.0, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 63, 10 ** 30):
        assert torch.equal(fg.attention(q, cache, table, n, window=window), want)
    assert not torch.equal(fg.attention(q, cache, table, n, window=5), want)
    for window in (-1, -2 ** 31, -2 ** 32 + 5, -10 ** 30):
        with pytest.raises(fg.Fp32GemmError):
            fg.attention(q, cache, table, n, window=window)
    with pytest.raises(ValueError):
        fg.attention(q, cache, table, n, window=4.5)


@gpu
def test_strides_and_tables_past_32_bits_are_refused():
    """Not taken for what their low 32 bits say."""
    require_gpu()
    dev = "cuda"
    far = torch.empty(2 ** 32 + 256, dtype=torch.float16, device=dev).as_strided((2, 1, 64), (2 ** 32 + 64, 64, 1))
    far.zero_()
    near = torch.zeros(2, 1, 64, dtype=torch.float16, device=dev)
    slots = torch.arange(2, dtype=torch.int32, device=dev)
    cache = fg.KVCache.empty(2, 16, 1, 64, torch.float16)
    table, n = torch.zeros(2, 2, dtype=torch.int32, device=dev), torch.ones(2, dtype=torch.int32, device=dev)
    calls = [lambda x: fg.norm_rope(x, None), lambda x: fg.norm_rope(near, x), lambda x: fg.norm_rope(near, None, out_q=x),
             lambda x: fg.cache_write(cache, x, near, slots), lambda x: fg.cache_write(cache, near, x, slots),
             lambda x: fg.rope_write(cache, x, near, near, slots), lambda x: fg.cache_read(cache, slots, out_k=x),
             lambda x: fg.attention(x, cache, table, n), lambda x: fg.attention(near, cache, table, n, out=x)]
    for call in calls:
        call(near)
        with pytest.raises(fg.Fp32GemmError):
            call(far)
    for call in (calls[0], calls[3], calls[7]):    # whose number of tokens is this operand's
        with pytest.raises(ValueError, match="2\\^31 tokens"):
            call(near[:1].expand(2 ** 32 + 2, 1, 64))
    del far
    wide = torch.empty(1, 2 ** 32 + 2, dtype=torch.int32, device=dev)
    wide[:, :2] = 0
    fg.attention(near[:1], cache, wide[:, :2].contiguous(), n[:1])
    with pytest.raises(fg.Fp32GemmError):
        fg.attention(near[:1], cache, wide, n[:1])
