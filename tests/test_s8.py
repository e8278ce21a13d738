"""The 8-bit linear layer (s8_quantize, s8_rmsnorm, s8gemm) against 64-bit references.

Codes, the stored residual sum and quantize's scales have to be equal to the
reference's; a norm's scale is off by one rounding to fp32; a product by the
fp32 roundings of its epilogue and the rounding to C's type, counted in
s8_reference.gemm.
"""
import os

import numpy as np
import pytest
import torch

import fp32_gemm_06_amd as fg
import s8_reference as ref
from gpu_util import require_gpu

gpu = pytest.mark.gpu
CONFIGS = fg.config_names(fg.KIND_S8GEMM)

# every configuration's tile edges, one less and one more, and sizes of one
EDGES = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 257]


def device(t, ld=None, offset=0, fill=None):
    """A GPU copy of a 2-D host tensor with leading dimension ld, its first element `offset`
    elements past an allocation's start; what lies around it holds `fill`."""
    r, c = t.shape
    ld = ld or max(1, c)
    if fill is None:
        fill = 77 if t.dtype == torch.int8 else float("nan")
    flat = torch.full((offset + max(1, r) * ld + 64,), fill, dtype=t.dtype, device="cuda")
    v = flat[offset: offset + max(1, r) * ld].view(max(1, r), ld)[:r, :c]
    v.copy_(t)
    return v, flat


def untouched(flat, view_shape, ld, offset, fill):
    """Whether everything in `flat` but the view's elements still holds `fill`."""
    r, c = view_shape
    mask = torch.ones_like(flat, dtype=torch.bool)
    if r and c:
        mask[offset: offset + r * ld].view(r, ld)[:, :c] = False
    rest = flat[mask]
    if isinstance(fill, float) and fill != fill:
        return bool(torch.isnan(rest).all())
    return bool((rest == fill).all())


def make_codes(g, rows, cols):
    return torch.randint(-128, 128, (rows, cols), generator=g, dtype=torch.int16).to(torch.int8)


def run_gemm(M, N, K, type=0, cfg=-1, beta=0.0, bias=False, relu=False, lda=None, ldb=None, ldc=None,
             offa=0, offb=0, offc=0, seed=0):
    g = torch.Generator().manual_seed(1000 * seed + M * 31 + N * 7 + K)
    A, B = make_codes(g, M, K), make_codes(g, N, K)
    sA = torch.rand(M, generator=g) * 0.1 + 1e-3
    sB = torch.rand(N, generator=g) * 0.01 + 1e-4
    C0 = torch.randn(M, N, generator=g).to(ref.TYPES[type])
    bv = torch.randn(N, generator=g) if bias else None
    pad = lambda k: -(-k // 16) * 16
    lda, ldb, ldc = lda or pad(K), ldb or pad(K), ldc or N
    dA, _ = device(A, lda, offa)
    dB, _ = device(B, ldb, offb)
    # beta = 0 must not read C: NaN in it
    dC, flat = device(C0 if beta else torch.full_like(C0, float("nan")), ldc, offc)
    dbias = bv.cuda() if bias else None
    rc = fg.fp32gemm_s8gemm_with_config(cfg, M, N, K, dA, lda, sA.cuda(), dB, ldb, sB.cuda(), beta,
                                        type, dC, ldc, dbias, fg.ACT_RELU if relu else fg.ACT_NONE)
    assert rc == 0, fg.strerror(rc)
    torch.cuda.synchronize()
    z, bound = ref.gemm(A, sA, B, sB, beta, C0, bv, relu, type)
    err = (dC.cpu().double() - z).abs()
    worst = float((err / bound).max())
    assert worst <= 1.0, f"{(M, N, K, type, cfg)}: {worst:.3g} times the bound"
    assert untouched(flat, (M, N), ldc, offc, float("nan"))
    return dC


# ---- refusals, on the CPU -----------------------------------------------------

GEMM = dict(M=4, N=4, K=4, A=16, lda=4, sA=16, B=16, ldb=4, sB=16, beta=0.0, type=0, C=16, ldc=4,
            bias=None, act=0)


def call_gemm(cfg=None, **kw):
    a = dict(GEMM, **kw)
    args = (a["M"], a["N"], a["K"], a["A"], a["lda"], a["sA"], a["B"], a["ldb"], a["sB"], a["beta"],
            a["type"], a["C"], a["ldc"], a["bias"], a["act"], 0)
    return fg.s8gemm(*args) if cfg is None else fg.fp32gemm_s8gemm_with_config(cfg, *args)


@pytest.mark.parametrize("kw,pos", [
    (dict(M=-1), 1), (dict(N=-1), 2), (dict(K=-1), 3), (dict(K=131072, lda=131072, ldb=131072), 3),
    (dict(A=None), 4), (dict(lda=3), 5), (dict(lda=(1 << 20) + 1), 5), (dict(sA=None), 6),
    (dict(sA=18), 6), (dict(B=None), 7), (dict(ldb=3), 8), (dict(ldb=(1 << 20) + 1), 8),
    (dict(sB=None), 9), (dict(sB=17), 9), (dict(type=3), 11), (dict(type=-1), 11),
    (dict(C=None), 12), (dict(C=18), 12), (dict(type=2, C=17), 12), (dict(ldc=3), 13),
    (dict(ldc=(1 << 20) + 1), 13), (dict(bias=18), 14), (dict(act=2), 15), (dict(act=-1), 15),
])
def test_gemm_argument_checks_need_no_gpu(kw, pos):
    assert call_gemm(**kw) == -pos
    assert call_gemm(cfg=0, **kw) == -pos - 1
    assert fg.strerror(-pos) == f"invalid argument {pos}"


def test_gemm_quick_returns_need_no_gpu():
    assert call_gemm(M=0, A=None, B=None, C=None, sA=None, sB=None) == 0
    assert call_gemm(N=0, A=None, B=None, C=None, sA=None, sB=None) == 0
    # an empty sum added to C itself
    assert call_gemm(K=0, A=None, B=None, sA=None, sB=None, beta=1.0) == 0
    assert call_gemm(cfg=len(CONFIGS)) == fg.ERR_CONFIG
    assert call_gemm(cfg=-2) == fg.ERR_CONFIG


def test_gemm_configurations_and_their_choice():
    assert len(CONFIGS) == fg.fp32gemm_num_configs(fg.KIND_S8GEMM) == len(set(CONFIGS))
    assert fg.fp32gemm_config_name(fg.KIND_S8GEMM, len(CONFIGS)) is None
    assert fg.fp32gemm_config_name(fg.KIND_S8GEMM, -1) is None
    assert fg.fp32gemm_config_max_rows(fg.KIND_S8GEMM, 0) == 2 ** 31 - 1
    assert fg.fp32gemm_config_max_rows(fg.KIND_S8GEMM, len(CONFIGS)) == -1
    name = lambda *s: CONFIGS[fg.fp32gemm_select_config(fg.KIND_S8GEMM, *s)]
    big = 2 ** 31 - 1
    for shape in [(1, 1, 1), (big, 1, 1), (big, 1 << 20, 131071), (1, 1 << 20, 131071), (0, 0, 0)]:
        assert name(*shape) in CONFIGS
    # dot products for a token, never above eight; tiles that grow with the shape
    assert name(1, 4096, 4096).startswith("gemv") and name(1, 512, 11008).startswith("gemv")
    assert not any(name(9, N, K).startswith("gemv") for N in (1, 64, 4096, 1 << 20) for K in (1, 4096, 131071))
    assert name(16, 11008, 4096).startswith("16x16") and name(4096, 4096, 4096).startswith("256x256")


@pytest.mark.parametrize("kw,pos", [
    (dict(trans=2), 1), (dict(M=-1), 2), (dict(K=-1), 3), (dict(type=3), 4), (dict(X=None), 5),
    (dict(X=18), 5), (dict(type=1, X=17), 5), (dict(ldx=7), 6), (dict(trans=1, ldx=3), 6),
    (dict(ldx=(1 << 20) + 1), 6), (dict(Q=None), 7), (dict(ldq=7), 8), (dict(trans=1, ldx=4, ldq=7), 8),
    (dict(ldq=(1 << 20) + 1), 8), (dict(scales=None), 9), (dict(scales=18), 9),
])
def test_quantize_argument_checks_need_no_gpu(kw, pos):
    a = dict(trans=0, M=4, K=8, type=0, X=16, ldx=8, Q=16, ldq=8, scales=16)
    a.update(kw)
    assert fg.s8_quantize(*a.values(), 0) == -pos


@pytest.mark.parametrize("kw,pos", [
    (dict(M=-1), 1), (dict(K=-1), 2), (dict(type=3), 3), (dict(X=None), 4), (dict(X=18), 4),
    (dict(ldx=7), 5), (dict(R=18), 6), (dict(ldr=7), 7), (dict(H=18), 8), (dict(ldh=7), 9),
    (dict(H=16, ldx=12), 9), (dict(R=64, H=64, ldr=12), 9), (dict(W=None), 10), (dict(W=18), 10),
    (dict(eps=-1e-6), 11), (dict(eps=float("nan")), 11), (dict(eps=float("inf")), 11),
    (dict(Q=None), 12), (dict(ldq=7), 13), (dict(scales=None), 14), (dict(scales=18), 14),
])
def test_rmsnorm_argument_checks_need_no_gpu(kw, pos):
    a = dict(M=4, K=8, type=0, X=16, ldx=8, R=32, ldr=8, H=48, ldh=8, W=16, eps=1e-5, Q=16, ldq=8,
             scales=16)
    a.update(kw)
    assert fg.s8_rmsnorm(*a.values(), 0) == -pos


def test_row_operators_of_no_rows_need_no_gpu():
    assert fg.s8_quantize(0, 0, 8, 0, None, 8, None, 8, None, 0) == 0
    assert fg.s8_rmsnorm(0, 8, 0, None, 8, None, 0, None, 0, None, 0.0, None, 8, None, 0) == 0


# ---- the product ----------------------------------------------------------------

@gpu
@pytest.mark.parametrize("cfg", range(len(CONFIGS)), ids=CONFIGS)
@pytest.mark.parametrize("aligned", [True, False], ids=["wide", "bytes"])
def test_gemm_every_configuration(cfg, aligned):
    require_gpu()
    for n, (M, N, K) in enumerate([(257, 129, 300), (65, 257, 512), (1, 1, 1), (16, 64, 128), (3, 70, 127),
                                   (130, 31, 1031), (300, 520, 2048), (128, 100, 5000), (33, 48, 1300),
                                   (17, 49, 640), (90, 16, 11008)]):
        ld = None if aligned else K + (n % 3)
        run_gemm(M, N, K, type=n % 3, cfg=cfg, lda=ld, ldb=ld, offa=0 if aligned else n % 5,
                 offb=0 if aligned else 3, beta=(0.0, 0.5)[n % 2], bias=n % 3 == 0, relu=n % 4 == 1, seed=cfg)


@gpu
@pytest.mark.parametrize("K", [1, 15, 16, 17, 63, 64, 127, 128, 129, 255, 257, 511, 640, 1023, 1025, 4099])
def test_gemm_k_ends_anywhere(K):
    """Every configuration with K inside a chunk, a slice, a stage; padding of 77s that must not count."""
    require_gpu()
    for cfg in range(len(CONFIGS)):
        run_gemm(40, 72, K, cfg=cfg, lda=-(-K // 16) * 16 + 16)
        run_gemm(40, 72, K, cfg=cfg, lda=K, ldb=K)


@gpu
@pytest.mark.parametrize("M", EDGES)
def test_gemm_ragged_rows_and_columns(M):
    require_gpu()
    for N in EDGES:
        run_gemm(M, N, 200, type=(M + N) % 3, bias=N % 2 == 1, relu=M % 2 == 1)


@gpu
@pytest.mark.parametrize("type", [0, 1, 2])
def test_gemm_strided_output_and_misaligned_c(type):
    require_gpu()
    for cfg in range(len(CONFIGS)):
        run_gemm(70, 90, 256, type=type, cfg=cfg, ldc=101, beta=1.0, bias=True)
        run_gemm(70, 88, 256, type=type, cfg=cfg, ldc=96, offc=1, beta=0.5)
        run_gemm(70, 96, 256, type=type, cfg=cfg, ldc=112, relu=True)


@gpu
def test_gemm_largest_sums():
    """K = 131071 of the largest codes: the sums reach 2^31 - 2^14 without wrapping."""
    require_gpu()
    K = 131071
    for cfg in range(len(CONFIGS)):
        A = torch.full((3, K + 1), -128, dtype=torch.int8, device="cuda")
        B = torch.full((5, K + 1), -128, dtype=torch.int8, device="cuda")
        B[1] = 127
        one = torch.ones(8, device="cuda")
        C = torch.empty(3, 5, device="cuda")
        rc = fg.fp32gemm_s8gemm_with_config(cfg, 3, 5, K, A, K + 1, one, B, K + 1, one, 0.0, 0, C, 5)
        assert rc == 0
        want = torch.tensor([K * 128 * 128, -K * 128 * 127] + [K * 128 * 128] * 3, dtype=torch.float32)
        assert torch.equal(C.cpu(), want.expand(3, 5))


@gpu
def test_gemm_empty_sum_is_the_epilogue():
    require_gpu()
    for type in (0, 1, 2):
        t = ref.TYPES[type]
        C = torch.tensor([[1.0, -2.0, 3.0], [4.0, -5.0, 0.5]]).to(t).cuda()
        bias = torch.tensor([0.5, 0.25, -8.0], device="cuda")
        assert fg.s8gemm(2, 3, 0, None, 1, None, None, 1, None, 2.0, type, C, 3, bias, fg.ACT_RELU) == 0
        assert torch.equal(C.cpu().float(), torch.tensor([[2.5, 0.0, 0.0], [8.5, 0.0, 0.0]]))
        C.fill_(float("nan"))
        assert fg.s8gemm(2, 3, 0, None, 1, None, None, 1, None, 0.0, type, C, 3) == 0
        assert torch.equal(C.cpu().float(), torch.zeros(2, 3))


@gpu
def test_gemm_scales_that_are_not_numbers_stay_in_their_row_and_column():
    require_gpu()
    g = torch.Generator().manual_seed(5)
    for cfg in range(len(CONFIGS)):
        A, B = make_codes(g, 20, 96).cuda(), make_codes(g, 40, 96).cuda()
        sA, sB = torch.ones(20, device="cuda"), torch.ones(40, device="cuda")
        sA[7], sB[11], sA[3] = float("nan"), float("nan"), 0.0
        C = torch.empty(20, 40, device="cuda")
        assert fg.fp32gemm_s8gemm_with_config(cfg, 20, 40, 96, A, 96, sA, B, 96, sB, 0.0, 0, C, 40) == 0
        nan = torch.isnan(C.cpu())
        want = torch.zeros(20, 40, dtype=torch.bool)
        want[7], want[:, 11] = True, True
        assert torch.equal(nan, want)
        assert fg.fp32gemm_s8gemm_with_config(cfg, 20, 40, 96, A, 96, sA, B, 96, sB, 0.0, 0, C, 40, None,
                                              fg.ACT_RELU) == 0
        assert torch.equal(torch.isnan(C.cpu()), want) and not bool((C < 0).any())
        assert bool((C[3][~torch.isnan(C[3])] == 0).all())


@gpu
def test_gemm_same_bits_whatever_the_configuration():
    """The sums are exact, so every configuration and both load paths give the same bits."""
    require_gpu()
    M, N, K = 100, 200, 1111
    outs = [run_gemm(M, N, K, type=0, cfg=cfg, bias=True, beta=0.5, lda=ld, ldb=ld).clone()
            for cfg in range(-1, len(CONFIGS)) for ld in (None, K)]
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


# ---- codes of rows and columns ------------------------------------------------------

def check_quantize(X, columns=False, ldx=None, ldq=None, offx=0, offq=0):
    V = X.t() if columns else X
    M, K = V.shape
    type = [t for t, d in ref.TYPES.items() if d == X.dtype][0]
    ldx = ldx or max(1, X.shape[1])
    ldq = ldq or max(1, K)
    dX, _ = device(X, ldx, offx)
    Q, flat = device(torch.zeros(M, K, dtype=torch.int8), ldq, offq)
    S = torch.full((M + 2,), 5.0, device="cuda")
    rc = fg.s8_quantize(int(columns), M, K, type, dX, ldx, Q, ldq, S[1:])
    assert rc == 0, fg.strerror(rc)
    torch.cuda.synchronize()
    q, s = ref.codes(V.double())
    what = (tuple(X.shape), str(X.dtype), columns)
    assert torch.equal(torch.isnan(S[1:-1].cpu()), torch.isnan(s)), what
    assert torch.equal(torch.nan_to_num(S[1:-1].cpu()), torch.nan_to_num(s)), what
    assert torch.equal(Q.cpu().long(), q), what
    assert untouched(flat, (M, K), ldq, offq, 77), what
    assert float(S[0]) == 5.0 and float(S[-1]) == 5.0
    return Q, S


ROW_LENGTHS = [1, 2, 7, 8, 9, 63, 64, 511, 512, 513, 2047, 2049, 4096, 4100, 8192, 8193, 11008, 16384, 16385,
               20000, 33000]


@gpu
@pytest.mark.parametrize("K", ROW_LENGTHS)
@pytest.mark.parametrize("dtype", list(ref.TYPES.values()), ids=str)
def test_quantize_rows(K, dtype):
    require_gpu()
    g = torch.Generator().manual_seed(K)
    for M in (1, 5):
        X = (torch.randn(M, K, generator=g) * 3).to(dtype)
        check_quantize(X)
        check_quantize(X, ldx=K + 3, ldq=-(-K // 16) * 16 + 16, offx=1, offq=5)


@gpu
@pytest.mark.parametrize("dtype", list(ref.TYPES.values()), ids=str)
@pytest.mark.parametrize("shape", [(1, 1), (1, 300), (300, 1), (31, 33), (32, 64), (65, 130), (200, 1000),
                                   (4097, 70), (9000, 33), (4096, 600),
                                   (2049, 200), (1025, 17), (20000, 1)])
def test_quantize_columns(shape, dtype):
    require_gpu()
    g = torch.Generator().manual_seed(shape[0])
    X = (torch.randn(*shape, generator=g) * 0.02).to(dtype)
    check_quantize(X, columns=True)
    check_quantize(X, columns=True, ldx=shape[1] + 5, ldq=shape[0] + 3, offx=1, offq=1)


def odd_rows(dtype, K=600):
    """Rows where a code is decided by the last bit, or where there is none."""
    big = float(torch.finfo(dtype).max)
    tiny = float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps
    X = torch.zeros(16, K)
    X[1] = (torch.arange(K) % 255 - 127) * 0.5            # halves, scale 0.5: every tie
    X[1, 0] = 63.5
    X[2, 5] = float("nan")
    X[3, 599] = float("inf")
    X[4, 0], X[4, 1] = float("-inf"), float("nan")
    X[5] = big
    X[6], X[6, 1::2] = -big, big / 2
    X[7] = tiny
    X[8] = torch.arange(K) * tiny
    X[9] = torch.linspace(-1, 1, K) * 1e-38
    X[10, 77] = -3.0                                      # one value
    X[11] = -0.0
    X[12] = 127.0
    X[12, ::3] = torch.arange(200) + 0.5 - 100
    X[13] = (torch.arange(K) - 300) * (127.0 / 254)
    X[14] = torch.linspace(-2.0 ** -100, 2.0 ** -100, K)
    X[15] = 1.0
    X[15, ::2] = 0.5 / 127                                # next to half a code
    return X.to(dtype)


@gpu
@pytest.mark.parametrize("dtype", list(ref.TYPES.values()), ids=str)
def test_quantize_rows_that_decide_by_a_bit_or_hold_no_number(dtype):
    require_gpu()
    X = odd_rows(dtype)
    check_quantize(X)
    check_quantize(X.t().contiguous(), columns=True)
    longer = torch.nn.functional.pad(X, (0, 5000))  # K over workgroups
    check_quantize(longer.t().contiguous(), columns=True)
    check_quantize(torch.cat([longer] * 9 + [longer[:5]]).t().contiguous(), columns=True, offx=1, offq=3)


@gpu
def test_quantize_values_next_to_halves():
    """fp32 values one step either side of (k + 1/2) scale, for many scales, among them subnormal ones."""
    require_gpu()
    rows = []
    for n, a in enumerate([127.0, 1.0, 0.3, 3.7e5, 2.9e38, 1.3e-30, 5e-37, 1.1e-38, 4e-43]):
        s = np.float32(a) / np.float32(127)
        mid = ((np.arange(127) + 0.5) * np.float64(s)).astype(np.float32)
        up, down = np.nextafter(mid, np.float32(np.inf)), np.nextafter(mid, np.float32(0))
        row = np.concatenate([[np.float32(a)], mid, up, down])
        rows.append(np.clip(row, 0, np.float32(a)) * np.where(np.arange(382) % 2, -1, 1).astype(np.float32))
    X = torch.from_numpy(np.stack(rows).astype(np.float32))
    check_quantize(X)
    check_quantize(X.t().contiguous(), columns=True)
    check_quantize(torch.nn.functional.pad(X, (0, 9000)).t().contiguous(), columns=True)
    check_quantize(torch.nn.functional.pad(X, (0, 16000)))  # rows of the longer kernels
    check_quantize(torch.nn.functional.pad(X, (0, 20000)))


@gpu
def test_quantize_no_values():
    require_gpu()
    S = torch.full((4,), 5.0, device="cuda")
    for trans in (0, 1):
        assert fg.s8_quantize(trans, 3, 0, 0, None, 3, None, 1, S) == 0
        assert S.tolist() == [0.0, 0.0, 0.0, 5.0]
    assert fg.s8_rmsnorm(4, 0, 2, None, 1, None, 0, None, 0, None, 1e-5, None, 1, S) == 0
    assert S.tolist() == [0.0] * 4


# ---- the norm -----------------------------------------------------------------------

def check_rmsnorm(X, R, W, eps, store=True, in_place=None, ld=None, off=0):
    M, K = X.shape
    type = [t for t, d in ref.TYPES.items() if d == X.dtype][0]
    ld = ld or K
    dX, fx = device(X, ld, off)
    dR, fr = device(R, ld, off) if R is not None else (None, None)
    dH, fh = (None, None) if not store else {"x": (dX, fx), "r": (dR, fr)}.get(
        in_place) or device(torch.zeros_like(X), ld, off)
    Q, flat = device(torch.zeros(M, K, dtype=torch.int8), ld, off)
    S = torch.full((M + 1,), 5.0, device="cuda")
    rc = fg.s8_rmsnorm(M, K, type, dX, ld, dR, ld, dH, ld, W.cuda(), eps, Q, ld, S)
    assert rc == 0, fg.strerror(rc)
    torch.cuda.synchronize()
    h, q, step, scale = ref.rmsnorm(X, R, W, eps)
    what = (tuple(X.shape), str(X.dtype), R is not None, in_place)
    assert torch.equal(Q.cpu().long(), q), what
    got = S[:-1].cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(scale)), what
    got, scale = torch.nan_to_num(got), torch.nan_to_num(scale)
    # one rounding to fp32 (its half step at the smallest values), after sums in 64 bits
    assert bool(((got - scale).abs() <= scale * (ref.U32 + 1e-11) + 2.0 ** -150).all()), what
    assert float(S[-1]) == 5.0
    assert untouched(flat, (M, K), ld, off, 77), what
    if store:
        assert torch.equal(torch.nan_to_num(dH.cpu().float(), nan=9.0), torch.nan_to_num(h.float(), nan=9.0)), what
        assert untouched(fh, (M, K), ld, off, float("nan")), what
    return S


@gpu
@pytest.mark.parametrize("K", ROW_LENGTHS)
@pytest.mark.parametrize("dtype", list(ref.TYPES.values()), ids=str)
def test_rmsnorm(K, dtype):
    require_gpu()
    g = torch.Generator().manual_seed(K)
    W = (1 + 0.2 * torch.randn(K, generator=g)).to(dtype)
    for M in (1, 6):
        X, R = ((torch.randn(M, K, generator=g) * 3).to(dtype) for _ in range(2))
        check_rmsnorm(X, R, W, 1e-5)
        check_rmsnorm(X, R, W, 1e-6, in_place="r")
        check_rmsnorm(X, R, W, 1e-5, in_place="x", ld=K + 5, off=1)
        check_rmsnorm(X, R, W, 0.0, store=False, ld=K + 1)
        check_rmsnorm(X, None, W, 1e-5, store=False)
        check_rmsnorm(X, None, W, 1.0, in_place="x")


@gpu
@pytest.mark.parametrize("dtype", list(ref.TYPES.values()), ids=str)
def test_rmsnorm_odd_rows(dtype):
    """Zeros, one value, ties, infinities and NaN; fp32 values whose squares pass fp32's range."""
    require_gpu()
    X = odd_rows(dtype)
    one = torch.ones(X.shape[1], dtype=dtype)
    for eps in (0.0, 1e-5):
        check_rmsnorm(X, None, one, eps)
        check_rmsnorm(X, torch.zeros_like(X), one, eps, in_place="r")
    W = one.clone()
    W[::2] = 0.0
    check_rmsnorm(X, None, W, 1e-5)
    check_rmsnorm(X, None, torch.zeros_like(W), 1e-5)
    check_rmsnorm(torch.nn.functional.pad(X, (0, 20000)), None, torch.nn.functional.pad(one, (0, 20000)), 1e-5)


# ---- sizes past one launch, offsets past 32 bits ----------------------------------------

@gpu
def test_more_rows_than_one_launch_takes():
    """Row operators beyond 2^21 rows, and a product whose configuration runs in several launches."""
    require_gpu()
    M, K = 2 ** 21 + 77, 5
    X = torch.randn(M, K, device="cuda")
    Q, S = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    assert fg.s8_quantize(0, M, K, 0, X, K, Q, K, S) == 0
    q, s = ref.codes(X.cpu().double())
    assert torch.equal(Q.cpu().long(), q) and torch.equal(S.cpu(), s)
    H = torch.empty_like(X)
    w = torch.rand(K)
    assert fg.s8_rmsnorm(M, K, 0, X, K, X, K, H, K, w.cuda(), 1e-5, Q, K, S) == 0
    h, q, _, s = ref.rmsnorm(X.cpu(), X.cpu(), w, 1e-5)
    assert torch.equal(H.cpu(), h) and torch.equal(Q.cpu().long(), q)
    assert bool(((S.cpu().double() - s).abs() <= s * (ref.U32 + 1e-11)).all())
    g = torch.Generator().manual_seed(1)
    M, N, K = 4 * 65535 * 2 + 9, 3, 33
    A, B = make_codes(g, M, K), make_codes(g, N, K)
    sA, sB = torch.rand(M, generator=g), torch.rand(N, generator=g)
    z, bound = ref.gemm(A, sA, B, sB, 0.0, None, None, False, 0)
    for cfg in (-1, CONFIGS.index("gemv_r2"), CONFIGS.index("16x16_k4_s4")):
        C = torch.full((M, N), float("nan"), device="cuda")
        assert fg.fp32gemm_s8gemm_with_config(cfg, M, N, K, A.cuda(), K, sA.cuda(), B.cuda(), K, sB.cuda(),
                                              0.0, 0, C, N) == 0
        assert bool(((C.cpu().double() - z).abs() <= bound).all()), cfg


@gpu
def test_offsets_past_32_bits():
    """The largest leading dimension with enough rows that byte offsets pass 2^32 in every operand."""
    require_gpu()
    ld, M, K, N = 1 << 20, 4100, 70, 50
    g = torch.Generator().manual_seed(2)
    X = torch.empty(M, ld, dtype=torch.bfloat16, device="cuda")[:, :K]
    X.copy_(torch.randn(M, K, generator=g).bfloat16())
    Q = torch.empty(M, ld, dtype=torch.int8, device="cuda")[:, :K]
    S = torch.empty(M, device="cuda")
    w = torch.ones(K, dtype=torch.bfloat16)
    assert fg.s8_rmsnorm(M, K, 2, X, ld, None, 0, X, ld, w.cuda(), 1e-5, Q, ld, S) == 0
    _, q, _, s = ref.rmsnorm(X.cpu(), None, w, 1e-5)
    assert torch.equal(Q.cpu().long(), q)
    assert fg.s8_quantize(0, M, K, 2, X, ld, Q, ld, S) == 0
    q, s = ref.codes(X.cpu().double())
    assert torch.equal(Q.cpu().long(), q) and torch.equal(S.cpu(), s)
    QT, ST = torch.empty(K, M, dtype=torch.int8, device="cuda"), torch.empty(K, device="cuda")
    assert fg.s8_quantize(1, K, M, 2, X, ld, QT, M, ST) == 0
    qt, st = ref.codes(X.cpu().double().t())
    assert torch.equal(QT.cpu().long(), qt) and torch.equal(ST.cpu(), st)
    B = make_codes(g, N, K)
    sB = torch.rand(N, generator=g)
    C = torch.empty(M, ld, dtype=torch.float16, device="cuda")[:, :N]
    z, bound = ref.gemm(Q.cpu(), S.cpu(), B, sB, 0.0, None, None, False, 1)
    for cfg in (-1, CONFIGS.index("256x256_k1_s2"), CONFIGS.index("64x64_k2_s4"), CONFIGS.index("gemv_r2k4")):
        C.fill_(float("nan"))
        assert fg.fp32gemm_s8gemm_with_config(cfg, M, N, K, Q, ld, S, B.cuda(), K, sB.cuda(), 0.0, 1, C, ld) == 0
        assert bool(((C.cpu().double() - z).abs() <= bound).all()), cfg
    # the weight's rows that far apart: C is its own leading dimension wide
    C2 = torch.empty(3, M, device="cuda")
    A = make_codes(g, 3, K).cuda()
    one = torch.ones(3, device="cuda")
    z, bound = ref.gemm(A.cpu(), one.cpu(), Q.cpu(), S.cpu(), 0.0, None, None, False, 0)
    for cfg in range(-1, len(CONFIGS)):
        C2.fill_(float("nan"))
        assert fg.fp32gemm_s8gemm_with_config(cfg, 3, M, K, A, K, one, Q, ld, S, 0.0, 0, C2, M) == 0
        assert bool(((C2.cpu().double() - z).abs() <= bound).all()), cfg


@gpu
def test_same_bits_from_call_to_call():
    require_gpu()
    g = torch.Generator().manual_seed(3)
    X = torch.randn(300, 5003, generator=g).cuda()
    w = torch.rand(5003, generator=g).cuda()
    runs = []
    for _ in range(5):
        Q, S = torch.empty(300, 5008, dtype=torch.int8, device="cuda")[:, :5003], torch.empty(300, device="cuda")
        assert fg.s8_rmsnorm(300, 5003, 0, X, 5003, None, 0, None, 0, w, 1e-5, Q, 5008, S) == 0
        C = torch.empty(300, 300, device="cuda")
        assert fg.s8gemm(300, 300, 5003, Q, 5008, S, Q, 5008, S, 0.0, 0, C, 300) == 0
        torch.matmul(X, X.t())
        runs.append((Q, S, C))
    for q, s, c in runs[1:]:
        assert torch.equal(q, runs[0][0]) and torch.equal(s, runs[0][1]) and torch.equal(c, runs[0][2])

# ---- scales at the ends of fp32's range ---------------------------------------------------

def run_extreme_scales(cfg, type, aligned, beta, bias):
    """(C, value in 64 bits, |value| bound, sum times scaleA) with scales from subnormal to the largest."""
    g = torch.Generator().manual_seed(17)
    top = float(np.float32(np.finfo(np.float32).max) / np.float32(127))  # the largest that s8_quantize makes
    sA = torch.tensor([top, -top, 2.0 ** 96, 2.0 ** 97, 1e30, 1.0, 1e-30, 1e-40, 2.0 ** -149, 0.0, top, 3e38,
                       3.5e33, 7e28, 8e28, 1e37, 2e20], dtype=torch.float32)
    sB = torch.tensor([1e-4, 1.0, 1e-30, 1e-33, 1e-36, 1e-38, 1e-40, 2.0 ** -149, 0.0, 1e20, top, -1e-5, 3e38],
                      dtype=torch.float32).repeat(6)
    M, N, K = len(sA), len(sB), 201
    A, B = make_codes(g, M, K), make_codes(g, N, K)
    A[10] = 0  # sums of zero under the largest scales
    ld = 208 if aligned else K
    dA, _ = device(A, ld)
    dB, _ = device(B, ld)
    t = ref.TYPES[type]
    C0 = torch.randn(M, N, generator=g).to(t)
    bv = torch.randn(N, generator=g) if bias else None
    C = C0.cuda() if beta else torch.full((M, N), float("nan"), dtype=t, device="cuda")
    rc = fg.fp32gemm_s8gemm_with_config(cfg, M, N, K, dA, ld, sA.cuda(), dB, ld, sB.cuda(), beta, type, C, N,
                                        bv.cuda() if bias else None)
    assert rc == 0, fg.strerror(rc)
    z, bound = ref.gemm(A, sA, B, sB, beta, C0, bv, False, type)
    return C.cpu(), z, bound, (A.double() @ B.double().t()) * sA.double()[:, None]


@gpu
@pytest.mark.parametrize("type", [0, 1, 2])
def test_gemm_scales_at_the_ends_of_their_range(type):
    """sum scaleA may pass fp32's range where sum scaleA scaleB does not: every element whose value is
    finite in C's type is within the bound, every other infinite with its sign, and a sum of zero is zero."""
    require_gpu()
    top = float(torch.finfo(ref.TYPES[type]).max)
    for cfg in range(-1, len(CONFIGS)):
        for aligned in (True, False):
            for beta, bias in ((0.0, False), (0.5, True)):
                C, z, bound, part = run_extreme_scales(cfg, type, aligned, beta, bias)
                what = (cfg, aligned, beta)
                inside, outside = z.abs() < 0.99 * top, z.abs() > 1.01 * top
                # what the case is about, and what it is told from
                assert int((inside & (part.abs() > 3.5e38) & (z.abs() > 0)).sum()) > 60
                assert int(outside.sum()) > 100
                err = (C.double() - z).abs()
                assert bool((err <= bound)[inside].all()), (what, (inside & ~(err <= bound)).nonzero()[:4].tolist())
                assert bool((torch.isinf(C) & (C.sign() == z.sign()))[outside].all()), what
                if not beta:
                    assert bool((C[10] == 0).all()) and bool((C[9] == 0).all()), what


@gpu
def test_gemm_same_bits_at_the_ends_of_the_scales_range():
    require_gpu()
    outs = [run_extreme_scales(cfg, 0, aligned, 0.5, True)[0]
            for cfg in range(-1, len(CONFIGS)) for aligned in (True, False)]
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@gpu
def test_layer_of_rows_near_the_largest_float():
    """Codes made from rows of 1e36, times a weight near 1e-4: every product is finite."""
    require_gpu()
    g = torch.Generator().manual_seed(23)
    X = torch.randn(5, 300, generator=g) * 1e36
    W = torch.randn(40, 300, generator=g) * 1e-4
    for x, w in ((X, W), (W[:9], X)):
        cx, sx = fg.quantize_s8(x.cuda())
        cw, sw = fg.quantize_s8(w.cuda())
        z, bound = ref.gemm(cx.cpu(), sx.cpu(), cw.cpu(), sw.cpu(), 0.0, None, None, False, 0)
        y = fg.gemm_s8(cx, sx, cw.t(), sw).cpu().double()
        assert bool(torch.isfinite(y).all()) and bool(((y - z).abs() <= bound).all())


@gpu
def test_tiles_of_more_than_one_launch():
    """A tile configuration past the tiles of one launch (2^21): rows 512 and up run in the second one.

    Values of 65520 and more round to infinity in fp16; next to that border either side is right,
    as far as the fp32 roundings of the epilogue (6 of them) can move a value.
    """
    require_gpu()
    M, N, K = 530, 1 << 20, 16
    cfg = CONFIGS.index("16x16_k4_s4")
    g = torch.Generator().manual_seed(4)
    A = make_codes(g, M, K).cuda()
    sA = torch.rand(M, generator=g).cuda()
    B = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda")
    sB = torch.rand(N, device="cuda")
    C = torch.full((M + 1, N), float("nan"), dtype=torch.float16, device="cuda")
    assert fg.fp32gemm_s8gemm_with_config(cfg, M, N, K, A, K, sA, B, K, sB, 0.0, 1, C, N) == 0
    assert bool(torch.isnan(C[M]).all())
    for n0 in range(0, N, 1 << 17):
        n = slice(n0, n0 + (1 << 17))
        z, bound = ref.gemm(A, sA, B[n], sB[n], 0.0, None, None, False, 1)
        got = C[:M, n].double()
        past = torch.isinf(got) & (got.sign() == z.sign()) & (z.abs() * (1 + 6.001 * ref.U32) >= 65520)
        near = z.abs() * (1 - 6.001 * ref.U32) < 65520
        assert bool((((got - z).abs() <= bound) & near | past).all()), n0


def test_gemm_choice_for_few_rows():
    """One and two rows are dot products whatever W's size, wide weights past the fitted sizes among them;
    five to eight rows, which read W twice as dot products, are tiles where W is wide."""
    sizes = [1, 64, 1000, 2048, 4096, 6400, 8448, 11008, 14336, 14592, 16384, 22784, 28672, 32000, 65536, 128256, 1 << 20]
    dots = lambda M, N, K: CONFIGS[fg.fp32gemm_select_config(fg.KIND_S8GEMM, M, N, K)].startswith("gemv")
    for N in sizes:
        for K in (1, 128, 443, 1024, 4096, 8192, 11008, 28672, 131071):
            assert dots(1, N, K) and dots(2, N, K), (N, K)
            for M in (5, 6, 7, 8):
                assert N <= 2048 or not dots(M, N, K), (M, N, K)
            for M in (9, 64):
                assert not dots(M, N, K), (M, N, K)
    assert dots(8, 131, 10653) and dots(4, 11008, 4096)


@pytest.mark.parametrize("name,mean,most", [("s8_aligned", 1.025, 1.55), ("s8_unaligned", 1.04, 1.85),
                                            ("s8_large", 1.01, 1.2), ("s8_wide_cold", 1.04, 1.45)])
def test_gemm_choice_against_recorded_times(name, mean, most):
    """The chosen configuration's time over the best one's, in the recorded times of all of them."""
    path = os.path.join(os.path.dirname(__file__), "..", "profiles", "sweeps", name + ".csv")
    with open(path) as f:
        lines = [line.split(",") for line in f.read().split("\n") if line]
    assert lines[0][3:] == CONFIGS
    ratios = []
    for line in lines[1:]:
        times = [float(t) if t else None for t in line[3:]]
        chosen = times[fg.fp32gemm_select_config(fg.KIND_S8GEMM, *map(int, line[:3]))]
        if chosen is not None:
            ratios.append(chosen / min(t for t in times if t is not None))
    assert len(ratios) > 0.9 * (len(lines) - 1)
    assert np.exp(np.log(ratios).mean()) < mean and max(ratios) < most
