"""The FP8 quantizer, the FP8 and grouped products and the FP8 experts against float64.

Tolerances.  A sum of K products in fp32, in any order, is off by at most about
K 2^-24 of the sum of magnitudes; a scaled FP8 sum has four more roundings per
block, so (K + 4 KB + 4) 2^-24 sum|p| covers it.  A bf16 output adds half a step,
2^-8 of the value.  bf16 outputs of FP8 operands may come from the FP8 matrix
instruction, whose sum over a block of 128 is off by at most 2^-11 of the
block's sum of magnitudes (twice the 2.3e-4 that the header states).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import fp8, formats, moe, mx
from tests.helpers import check_close

pytestmark = pytest.mark.gpu

BF16, F32, FP8 = 1, 0, 4
EPS32, HALF_BF16, FP8_SUM = 2.0 ** -24, 2.0 ** -8, 2.0 ** -11


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from expert_cached_ffn_amd import ops as _ops
    _ops.version()
    return _ops


def say(*a):
    print(*a, flush=True)


def cdiv(a, b):
    return -(-a // b)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes_of(g, *shape):
    """E4M3 codes of a bell curve reaching +-448, as bytes."""
    v = torch.randn(shape, generator=g, device="cuda").mul_(112).clamp_(-448, 448)
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def scales_of(g, *shape):
    return torch.rand(shape, generator=g, device="cuda").add_(0.5).mul_(0.01)


def values(codes, scales, rows):
    """Codes times their blocks' scales, float64 on the GPU."""
    n, K = codes.shape
    v = codes.contiguous().view(torch.float8_e4m3fn).double()
    i = torch.arange(n, device="cuda") // rows
    j = torch.arange(K, device="cuda") // 128
    return v * scales.double()[i][:, j]


def check_product(got, a, w, K, out, fp8_ops, what):
    """got against a @ w.T (float64), each output within the bound of the module's docstring."""
    ref, mag = a @ w.T, a.abs() @ w.abs().T
    KB = cdiv(K, 128)
    tol = (K + 4 * KB + 4) * EPS32 * mag
    if out == BF16:
        tol = tol + HALF_BF16 * (ref.abs() + tol)
        if fp8_ops:
            tol = tol + FP8_SUM * mag * (1 + HALF_BF16)
    d = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all(), what
    worst = (d / (tol + 1e-300)).max().item() if d.numel() else 0.0
    assert worst <= 1, f"{what}: {worst:.3f} of the bound"


# ----------------------------------------------------------------------------- quantizer

QUANT = [(1, 16, 0), (1, 128, 0), (3, 112, 16), (5, 144, 0), (17, 2048, 80), (128, 256, 0), (129, 400, 8), (300, 768, 0), (1000, 4096, 0)]


@pytest.mark.parametrize("x_dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("n,K,pad", QUANT)
def test_quantize_bit_exact(ops, x_dtype, rows, n, K, pad):
    say("quantize", x_dtype, rows, n, K, pad)
    rng = np.random.default_rng(n * 1000 + K + rows)
    x = rng.standard_normal((n, K + pad)) * np.exp(rng.uniform(-20, 20, (n, 1)))
    x[0, :8] = [448.0, 17.0, 19.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10, -0.0, 0.0]   # ties on the scale's own grid
    if n > 2:
        x[1, :], x[2, :] = 0.0, 2.0 ** -133                                         # nothing; only subnormals
    if K > 128:
        x[0, 128:min(K, 256)] *= 1e30
    xt = torch.from_numpy(x.astype(np.float32)).cuda()
    if x_dtype == BF16:
        xt = xt.to(torch.bfloat16)
    ldc = cdiv(K, 16) * 16 + 32
    codes = torch.full((n, ldc), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((cdiv(n, rows) + 1, cdiv(K, 128)), -7.0, device="cuda")
    ops.ft_fp8_quantize(xt, x_dtype, K + pad, n, K, rows, codes, ldc, scales)
    torch.cuda.synchronize()
    ref_c, ref_s = fp8.quantize(xt[:, :K].double().cpu().numpy(), rows)
    assert np.array_equal(scales[:-1].double().cpu().numpy(), ref_s, equal_nan=True)
    got = codes.cpu().numpy()
    assert np.array_equal(mx.e4m3_to_f64(got[:, :K]), mx.e4m3_to_f64(ref_c))
    assert np.array_equal(got[:, :K], ref_c)
    assert np.all(got[:, K:] == 0xA5) and torch.all(scales[-1] == -7.0)


def test_quantize_bad_blocks(ops):
    x = torch.ones((4, 384), device="cuda")
    x[1, 5], x[2, 200], x[3, 383] = float("nan"), float("inf"), -float("inf")
    for dt, xt in ((F32, x), (BF16, x.to(torch.bfloat16))):
        codes = torch.empty((4, 384), dtype=torch.uint8, device="cuda")
        scales = torch.empty((4, 3), device="cuda")
        ops.ft_fp8_quantize(xt, dt, 384, 4, 384, 1, codes, 384, scales)
        ref_c, ref_s = fp8.quantize(x.double().cpu().numpy())
        assert np.array_equal(codes.cpu().numpy(), ref_c)
        np.testing.assert_array_equal(scales.double().cpu().numpy(), ref_s)
        big = torch.empty((1, 3), device="cuda")
        ops.ft_fp8_quantize(xt, dt, 384, 4, 384, 128, codes, 384, big)
        assert torch.isnan(big).all() and not codes.any()


# ----------------------------------------------------------------------------- dense product

GEMM = [(1, 1, 16), (1, 16, 128), (1, 4096, 4096), (2, 100, 144), (5, 129, 1040), (16, 64, 128), (17, 200, 400), (33, 1001, 2000),
        (64, 256, 768), (65, 130, 272), (100, 128, 128), (128, 512, 512), (200, 77, 656), (255, 257, 384), (256, 256, 1024),
        (300, 520, 4096), (513, 300, 112), (1030, 640, 896), (70, 100, 8400), (1000, 6200, 400), (1000, 6200, 8352),
        (3600, 4100, 272), (3600, 4100, 8320)]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("M,N,K", GEMM)
def test_fp8_gemm(ops, out, M, N, K):
    say("gemm", out, M, N, K)
    g = gen(M * 7 + N * 3 + K)
    lda, ldw, ldo = K + 48, K + 16, N + 5
    a = torch.full((M, lda), 0x7F, dtype=torch.uint8, device="cuda")     # NaN codes behind the rows
    w = torch.full((N, ldw), 0xFF, dtype=torch.uint8, device="cuda")
    a[:, :K], w[:, :K] = codes_of(g, M, K), codes_of(g, N, K)
    sa, sw = scales_of(g, M, cdiv(K, 128)), scales_of(g, cdiv(N, 128), cdiv(K, 128))
    dt = torch.bfloat16 if out == BF16 else torch.float32
    o = torch.full((M, ldo), -3.0, dtype=dt, device="cuda")
    ops.ft_fp8_gemm(a, lda, sa, w, ldw, sw, M, N, K, out, o, ldo)
    torch.cuda.synchronize()
    check_product(o[:, :N], values(a[:, :K], sa, 1), values(w[:, :K], sw, 128), K, out, True, (M, N, K))
    assert torch.all(o[:, N:] == -3.0)


def test_fp8_gemm_wide_range_and_nan(ops):
    """Uniform code bytes (the widest range of products), a row and a weight block with NaN."""
    M, N, K = 40, 300, 640
    for out in (BF16, F32):
        g = gen(5)
        a, w = (torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8) for s in ((M, K), (N, K)))
        for t in (a, w):
            t[(t & 0x7F) == 0x7F] = 0x31
        sa, sw = scales_of(g, M, 5) * torch.exp(torch.randn((M, 5), generator=g, device="cuda") * 3), scales_of(g, 3, 5)
        o = torch.empty((M, N), dtype=torch.bfloat16 if out == BF16 else torch.float32, device="cuda")
        ops.ft_fp8_gemm(a, K, sa, w, K, sw, M, N, K, out, o, N)
        check_product(o, values(a, sa, 1), values(w, sw, 128), K, out, True, out)
        good = o.clone()
        a[7, 130] = 0x7F
        sw[1, 4] = float("nan")
        sa[9, 0] = float("inf")
        ops.ft_fp8_gemm(a, K, sa, w, K, sw, M, N, K, out, o, N)
        assert torch.isnan(o[7]).all() and torch.isnan(o[:, 128:256]).all() and not torch.isfinite(o[9]).any()
        rows = [m for m in range(M) if m not in (7, 9)]
        cols = [n for n in range(N) if not 128 <= n < 256]
        assert torch.equal(o[rows][:, cols], good[rows][:, cols])


# ----------------------------------------------------------------------------- grouped product

def groups(rng, E, rows, empty=0.3):
    """Row counts of E groups summing to rows, some of them empty."""
    p = rng.random(E) ** 3 * (rng.random(E) > empty)
    if p.sum() == 0:
        p[rng.integers(E)] = 1
    return rng.multinomial(rows, p / p.sum())


def make_grouped(g, rng, dtype, T, k, E, N, K, gather, counts, pad=0):
    es = 2 if dtype == BF16 else 1
    rows = T * k
    off = np.zeros(E + 1, np.int32)
    off[1:] = np.cumsum(counts)
    n = T if gather else rows
    if dtype == BF16:
        a = torch.full((n, K + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        a[:, :K] = torch.randn((n, K), generator=g, device="cuda").to(torch.bfloat16)
        w = (torch.randn((E, N, K), generator=g, device="cuda") * 0.05).to(torch.bfloat16)
        sa = sw = None
        a64, w64 = a[:, :K].double(), w.double()
        off_s = 0
        stride = cdiv(N * K * 2, 256) * 256 + 256
    else:
        a = torch.full((n, K + pad), 0x7F, dtype=torch.uint8, device="cuda")
        a[:, :K] = codes_of(g, n, K)
        w = codes_of(g, E, N, K)
        sa, sw = scales_of(g, n, cdiv(K, 128)), scales_of(g, E, cdiv(N, 128), cdiv(K, 128))
        a64 = values(a[:, :K], sa, 1)
        w64 = torch.stack([values(w[e], sw[e], 128) for e in range(E)])
        off_s = cdiv(N * K, 256) * 256 + 256
        stride = cdiv(off_s + sw[0].numel() * 4, 256) * 256
    slots = rng.permutation(E + 2)[:E].astype(np.int32)
    pool = torch.full((E + 2, stride), 0xFF, dtype=torch.uint8, device="cuda")     # NaN where nothing is laid
    off_w = 256 if dtype == BF16 else 0        # bf16 slots: one part in front
    for e in range(E):
        pool[slots[e], off_w:off_w + N * K * es] = w[e].contiguous().view(torch.uint8).view(-1)
        if sw is not None:
            pool[slots[e], off_s:off_s + sw[e].numel() * 4] = sw[e].contiguous().view(torch.uint8).view(-1)
    src = rng.permutation(rows).astype(np.int32) if gather else None
    return dict(a=a, sa=sa, pool=pool, stride=stride, off_w=off_w, off_s=off_s, slots=slots, off=off, src=src, a64=a64, w64=w64)


def run_grouped(ops, d, dtype, T, k, E, N, K, out, pad=0, ldo=None, slots=None, off=None, stream=None, o=None):
    ldo = ldo or N
    dt = torch.bfloat16 if out == BF16 else torch.float32
    o = torch.full((T * k, ldo), -3.0, dtype=dt, device="cuda") if o is None else o
    ops.ft_grouped_gemm(dtype, d["a"], K + pad, d["sa"], d["pool"], d["stride"], d["off_w"], d["off_s"], E + 2,
                        torch.from_numpy(d["slots"] if slots is None else slots).cuda(), T, k, E,
                        torch.from_numpy(d["off"] if off is None else off).cuda(),
                        None if d["src"] is None else torch.from_numpy(d["src"]).cuda(), N, K, out, o, ldo, stream=stream)
    torch.cuda.synchronize()
    return o


def check_grouped(d, o, dtype, k, E, N, K, out, skip=(), what=""):
    off = d["off"]
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi or e in skip:
            continue
        at = torch.arange(lo, hi) if d["src"] is None else torch.from_numpy(d["src"][lo:hi] // k).long()
        check_product(o[lo:hi, :N], d["a64"][at.cuda()], d["w64"][e], K, out, dtype == FP8, (what, e, hi - lo))


GROUPED = [  # T, k, E, N, K, gather, pad
    (1, 1, 1, 16, 16, True, 0), (1, 2, 4, 100, 144, True, 16), (3, 2, 5, 64, 128, False, 0), (5, 6, 40, 96, 256, True, 0),
    (16, 4, 8, 130, 400, True, 32), (64, 8, 16, 256, 512, True, 0), (33, 3, 300, 48, 64, False, 16), (100, 2, 3, 257, 272, False, 0),
    (130, 2, 2, 64, 1024, True, 0), (600, 1, 4, 300, 336, False, 0), (700, 4, 7, 128, 192, True, 16), (1500, 2, 5, 520, 768, True, 0),
    (64, 1, 1, 512, 2048, False, 0), (40, 2, 3, 80, 4352, True, 0), (130, 1, 2, 90, 12304, True, 0), (1500, 2, 20, 2100, 208, True, 0),
    (4000, 3, 12, 1500, 336, True, 16), (4000, 3, 12, 1500, 768, False, 0),
]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("T,k,E,N,K,gather,pad", GROUPED)
def test_grouped_gemm(ops, dtype, out, T, k, E, N, K, gather, pad):
    say("grouped", dtype, out, T, k, E, N, K, gather, pad)
    rng = np.random.default_rng(T * 131 + E * 17 + N + K)
    counts = groups(rng, E, T * k)
    d = make_grouped(gen(T + N + K), rng, dtype, T, k, E, N, K, gather, counts, pad)
    o = run_grouped(ops, d, dtype, T, k, E, N, K, out, pad, ldo=N + 3)
    check_grouped(d, o, dtype, k, E, N, K, out)
    assert torch.all(o[:, N:] == -3.0)


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("T,k,E", [(9, 2, 6), (200, 3, 6)])
def test_grouped_slots_and_short_offsets(ops, dtype, T, k, E):
    """A skipped group, groups without weights, offsets that end before the rows do, weights in any slot."""
    N, K = 144, 208
    rng = np.random.default_rng(T)
    rows = T * k
    counts = np.full(E, (rows - 3) // E)
    d = make_grouped(gen(T), rng, dtype, T, k, E, N, K, True, counts)
    slots = d["slots"].copy()
    slots[1], slots[2], slots[4] = -2, -1, E + 2
    for out in (BF16, F32):
        o = run_grouped(ops, d, dtype, T, k, E, N, K, out, slots=slots)
        check_grouped(d, o, dtype, k, E, N, K, out, skip=(1, 2, 4))
        off = d["off"]
        assert torch.all(o[off[1]:off[2]] == -3.0)
        for e in (2, 4):
            assert torch.isnan(o[off[e]:off[e + 1]]).all()
        assert off[E] < rows and torch.all(o[off[E]:] == -3.0)
    # offsets past the rows are held at T*k, and a row that names no token is computed from zeros
    off = d["off"].copy()
    off[E] = rows + 1000
    d["src"][off[0]] = -1
    d["src"][off[0] + 1] = rows + 5
    o = run_grouped(ops, d, dtype, T, k, E, N, K, F32, off=off)
    assert torch.all(o[off[0]:off[0] + 2] == 0)
    at = torch.from_numpy(d["src"][off[E - 1]:] // k).long().cuda()
    check_product(o[off[E - 1]:], d["a64"][at], d["w64"][E - 1], K, F32, dtype == FP8, "last group")


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("E", [64, 1024, 4096])
def test_grouped_many_groups(ops, dtype, E):
    """Up to 4096 groups, the limit, many of them empty or of one row; then all rows in the last one."""
    T, k, N, K = 300, 2, 16, 32
    rng = np.random.default_rng(3)
    counts = rng.multinomial(T * k, np.full(E, 1 / E))
    d = make_grouped(gen(4), rng, dtype, T, k, E, N, K, True, counts)
    off = torch.from_numpy(d["off"]).cuda()
    o = run_grouped(ops, d, dtype, T, k, E, N, K, F32)
    e = torch.searchsorted(off[1:].long(), torch.arange(T * k, device="cuda"), right=True)
    a = d["a64"][torch.from_numpy(d["src"] // k).long().cuda()]
    ref = (d["w64"][e] * a[:, None, :]).sum(2)
    mag = (d["w64"][e] * a[:, None, :]).abs().sum(2)
    assert ((o.double() - ref).abs() <= (K + 8) * EPS32 * mag).all()
    last = np.zeros(E + 1, np.int32)
    last[E] = T * k
    o = run_grouped(ops, d, dtype, T, k, E, N, K, F32, off=last)
    check_product(o, a, d["w64"][E - 1], K, F32, False, "last")


def test_rows_past_four_gigabytes(ops):
    """Operand rows whose byte offsets pass 32 bits, dense and in groups; the rows at the far end are checked."""
    M, N, K = 1_060_000, 32, 4096
    g = gen(21)
    base = codes_of(g, 5000, K)
    a = torch.empty((M, K), dtype=torch.uint8, device="cuda")
    for i in range(0, M, 5000):
        a[i:i + 5000] = base[:min(5000, M - i)].roll(i // 5000, 0)
    assert a.numel() > 1 << 32
    sa, w, sw = scales_of(g, M, 32), codes_of(g, 2, N, K), scales_of(g, 2, 1, 32)
    o = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    ops.ft_fp8_gemm(a, K, sa, w[0], K, sw[0], M, N, K, BF16, o, N)
    torch.cuda.synchronize()
    for at in (0, 524_000, 1_048_500, M - 300):
        check_product(o[at:at + 300], values(a[at:at + 300], sa[at:at + 300], 1), values(w[0], sw[0], 128), K, BF16, True, at)
    stride = N * K + 256
    pool = torch.zeros((2, stride), dtype=torch.uint8, device="cuda")
    for e in range(2):
        pool[e, :N * K] = w[e].reshape(-1)
        pool[e, N * K:N * K + 128] = sw[e].reshape(-1).view(torch.uint8)
    off = torch.tensor([0, 1_048_700, M], dtype=torch.int32, device="cuda")
    ops.ft_grouped_gemm(FP8, a, K, sa, pool, stride, 0, N * K, 2, None, M, 1, 2, off, None, N, K, BF16, o, N)
    torch.cuda.synchronize()
    for at, e in ((0, 0), (1_048_400, 0), (1_048_700, 1), (M - 300, 1)):
        check_product(o[at:at + 300], values(a[at:at + 300], sa[at:at + 300], 1), values(w[e], sw[e], 128), K, BF16, True, at)


def test_results_repeat_and_streams(ops):
    """Same bits on every run, on a stream of its own, and from two streams at once."""
    T, k, E, N, K = 70, 4, 9, 272, 640
    for dtype in (BF16, FP8):
        rng = np.random.default_rng(8)
        d = make_grouped(gen(9), rng, dtype, T, k, E, N, K, True, groups(rng, E, T * k))
        first = run_grouped(ops, d, dtype, T, k, E, N, K, F32)
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        slots, off, src = (torch.from_numpy(d[n]).cuda() for n in ("slots", "off", "src"))
        torch.cuda.synchronize()
        outs = []
        for i in range(6):
            o = [torch.empty((T * k, N), device="cuda") for _ in range(2)]
            torch.cuda.synchronize()
            for s in (s1, s2):
                ops.ft_grouped_gemm(dtype, d["a"], K, d["sa"], d["pool"], d["stride"], d["off_w"], d["off_s"], E + 2, slots,
                                    T, k, E, off, src, N, K, F32, o[s is s2], N, stream=s)
            outs += o
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, first)


# ----------------------------------------------------------------------------- FP8 experts

def fp8_experts(rng, E, H, I, std=0.05):
    """E experts as storage arrays and float64 matrices."""
    arrays, mats = [], []
    for _ in range(E):
        d, m = {}, []
        for n, s in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I))):
            c, sc = fp8.quantize(rng.standard_normal(s) * std, 128)
            sc = (sc * rng.uniform(1.0, 1.9, sc.shape)).astype(np.float32)      # a checkpoint's scales: any fp32
            d[f"{n}_codes"], d[f"{n}_scales"] = c, sc
            m.append(fp8.to_f64(c, sc, 128))
        arrays.append(d)
        mats.append(m)
    return arrays, mats


def expert_and_allowance(x, wg, wu, wd):
    """The oracle's expert on rows x, and how far the hidden vector's rounding may carry an output: g and u
    are off by at most 2^-11 of their sums of magnitudes, so each hidden value lies in an interval, and
    its code may be any that the interval's ends round to (with the block scale of either)."""
    xq = fp8.to_f64(*fp8.quantize(x))
    g, u = xq @ wg.T, xq @ wu.T
    eg, eu = (FP8_SUM * (np.abs(xq) @ np.abs(w).T) for w in (wg, wu))
    silu = g / (1 + np.exp(-g))
    h = silu * u
    eh = (np.abs(silu) + 1.1 * eg) * eu + 1.1 * eg * np.abs(u) + 2.0 ** -20 * np.abs(h)      # |silu'| < 1.1
    q = fp8.to_f64(*fp8.quantize(h))
    allow = np.zeros_like(h)
    m = fp8.block_max(h, 1)
    me = fp8.block_max(np.abs(h) + eh, 1)
    ml = fp8.block_max(np.maximum(np.abs(h) - eh, 0), 1)
    for mm in (m, me, ml):
        S = fp8.spread(fp8.scale_of(mm), 1, *h.shape)
        for v in (h, h - eh, h + eh):
            z = mx.e4m3_to_f64(mx.round_to_e4m3(v / S)) * S
            allow = np.maximum(allow, np.abs(z - q))
    y = q @ wd.T
    slack = FP8_SUM * (np.abs(q) @ np.abs(wd).T)
    return y, allow @ np.abs(wd).T + slack


def layer_case(rng, T, k, E, H, I, shared):
    arrays, mats = fp8_experts(rng, E + (1 if shared else 0), H, I)
    from expert_cached_ffn_amd import layer as L
    shape = L.LayerShape(H, I, E, k, "fp8", "bf16", "softmax", True, shared)
    lay = L.MoELayer(shape, T)
    blobs = [L.pack_expert(lay.layout, a) for a in arrays]
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    return lay, blobs, mats, x, logits


FFN = [(1, 2, 4, 256, 128, False), (1, 6, 16, 512, 256, True), (3, 2, 5, 208, 144, True), (5, 4, 8, 384, 272, False), (17, 3, 8, 256, 384, True),
       (64, 8, 16, 512, 128, False), (90, 4, 6, 272, 208, True), (300, 2, 3, 384, 256, True), (700, 2, 4, 256, 144, False),
       (700, 4, 16, 144, 1040, True), (6000, 2, 4, 128, 1040, True)]


@pytest.mark.parametrize("T,k,E,H,I,shared", FFN)
def test_fp8_layer(ops, T, k, E, H, I, shared):
    """Routing, permutation, the FP8 experts and the combine together, by the step calls and by the layer call."""
    say("layer", T, k, E, H, I, shared)
    rng = np.random.default_rng(T * 31 + E + H)
    lay, blobs, mats, x, logits = layer_case(rng, T, k, E, H, I, shared)
    pool = torch.from_numpy(np.stack(blobs[:E])).cuda()
    sh = torch.from_numpy(blobs[E]).cuda() if shared else None
    xd, lg = x.cuda(), torch.from_numpy(logits).cuda()
    out = lay.forward(T, xd, pool, logits=lg, shared_blob=sh).clone()
    torch.cuda.synchronize()
    y_rows = lay.y_rows[:T * k].cpu().numpy()
    ids, w, pos = lay.ids[:T].cpu().numpy(), lay.w[:T].cpu().numpy().astype(np.float64), lay.row_pos[:T * k].cpu().numpy()
    x64 = x.double().numpy()
    ref, allow = np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not t.size:
            continue
        y, al = expert_and_allowance(x64[t], *mats[e])
        check_close(y_rows[pos[t * k + j]], y, what=f"y rows of expert {e}", allow=al)
        ref[t] += w[t, j][:, None] * y
        allow[t] += w[t, j][:, None] * al
    if shared:
        y, al = expert_and_allowance(x64, *mats[E])
        check_close(lay.y_shared[:T].cpu().numpy(), y, what="shared rows", allow=al)
        ref, allow = ref + y, allow + al
    got = formats.bf16_to_f64(out.cpu().numpy().view(np.uint16))
    check_close(got, ref, bf16_out=True, what="layer", allow=allow)
    # the layer call, twice on one workspace, gives the same
    for _ in range(2):
        again = lay.forward_layer(T, xd, pool, logits=lg, shared_blob=sh)
        torch.cuda.synchronize()
        check_close(formats.bf16_to_f64(again.cpu().numpy().view(np.uint16)), ref, bf16_out=True, what="layer call", allow=allow)


@pytest.mark.parametrize("T", [2, 40, 200])
def test_fp8_ffn_stages_slots_and_scratch(ops, T):
    """The two stages in calls of their own, rows of skipped and absent experts, the call without a workspace."""
    k, E, H, I = 3, 8, 256, 272
    rng = np.random.default_rng(T)
    lay, blobs, mats, x, logits = layer_case(rng, T, k, E, H, I, True)
    pool, sh = torch.from_numpy(np.stack(blobs[:E])).cuda(), torch.from_numpy(blobs[E]).cuda()
    xd = x.cuda()
    lay.route_permute(T, logits=torch.from_numpy(logits).cuda())
    lay.ffn(T, xd, pool, shared_blob=sh)
    torch.cuda.synchronize()
    whole, whole_sh = lay.y_rows.clone(), lay.y_shared.clone()
    lay.y_rows.fill_(-3), lay.y_shared.fill_(-3)
    from expert_cached_ffn_amd import _lib
    lay.ffn(T, xd, pool, shared_blob=sh, mode=_lib.FT_FFN_GATE_UP_ONLY)
    torch.cuda.synchronize()
    assert torch.all(lay.y_rows == -3) and torch.all(lay.y_shared == -3)
    lay.ffn(T, xd, pool, shared_blob=sh, mode=_lib.FT_FFN_DOWN_ONLY)
    torch.cuda.synchronize()
    assert torch.equal(lay.y_rows, whole) and torch.equal(lay.y_shared, whole_sh)
    slots = torch.arange(E, dtype=torch.int32, device="cuda")
    slots[1], slots[4], slots[6] = -2, -1, E
    lay.y_rows.fill_(-3)
    lay.ffn(T, xd, pool, slot_of_expert=slots)
    torch.cuda.synchronize()
    off = lay.offsets.cpu().numpy()
    for e in range(E):
        rows = lay.y_rows[off[e]:off[e + 1]]
        if e == 1:
            assert torch.all(rows == -3)
        elif e in (4, 6):
            assert torch.isnan(rows).all()
        else:
            assert torch.equal(rows, whole[off[e]:off[e + 1]])
    lay.y_rows.fill_(-3), lay.y_shared.fill_(-3)
    ops.ft_moe_grouped_ffn_noalloc(lay.layout, pool, None, sh, xd, BF16, T, k, E, lay.offsets, lay.sorted_rows, lay.y_rows,
                                   lay.y_shared)
    torch.cuda.synchronize()
    assert torch.equal(lay.y_rows, whole) and torch.equal(lay.y_shared, whole_sh)


def test_fp8_experts_through_the_cache(ops):
    """Decode steps whose experts come from the pinned bank into cache slots: misses, hits and evictions, then a
    dense FP8 product on the layer's output, as an FP8 model's step runs them."""
    n_layers, T, k, E, H, I, cap = 2, 3, 2, 6, 256, 128, 7
    rng = np.random.default_rng(77)
    lay, _, _, _, _ = layer_case(rng, T, k, E, H, I, False)
    arrays, mats = fp8_experts(rng, n_layers * E, H, I)
    from expert_cached_ffn_amd import layer as L
    eb = int(lay.layout.expert_bytes)
    bank = torch.empty((n_layers * E, eb), dtype=torch.uint8, pin_memory=True)
    for i, a in enumerate(arrays):
        bank[i] = torch.from_numpy(L.pack_expert(lay.layout, a))
    pool = torch.empty((cap, eb), dtype=torch.uint8, device="cuda")
    cache = ops.ExpertCache(lay.layout, n_layers, E, cap, pool, bank, torch.cuda.Stream())
    slots = torch.empty(E, dtype=torch.int32, device="cuda")
    wc, ws = fp8.quantize(rng.standard_normal((200, H)) * 0.1, 128)
    wd, wsd = torch.from_numpy(wc).cuda(), torch.from_numpy(ws.astype(np.float32)).cuda()
    xq, xs = torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty((T, 2), device="cuda")
    head = torch.empty((T, 200), device="cuda")
    for step in range(4):
        for l in range(n_layers):
            x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
            logits = rng.standard_normal((T, E)).astype(np.float32)
            lay.route_permute(T, logits=torch.from_numpy(logits).cuda())
            cache.step(l, lay.ids, T, k, slots)
            xd = x.cuda()
            lay.ffn(T, xd, pool, slot_of_expert=slots)
            lay.combine(T)
            ops.ft_fp8_quantize(lay.out, BF16, H, T, H, 1, xq, H, xs)
            ops.ft_fp8_gemm(xq, H, xs, wd, H, wsd, T, 200, H, F32, head, 200)
            torch.cuda.synchronize()
            ids, w = lay.ids.cpu().numpy(), lay.w.cpu().numpy().astype(np.float64)
            ref, allow = np.zeros((T, H)), np.zeros((T, H))
            for t in range(T):
                for j in range(k):
                    y, al = expert_and_allowance(x[t:t + 1].double().numpy(), *mats[l * E + ids[t, j]])
                    ref[t] += w[t, j] * y[0]
                    allow[t] += w[t, j] * al[0]
            got = formats.bf16_to_f64(lay.out.cpu().numpy().view(np.uint16))
            check_close(got, ref, bf16_out=True, what=f"step {step} layer {l}", allow=allow)
            rc, rs = fp8.quantize(got)
            assert np.array_equal(xq.cpu().numpy(), rc)
            check_product(head, torch.from_numpy(fp8.to_f64(rc, rs)).cuda(), torch.from_numpy(fp8.to_f64(wc, ws, 128)).cuda(), H, F32,
                          False, "head")
    s = cache.stats()
    assert s["hits"] > 0 and s["evictions"] > 0
    cache.destroy()


@pytest.mark.parametrize("T", [1, 5, 40, 300])
def test_replayed_from_a_graph(ops, T):
    """Quantizer, experts, combine and a dense product captured once and replayed, with eager runs between the replays."""
    k, E, H, I = 2, 6, 256, 272
    rng = np.random.default_rng(T)
    lay, blobs, _, x, logits = layer_case(rng, T, k, E, H, I, True)
    pool, sh = torch.from_numpy(np.stack(blobs[:E])).cuda(), torch.from_numpy(blobs[E]).cuda()
    xd, lg = x.cuda(), torch.from_numpy(logits).cuda()
    w, ws = codes_of(gen(1), 300, H), scales_of(gen(2), 3, 2)
    xq, xs = torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty((T, 2), device="cuda")
    head = torch.empty((T, 300), dtype=torch.bfloat16, device="cuda")
    gout = torch.empty((T * k, I), dtype=torch.bfloat16, device="cuda")

    def step():
        out = lay.forward(T, xd, pool, logits=lg, shared_blob=sh)
        ops.ft_fp8_quantize(out, BF16, H, T, H, 1, xq, H, xs)
        ops.ft_fp8_gemm(xq, H, xs, w, H, ws, T, 300, H, BF16, head, 300)
        ops.ft_grouped_gemm(FP8, xq, H, xs, pool, int(lay.layout.expert_bytes), int(lay.layout.off_up), int(lay.layout.off_sup), E,
                            None, T, k, E, lay.offsets, lay.sorted_rows, I, H, BF16, gout, I)
        return out

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        xd.copy_(torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (lay.out[:T], head, gout)]
        for t in (lay.out, head, gout):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (lay.out[:T], head, gout)):
            assert torch.equal(a, b)
