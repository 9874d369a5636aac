"""The FP8 operators with float32 scales per 128 elements, against their
definitions in float64 (plain128).

Tolerances. Quantization is defined bit for bit. The norm's sums are float:
with n columns its y is off by at most (n / 2 + 8) 2^-24 relative (a sum of n
squares, halved by the root, and a handful of roundings), which may move a code
by one step where y sits on a tie, so codes are held to half a step plus that.
The GEMM adds 128 products per K-block in fp32 (the tensor cores' order and
rounding are not specified: 2^-23 per addition), then K / 128 scaled sums.
"""

import numpy as np
import pytest
import torch

import plain128 as P

pytestmark = pytest.mark.gpu

E4M3, E5M2 = 1, 2
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U32 = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def values(rows, cols, dtype, seed, pad=0):
    """Normal values with large rows, large columns, a zero tile and a tile of
    tiny values; `pad` more columns that no call is given."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols + pad, generator=g)
    x[:, :: max(1, cols // 3)] *= 30
    x[:: max(1, rows // 3)] *= 5
    if cols > 128:
        x[rows // 2, :128] = 0
        x[rows // 2, 128:256] *= 1e-6
    return x.to(dtype).cuda()[:, :cols]


SHAPES = [(1, 1), (1, 128), (3, 16), (5, 130), (128, 128), (129, 255), (257, 1000), (7, 4104),
          (1000, 40), (260, 392)]


@pytest.mark.parametrize("direction", ["rows", "cols", "both"])
@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_quantize_equals_the_definition(mx, cuda, shape, block, direction):
    rows, cols = shape
    for i, (dt, fmt, pow2, pad) in enumerate([("bf16", E4M3, False, 0), ("fp16", E5M2, False, 8),
                                              ("fp32", E4M3, True, 3), ("bf16", E5M2, True, 64),
                                              ("fp32", E5M2, False, 4)]):
        x = values(rows, cols, DT[dt], seed=rows + cols + i, pad=pad)
        got = mx.quantize128(x, fmt, block=block, direction=direction, pow2=pow2)
        x64 = f64(x)
        want = ()
        if direction != "cols":
            want += P.quantize(x64, fmt, block, pow2)
        if direction != "rows":
            want += P.quantize(x64.T, fmt, block, pow2)
        assert len(got) == len(want)
        for a, b in zip(got, want):
            a = a.cpu().numpy()
            assert a.shape == b.shape and a.dtype == b.dtype
            assert np.array_equal(a, b), (dt, fmt, pow2)


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("block", [False, True])
def test_quantize_extremes(mx, cuda, fmt, block):
    """NaN and Inf stay in their tile; the largest, the smallest and subnormal
    magnitudes; -0."""
    x = np.ones((256, 384), np.float32)
    x[3, 5] = np.nan
    x[130, 130] = np.inf
    x[131, 300] = -np.inf
    x[10, 128:256] = 3.0e38
    x[11, 128:256] = np.linspace(1e-45, 3e-38, 128)
    x[12, 128:256] = np.linspace(1e-38, 2e-35, 128)     # scales around 2^-126
    x[13, 128:256] = np.linspace(1e-30, 2e-22, 128)     # scales around 2^-80
    x[14, 128:256] = -0.0
    t = torch.from_numpy(x).cuda()
    got = mx.quantize128(t, fmt, block=block, direction="both")
    want = P.quantize(x.astype(np.float64), fmt, block, False) + \
        P.quantize(x.T.astype(np.float64), fmt, block, False)
    for a, b in zip(got, want):
        a = a.cpu().numpy()
        if a.dtype == np.uint8:
            assert np.array_equal(a, b)
        else:
            assert np.array_equal(a, b, equal_nan=True)


def test_quantize_ties(mx, cuda):
    """Every tie of the E4M3 grid under scale 1 goes to the even code."""
    grid = P.decode(np.arange(0x7F, dtype=np.uint8), E4M3)
    mid = (grid[:-1] + grid[1:]) / 2
    x = np.zeros((2, 128), np.float32)
    x[0, :126], x[1, :126] = mid, -mid
    x[:, 127] = 448.0
    codes, scales = mx.quantize128(torch.from_numpy(x).cuda(), E4M3)
    assert np.array_equal(scales.cpu().numpy(), np.ones((2, 1)))
    assert np.array_equal(codes.cpu().numpy(), P.encode(x, E4M3))


@pytest.mark.parametrize("block", [False, True])
def test_quantize_writes_nothing_beyond_its_rows(mx, cuda, block):
    """Into larger buffers of a caller: the padding to 16 codes reads zero, all
    else keeps its bytes."""
    rows, cols = 131, 267
    x = values(rows, cols, torch.bfloat16, 5)
    big, big_t = (torch.full((n + 2, 512), 0xAB, dtype=torch.uint8, device=cuda) for n in (rows, cols))
    if block:
        s, st = torch.full((2, 3), -1.0, device=cuda), torch.full((3, 2), -1.0, device=cuda)
    else:
        held, held_t = torch.full((4, 140), -1.0, device=cuda), torch.full((3, 272), -1.0, device=cuda)
        s, st = held[:3].t()[:rows], held_t[:2].t()[:cols]
    mx.quantize128(x, block=block, direction="both", out=(big[:rows, :cols], s, big_t[:cols, :rows], st))
    want = P.quantize(f64(x), E4M3, block, False) + P.quantize(f64(x).T, E4M3, block, False)
    for held_codes, n, m, codes in ((big, rows, cols, want[0]), (big_t, cols, rows, want[2])):
        b = held_codes.cpu().numpy()
        assert np.array_equal(b[:n, :m], codes)
        end = (m + 15) // 16 * 16
        assert not b[:n, m:end].any() and np.all(b[:n, end:] == 0xAB) and np.all(b[n:] == 0xAB)
    assert np.array_equal(s.cpu().numpy(), want[1]) and np.array_equal(st.cpu().numpy(), want[3])
    if not block:
        assert bool((held[3] == -1).all()) and bool((held[:, 132:] == -1).all())
        assert bool((held_t[2] == -1).all()) and bool((held_t[:, 268:] == -1).all())


# ---------------------------------------------------------------- the norm --

NORM_SHAPES = [(1, 1), (1, 2048), (3, 24), (5, 130), (33, 1000), (2, 4096), (3, 8192), (2, 8200),
               (2, 16384), (2, 16400), (700, 136), (4, 1001)]


def check_codes(codes, scales, y, fmt, pow2):
    """Codes and scales of y (float64) with y off by at most (n/2 + 8) u."""
    n = y.shape[1]
    slack = (n / 2 + 8) * U32
    amax = P.amax_of(y, False)
    s = scales.cpu().numpy().astype(np.float64)
    if pow2:   # one of the two scales that amax (1 +- slack) may ask for
        lo = P.scale_of(amax * (1 - slack), fmt, True)
        hi = P.scale_of(amax * (1 + slack), fmt, True)
        assert np.all((s == lo) | (s == hi))
    else:
        want = np.maximum(amax / P.MAXV[fmt], P.TINY)
        assert np.all(np.abs(s - want) <= (slack + 2 * U32) * want)
    full = P.spread(s, *y.shape, False)
    v = P.decode(codes.cpu().numpy(), fmt) * full
    rel = 2.0 ** -(P.MANT[fmt] + 1)                       # half a step of a normal code
    low = 2.0 ** (P.LOW[fmt] - P.MANT[fmt] - 1) * full    # and of a subnormal one
    assert np.all(np.abs(v - y) <= np.maximum(rel * np.abs(y), low) + (slack + 2 * U32) * 1.1 * np.abs(y))


@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_norm_equals_the_definition(mx, cuda, shape):
    rows, cols = shape
    for i, (dt, fmt, pow2, res, pad) in enumerate([("bf16", E4M3, False, True, 0),
                                                   ("fp16", E5M2, False, False, 8),
                                                   ("fp32", E4M3, True, True, 5),
                                                   ("bf16", E4M3, True, False, 64)]):
        t = DT[dt]
        x = values(rows, cols, t, 7 + i, pad)
        r = values(rows, cols, t, 17 + i) if res else None
        w = (1 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(i))).to(t).cuda()
        codes, scales, h, y = mx.rms_norm_quantize(x, w, r, eps=1e-5, format=fmt, pow2=pow2,
                                                   return_y=True)
        h64, y64 = P.norm(f64(x), None if r is None else f64(r), f64(w), float(np.float32(1e-5)))
        check_codes(codes, scales, y64, fmt, pow2)
        slack = (cols / 2 + 8) * U32
        tiny = torch.finfo(t).tiny if t != torch.float16 else 2.0 ** -25
        assert np.all(np.abs(f64(y) - y64) <= (half_step(t) + slack) * np.abs(y64) + tiny)
        if res:   # one float addition and one rounding
            assert np.all(np.abs(f64(h) - h64) <= (half_step(t) + U32) * np.abs(h64) + tiny)
        else:
            assert h is None


@pytest.mark.parametrize("shape", [(450, 4104), (700, 5120), (320, 6144), (500, 7168), (310, 8184), (500, 1016),
                                   (3000, 1024)], ids=str)
def test_norm_and_gradient_of_wide_rows(mx, cuda, shape):
    """More rows than CTAs at every spread of a wide row over threads."""
    rows, cols = shape
    for i, t in enumerate((torch.bfloat16, torch.float32)):
        x, r, g = (values(rows, cols, t, 77 + 10 * i + j) for j in range(3))
        w = (1 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(i))).to(t).cuda()
        codes, scales, h, _ = mx.rms_norm_quantize(x, w, r, eps=1e-5)
        h64, y64 = P.norm(f64(x), f64(r), f64(w), float(np.float32(1e-5)))
        check_codes(codes, scales, y64, E4M3, False)
        # one float addition and one rounding
        assert np.all(np.abs(f64(h) - h64) <= (half_step(t) + U32) * np.abs(h64) + torch.finfo(t).tiny)
        check_gradient(mx, g, x, w, r)


def test_norm_in_place_and_zero_rows(mx, cuda):
    x, r = values(9, 512, torch.bfloat16, 1), values(9, 512, torch.bfloat16, 2)
    x[4], r[4] = 0, 0
    w = torch.ones(512, device=cuda, dtype=torch.bfloat16)
    want = mx.rms_norm_quantize(x, w, r)
    held = r.clone()
    got = mx.rms_norm_quantize(x, w, held, h_out=held)
    assert got[2] is held
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a, b)
    assert not got[0][4].any() and bool((got[1][4] == P.TINY).all())


def test_norm_nan_stays_in_its_row(mx, cuda):
    x = values(4, 384, torch.float32, 3)
    w = torch.ones(384, device=cuda)
    clean = mx.rms_norm_quantize(x, w)
    x[2, 7] = float("nan")
    codes, scales, _, _ = mx.rms_norm_quantize(x, w)
    assert bool((codes[2] == 0x7F).all()) and bool(torch.isnan(scales[2]).all())
    for i in (0, 1, 3):
        assert torch.equal(codes[i], clean[0][i]) and torch.equal(scales[i], clean[1][i])


# no multiples of 8: every spread of a row over threads, more rows than CTAs
ODD_SHAPES = [(9, 3), (5000, 7), (4801, 241), (5324, 355), (3000, 1001), (2600, 1017), (1, 1019),
              (460, 1027), (600, 1019), (1100, 1030), (900, 3001), (450, 7004), (300, 9001),
              (200, 16369), (170, 16371), (50, 4099)]


def check_gradient(mx, g, h, w, gr):
    (rows, cols), t = h.shape, h.dtype
    gh, gw = mx.rms_norm_bwd(g, h, w, eps=1e-5, grad_residual=gr)
    eps = float(np.float32(1e-5))
    want, want_w = P.norm_bwd(f64(g), f64(h), f64(w), eps, None if gr is None else f64(gr))
    # each term of the sum, by its magnitude: n / 2 + 8 roundings of r, the
    # mean's n more
    h64, gw64 = f64(h), f64(g) * f64(w)
    r = 1 / np.sqrt((h64 * h64).mean(1, keepdims=True) + eps)
    n = np.abs(h64 * r)
    mag = r * (np.abs(gw64) + n * (np.abs(gw64) * n).mean(1, keepdims=True))
    err = (2 * cols + 16) * U32 * mag
    tiny = torch.finfo(t).tiny if t != torch.float16 else 2.0 ** -25
    assert np.all(np.abs(f64(gh) - want) <= half_step(t) * np.abs(want) + (1 + 2 ** -8) * err + tiny)
    mag_w = (np.abs(f64(g)) * n).sum(0)
    assert np.all(np.abs(f64(gw) - want_w) <= (cols / 2 + rows + 16) * U32 * mag_w)
    return gh, gw


@pytest.mark.parametrize("shape", NORM_SHAPES + [(1500, 64), (333, 2048)] + ODD_SHAPES, ids=str)
def test_norm_gradient_equals_the_formula(mx, cuda, shape):
    rows, cols = shape
    for i, (dt, res) in enumerate([("bf16", True), ("fp16", False), ("fp32", True)]):
        t = DT[dt]
        h, g = values(rows, cols, t, 27 + i), values(rows, cols, t, 37 + i)
        gr = values(rows, cols, t, 47 + i) if res else None
        w = (1 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(i))).to(t).cuda()
        gh, gw = check_gradient(mx, g, h, w, gr)
        # the same call gives the same bits, and works in place
        again = mx.rms_norm_bwd(g, h, w, eps=1e-5, grad_residual=gr)
        assert torch.equal(again[0], gh) and torch.equal(again[1], gw)
        held = g.clone()
        got = mx.rms_norm_bwd(held, h, w, eps=1e-5, grad_residual=gr, out=held)
        assert torch.equal(got[0], gh) and torch.equal(got[1], gw)


@pytest.mark.parametrize("shape", [(70, 131), (33, 3000), (700, 5001), (3, 16392)], ids=str)
def test_norm_gradient_of_unaligned_tensors(mx, cuda, shape):
    """Tensors that start at any element, each at another."""
    rows, cols = shape
    for t in (torch.bfloat16, torch.float32):
        g, h, gr = (torch.empty(rows * cols + 8, dtype=t, device=cuda)[i:i + rows * cols].view(rows, cols)
                    .copy_(values(rows, cols, t, 57 + i)) for i in (1, 2, 3))
        w = torch.ones(cols + 1, dtype=t, device=cuda)[1:]
        check_gradient(mx, g, h, w, gr)
        check_gradient(mx, values(rows, cols, t, 61), values(rows, cols, t, 62), w, None)


@pytest.mark.parametrize("shape", [(2, 1), (2, 2), (4, 3), (3, 5), (5, 3), (1, 7), (700, 1), (1300, 5)], ids=str)
def test_norm_gradient_of_few_columns(mx, cuda, shape):
    """Rows shorter than a vector of 8, several of which share the tensors' last,
    incomplete one; tensors that end with their storage."""
    rows, cols = shape
    for t in (torch.bfloat16, torch.float16, torch.float32):
        def at_end(seed):
            held = torch.full((rows * cols + 8,), float("nan"), dtype=t, device=cuda)
            return held[8:].view(rows, cols).copy_(values(rows, cols, t, seed))
        g, h, gr = (at_end(71 + i) for i in range(3))
        w = (1 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(5))).to(t).cuda()
        check_gradient(mx, g, h, w, None)
        gh, gw = check_gradient(mx, g, h, w, gr)
        got = mx.rms_norm_bwd(g, h, w, eps=1e-5, grad_residual=gr, out=gr)
        assert torch.equal(got[0], gh) and torch.equal(got[1], gw)


@pytest.mark.parametrize("cols", [3, 131, 355, 1001, 2003, 9001])
def test_norm_gradient_nan_stays_in_its_row(mx, cuda, cols):
    """Rows that share 16 bytes with one that holds NaN or Inf."""
    for t in (torch.bfloat16, torch.float32):
        g, h, gr = (values(20, cols, t, 67 + i) for i in range(3))
        w = torch.ones(cols, dtype=t, device=cuda)
        clean = mx.rms_norm_bwd(g, h, w, grad_residual=gr)[0]
        for x in (g, h, gr):
            x[3], x[10] = float("nan"), float("inf")
        got = mx.rms_norm_bwd(g, h, w, grad_residual=gr)[0]
        rest = [i for i in range(20) if i not in (3, 10)]
        assert torch.isnan(got[[3, 10]]).all() and torch.equal(got[rest], clean[rest])


# ---------------------------------------------------------------- the GEMM --

def operand(rows, K, fmt, block, seed):
    """Codes and scales in the quantizers' layouts, and the float64 values."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)).astype(np.float32)
    x[:: max(1, rows // 5)] *= 20
    codes, s = P.quantize(x.astype(np.float64), fmt, block, False)
    held = torch.full((rows, (K + 15) // 16 * 16), 0xFF, dtype=torch.uint8)   # padding: NaN codes
    held[:, :K] = torch.from_numpy(codes)
    held = held.cuda()[:, :K]
    st = torch.from_numpy(s).cuda()
    if not block:
        nb = s.shape[1]
        laid = torch.full((nb, (rows + 3) // 4 * 4), float("nan"), device="cuda")
        laid[:, :rows] = st.t()
        st = laid.t()[:rows]
    v = P.decode(codes, fmt) * P.spread(s, rows, K, block)
    return (held, st), v


GEMM_SHAPES = [(1, 128, 128), (1, 1, 1), (7, 130, 96), (16, 1536, 2048), (17, 392, 640), (33, 264, 1000),
               (64, 512, 4096), (65, 200, 384), (100, 72, 257), (128, 1024, 2048), (200, 2056, 512),
               (300, 520, 1111), (1, 2048, 4100), (1500, 129, 128), (2200, 2056, 256),
               (129, 4096, 128), (3, 5, 7000), (2563, 2056, 1500),
               (4099, 1030, 640), (1024, 4872, 1024),
               # every tile width and orientation, with K split 1, 2, 4 and 8 ways
               (1, 32, 1289), (2, 33, 1168), (129, 4968, 84), (135, 160, 2563), (257, 149, 3686),
               (265, 336, 4927), (284, 135, 2597), (292, 399, 1697), (340, 386, 1466), (397, 264, 1831),
               (548, 949, 3685), (685, 343, 3379), (775, 283, 2005), (900, 3656, 78), (1265, 536, 5790),
               (1329, 1916, 5019), (1860, 1245, 424), (2838, 1865, 4884),
               (288, 16, 6143), (1201, 17, 2623), (2054, 16, 2489), (33, 1467, 6685), (2417, 70, 3183),
               (1431, 133, 7695), (1200, 21, 2222), (2808, 17, 1969), (2856, 138, 399),
               (2564, 132, 520), (697, 145, 7973), (37, 4784, 5026), (72, 5302, 7758),
               (137, 5359, 7915)]


@pytest.mark.parametrize("block", [True, False])
@pytest.mark.parametrize("shape", GEMM_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_gemm_equals_the_definition(mx, cuda, shape, block):
    M, N, K = shape
    fmts = [(E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2)][(M + N + K) % 3]
    a, av = operand(M, K, fmts[0], False, 1)
    b, bv = operand(N, K, fmts[1], block, 2)
    want = av @ bv.T
    mag = np.abs(av) @ np.abs(bv).T
    err = (128 * 2 * U32 + (-(-K // 128) + 12) * U32) * mag   # (+ 8 of a split's sums, 2 of scales)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    for out_dtype in (torch.float32, torch.bfloat16):
        out = torch.full((M, N), float("nan"), dtype=out_dtype, device=cuda)
        d = mx.gemm128(*a, *b, a_format=fmts[0], b_format=fmts[1], out_dtype=out_dtype, out=out,
                       status=status)
        assert d is out
        tol = err + half_step(out_dtype) * (np.abs(want) + err)
        assert np.all(np.abs(f64(d) - want) <= tol)
        again = mx.gemm128(*a, *b, a_format=fmts[0], b_format=fmts[1], out_dtype=out_dtype)
        assert torch.equal(again, d)
    assert status.item() == 0


@pytest.mark.parametrize("shape", [(5, 200, 300), (130, 140, 512), (600, 700, 260)], ids=str)
@pytest.mark.parametrize("block", [True, False])
def test_gemm_of_integers_is_exact(mx, cuda, shape, block):
    """Small integers under power-of-two scales: every partial sum is exact, in
    any order, so the product is."""
    M, N, K = shape
    rng = np.random.default_rng(3)
    sides = []
    for rows, blk in ((M, False), (N, block)):
        v = rng.integers(-8, 9, (rows, K)).astype(np.float64)
        codes = P.encode(v, E4M3)
        held = torch.zeros(rows, (K + 15) // 16 * 16, dtype=torch.uint8)
        held[:, :K] = torch.from_numpy(codes)
        nb = (K + 127) // 128
        s = 2.0 ** rng.integers(-2, 3, ((rows + 127) // 128 if blk else rows, nb))
        st = torch.from_numpy(s).float().cuda()
        if not blk:
            laid = torch.zeros(nb, (rows + 3) // 4 * 4, device="cuda")
            laid[:, :rows] = st.t()
            st = laid.t()[:rows]
        sides.append(((held.cuda()[:, :K], st), v * P.spread(s, rows, K, blk)))
    (a, av), (b, bv) = sides
    d = mx.gemm128(*a, *b, out_dtype=torch.float32)
    assert np.array_equal(f64(d), av @ bv.T)


@pytest.mark.parametrize("shape", [(8, 136), (300, 520)], ids=str)
@pytest.mark.parametrize("block", [True, False])
def test_gemm_scale_products_round_to_float(mx, cuda, shape, block):
    """One K-block of small integers, whose sum is exact, under scales from 2^-126
    to 2^100: every value is that sum times the scales' product rounded to float
    (2^-126 and more: its own rounding alone), rounded once."""
    M, N = shape
    K = 128
    rng = np.random.default_rng(9)
    a, b = (rng.integers(-8, 9, (n, K)).astype(np.float64) for n in (M, N))
    sa = np.float32(rng.uniform(1, 2, M) * 2.0 ** rng.integers(-126, 101, M))
    sb = np.float32(rng.uniform(1, 2, N) * 2.0 ** rng.integers(-126, 101, N))
    if block:
        sb = np.repeat(np.float32([1.7 * 2.0 ** 90, 1.3 * 2.0 ** -80, 1.1 * 2.0 ** -20] * 2), 128)[:N]
    scales = [torch.from_numpy(sa).cuda().view(M, 1),
              torch.from_numpy(sb[::128].copy() if block else sb).cuda().view(-1, 1)]
    codes = [torch.from_numpy(P.encode(v, E4M3)).cuda() for v in (a, b)]
    d = mx.gemm128(codes[0], scales[0], codes[1], scales[1], out_dtype=torch.float32).cpu().numpy()
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        p = sa[:, None] * sb[None]
        want = np.float32(p.astype(np.float64) * (a @ b.T))
    assert p.dtype == np.float32 and np.any((p < 2.0 ** -126) & (p > 0)) and np.isinf(p).any()
    assert np.array_equal(d, want, equal_nan=True)


def test_gemm_nan_scale_reaches_its_row_alone(mx, cuda):
    for M in (8, 300):
        x = torch.randn(M, 512, device=cuda)
        w = torch.randn(256, 512, device=cuda)
        x[5, 200] = float("inf")
        d = mx.gemm128(*mx.quantize128(x), *mx.quantize128(w, block=True))
        bad = torch.isnan(d).all(1)
        assert bad.nonzero().flatten().tolist() == [5] and bool(torch.isfinite(d[:5]).all())


@pytest.mark.parametrize("rows", [(0, 5, 0, 130), (128, 300, 256, 200), (256, 700, 128, 600)], ids=str)
def test_gemm_of_slices_of_larger_operands(mx, cuda, rows):
    """Rows and K-blocks of larger codes and scales give what copies of them give:
    pitches beyond the least, and other codes behind a row's end."""
    a0, M, b0, N = rows
    a = mx.quantize128(torch.randn(1000, 1280, device=cuda))
    b = mx.quantize128(torch.randn(900, 1280, device=cuda))
    bb = mx.quantize128(torch.randn(900, 1280, device=cuda), block=True)

    def copied(codes, scales, block):
        n, k = codes.shape
        held = torch.full((n, (k + 15) // 16 * 16), 0x7F, dtype=torch.uint8, device=cuda)
        held[:, :k] = codes
        if block:
            return held[:, :k], scales.clone()
        laid = torch.full((scales.shape[1], (n + 3) // 4 * 4), float("nan"), device=cuda)
        laid[:, :n] = scales.t()
        return held[:, :k], laid.t()[:n]

    for k0, k1 in ((0, 1280), (256, 1280), (128, 901)):
        t0, t1 = k0 // 128, (k1 + 127) // 128
        sa = a[0][a0:a0 + M, k0:k1], a[1][a0:a0 + M, t0:t1]
        sides = [(b[0][b0:b0 + N, k0:k1], b[1][b0:b0 + N, t0:t1], False)]
        if k0 == 0:
            blocks = bb[1][b0 // 128:(b0 + N + 127) // 128, :t1]
            sides.append((bb[0][b0:b0 + N, :k1], blocks, True))
        for cb, scb, block in sides:
            got = mx.gemm128(*sa, cb, scb)
            assert torch.isfinite(got).all()
            assert torch.equal(got, mx.gemm128(*copied(*sa, False), *copied(cb, scb, block)))


def test_gemm_empty(mx, cuda):
    a = mx.quantize128(torch.randn(5, 256, device=cuda))
    none = torch.empty(0, 256, dtype=torch.uint8, device=cuda)
    d = mx.gemm128(*a, none, torch.empty(0, 2, device=cuda))
    assert d.shape == (5, 0)
    z = mx.gemm128(torch.empty(5, 0, dtype=torch.uint8, device=cuda), torch.empty(5, 0, device=cuda),
                   torch.empty(7, 0, dtype=torch.uint8, device=cuda), torch.empty(1, 0, device=cuda))
    assert z.shape == (5, 7) and not z.any()
    assert mx.quantize128(torch.empty(0, 256, device=cuda))[0].shape == (0, 256)
    gh, gw = mx.rms_norm_bwd(*[torch.empty(0, 64, device=cuda)] * 2, torch.ones(64, device=cuda))
    assert gh.shape == (0, 64) and not gw.any()


# ------------------------------------------------------- together, as used --

def layer_inputs(T, K, N, seed=0):
    g = torch.Generator().manual_seed(seed)
    x, r = torch.randn(T, K, generator=g), torch.randn(T, K, generator=g)
    nw = 1 + 0.1 * torch.randn(K, generator=g)
    w = torch.randn(N, K, generator=g) * K ** -0.5
    return [t.bfloat16().cuda() for t in (x, r, nw, w)]


@pytest.mark.parametrize("T,K,N", [(1, 256, 384), (100, 392, 520), (1037, 1024, 640)])
def test_norm_linear_forward_and_backward(mx, cuda, T, K, N):
    """A pre-norm linear layer's two passes are the operators run one after the
    other: every gradient equals, bit for bit, what the operators give, and
    lies near the float64 layer's (FP8's half step of 2^-4 per operand; the
    errors of K products average out)."""
    x, r, nw, w = [t.requires_grad_() for t in layer_inputs(T, K, N)]
    y, h = mx.rms_norm_linear128(x, nw, w, residual=r)
    gy, gh_in = torch.randn_like(y), torch.randn_like(h)
    torch.autograd.backward([y, h], [gy, gh_in])
    with torch.no_grad():
        c, s, h2, n = mx.rms_norm_quantize(x, nw, r, return_y=True)
        wq = mx.quantize128(w, block=True, direction="both")
        assert torch.equal(h, h2) and torch.equal(y, mx.gemm128(c, s, wq[0], wq[1]))
        g = mx.quantize128(gy, direction="both")
        gn = mx.gemm128(g[0], g[1], wq[2], wq[3])
        gw = mx.gemm128(g[2], g[3], *mx.quantize128(n, direction="cols"), out_dtype=torch.float32)
        gh, gnw = mx.rms_norm_bwd(gn, h2, nw, grad_residual=gh_in)
        assert torch.equal(w.grad, gw.bfloat16()) and torch.equal(nw.grad, gnw.bfloat16())
        assert torch.equal(x.grad, gh) and torch.equal(r.grad, gh)
    n64 = P.norm(f64(x), f64(r), f64(nw), 1e-6)
    gn64 = f64(gy) @ f64(w)
    wants = [(y, n64[1] @ f64(w).T), (w.grad, f64(gy).T @ n64[1])]
    wants += list(zip((x.grad, nw.grad), P.norm_bwd(gn64, n64[0], f64(nw), 1e-6, f64(gh_in))))
    for got, want in wants:
        # two operands, each off by at most 2^-4 of its value, uncorrelated
        assert np.linalg.norm(f64(got) - want) <= 2 * 2.0 ** -4 * np.linalg.norm(want)


def test_norm_linear_gradients_accumulate_apart(mx, cuda):
    """Two backward passes into the same leaves of three dimensions: twice one
    pass's gradient (exactly: a doubling), in memory of their own."""
    x, r, nw, w = layer_inputs(60, 256, 136)
    x, r = (t.view(4, 15, 256).requires_grad_() for t in (x, r))
    nw.requires_grad_(), w.requires_grad_()
    gy, gh = (torch.randn(4, 15, n, device=cuda).bfloat16() for n in (136, 256))
    once = torch.autograd.grad(mx.rms_norm_linear128(x, nw, w, residual=r), (x, r, nw, w), (gy, gh))
    for _ in range(2):
        torch.autograd.backward(mx.rms_norm_linear128(x, nw, w, residual=r), (gy, gh))
    for t, g in zip((x, r, nw, w), once):
        assert torch.equal(t.grad, 2 * g)
    assert x.grad.untyped_storage().data_ptr() != r.grad.untyped_storage().data_ptr()


def test_linear_gradients_by_what_is_asked(mx, cuda):
    x, _, _, w = layer_inputs(70, 256, 136)
    gy = torch.randn(2, 35, 136, device=cuda).bfloat16()
    both = [x.clone().requires_grad_(), w.clone().requires_grad_()]
    y = mx.linear128(both[0].view(2, 35, 256), both[1], grad_format=E5M2)
    y.backward(gy)
    for i in (0, 1):
        one = [t.clone().requires_grad_(i == j) for j, t in enumerate((x, w))]
        mx.linear128(one[0].view(2, 35, 256), one[1], grad_format=E5M2).backward(gy)
        assert torch.equal(one[i].grad, both[i].grad) and one[1 - i].grad is None
    # no residual: h is x itself, and the norm's gradient reaches it alone
    z = x.clone().requires_grad_()
    nw = torch.ones(256, device=cuda, dtype=torch.bfloat16)
    out, h = mx.rms_norm_linear128(z, nw, w)
    assert h is z
    out.backward(gy.view(70, 136))
    assert torch.isfinite(z.grad).all()


def test_layer_in_a_graph_and_on_another_stream(mx, cuda):
    """The forward pass captured once and replayed on new inputs, twice, equals
    eager calls; two captured graphs with buffers of their own do not meet."""
    x, r, nw, w = layer_inputs(48, 512, 640)
    wc, ws = mx.quantize128(w, block=True)
    sx, sr = x.clone(), r.clone()

    def step(a, b):
        c, s, h, _ = mx.rms_norm_quantize(a, nw, b)
        return mx.gemm128(c, s, wc, ws), h

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(sx, sr)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step(sx, sr)))
    for seed in (1, 2):
        x2, r2, _, _ = layer_inputs(48, 512, 640, seed)
        sx.copy_(x2)
        sr.copy_(r2)
        want = step(x2, r2)
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, out in graphs:
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        got = step(x, r)
    side.synchronize()
    want = step(x, r)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_training_step_in_a_graph(mx, cuda):
    """Both layers' forward and backward pass captured once; replays on new inputs
    give what eager passes give."""
    x, r, nw, w = layer_inputs(96, 512, 512)
    leaves = [t.clone().requires_grad_() for t in (x, r, nw, w)]
    gy = torch.randn(96, 512, device=cuda).bfloat16()

    def step(lx, lr, lnw, lw):
        y, h = mx.rms_norm_linear128(lx, lnw, lw, residual=lr)
        z = mx.linear128(y, lw, grad_format=E5M2)
        return torch.autograd.grad([z, h], [lx, lr, lnw, lw], [gy, gy])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*leaves)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*leaves)
    for seed in (0, 3):
        new = layer_inputs(96, 512, 512, seed)
        with torch.no_grad():
            for t, n in zip(leaves, new):
                t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step(*(n.requires_grad_() for n in new))):
            assert torch.equal(a, b)


def test_norm_gradient_in_a_graph(mx, cuda):
    h, g = values(300, 512, torch.bfloat16, 1), values(300, 512, torch.bfloat16, 2)
    w = torch.ones(512, device=cuda, dtype=torch.bfloat16)
    want = mx.rms_norm_bwd(g, h, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mx.rms_norm_bwd(g, h, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = mx.rms_norm_bwd(g, h, w)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_both_marshalling_paths_give_the_same(mx, cuda):
    """The C++ module makes the plain calls, Python those with buffers of the
    caller's: same tensors, layouts included. An unusual call is left to Python."""
    from fp8_quantization_mx_b200 import ops128
    x, r = values(130, 300, torch.bfloat16, 1), values(130, 300, torch.bfloat16, 2)
    w = torch.ones(300, device=cuda, dtype=torch.bfloat16)
    wq = mx.quantize128(values(200, 300, torch.bfloat16, 3), block=True)
    calls = [lambda: mx.quantize128(x, E5M2, direction="both", pow2=True),
             lambda: mx.quantize128(x, block=True, direction="cols"),
             lambda: mx.rms_norm_quantize(x, w, r, return_y=True), lambda: mx.rms_norm_quantize(x, w),
             lambda: mx.rms_norm_bwd(x, r, w, grad_residual=x),
             lambda: mx.gemm128(*mx.quantize128(x), *wq, out_dtype=torch.float32)]
    assert ops128._fast or ops128._bind_fast()
    fast, was = [c() for c in calls], ops128._fast
    try:
        ops128._fast = False
        slow = [c() for c in calls]
    finally:
        ops128._fast = was
    for a, b in zip(fast, slow):
        for s, t in zip(a if isinstance(a, tuple) else (a,), b if isinstance(b, tuple) else (b,)):
            assert (s is None) == (t is None)
            if s is not None:
                assert torch.equal(s, t) and s.stride() == t.stride() and s.dtype == t.dtype
    assert was.quantize(x.double(), E4M3, False, 1, False) is None
    assert was.gemm(x, x, x, x, E4M3, E4M3, False) is None
    assert was.norm(x, w[:299], None, 1e-6, E4M3, False, False) is None
    assert was.norm(x, w, None, "eps", E4M3, False, False) is None
    assert was.norm(x, w, None, -1.0, E4M3, False, False) == 1       # the library's refusal
    with pytest.raises(mx.MXError):
        mx.rms_norm_quantize(x, w, eps=-1.0)


def test_tensor_layer_refuses(mx, cuda):
    x, w = torch.zeros(8, 256, device=cuda), torch.zeros(256, device=cuda)
    c, s = mx.quantize128(x)
    bad = [
        (lambda: mx.quantize128(x.double()), "bfloat16"), (lambda: mx.quantize128(x[0]), "rows, cols"),
        (lambda: mx.quantize128(x.t()), "contiguous rows"), (lambda: mx.quantize128(x, 0), "E4M3"),
        (lambda: mx.quantize128(x, direction="up"), "direction"),
        (lambda: mx.quantize128(x.expand(8, 256)[:1].expand(8, 256)), "overlapping"),
        (lambda: mx.quantize128(x, out=(c,)), "2 tensors"),
        (lambda: mx.quantize128(x, out=(c[:, :128], s)), "must be"),
        (lambda: mx.quantize128(x, out=(c, s.contiguous())), "tile by tile"),
        (lambda: mx.quantize128(x, out=(torch.zeros(8, 256, device=cuda), s)), "uint8"),
        (lambda: mx.quantize128(x[:, :250], out=(torch.empty(8, 250, dtype=torch.uint8, device=cuda), s)),
         "16 bytes apart"),
        (lambda: mx.rms_norm_quantize(x, w.bfloat16()), "weight"), (lambda: mx.rms_norm_quantize(x, w[:5]), "weight"),
        (lambda: mx.rms_norm_quantize(x, w, x[:4]), "residual"), (lambda: mx.rms_norm_quantize(x, w, h_out=x), "h_out"),
        (lambda: mx.rms_norm_bwd(x, x.t().contiguous().t(), w), "contiguous"),
        (lambda: mx.rms_norm_bwd(None, x, w), "grad_y"), (lambda: mx.rms_norm_bwd(x, x, w, grad_residual=x[:4]), "grad_residual"),
        (lambda: mx.gemm128(c, s, c[:, :128], s), "b_codes"), (lambda: mx.gemm128(c, s.contiguous(), c, s), "a_scales"),
        (lambda: mx.gemm128(c, s, c, s[:4]), "b_scales"), (lambda: mx.gemm128(c, s, c, s, a_format=3), "a_format"),
        (lambda: mx.gemm128(c, s, c, s, out_dtype=torch.float16), "out_dtype"),
        (lambda: mx.gemm128(c, s, c, s, out=torch.empty(8, 9, device=cuda)), "out"),
        (lambda: mx.gemm128(c, s, c, s, status=torch.zeros(1, device=cuda)), "status"),
        # a view whose last row's padding lies outside the storage
        (lambda: mx.gemm128(c.view(-1)[:2040].as_strided((8, 250), (256, 1), 6), s, c, s), "outside its storage"),
    ]
    for call, words in bad:
        with pytest.raises(ValueError, match=words):
            call()


def test_lazily_negated_tensors_are_refused(mx, cuda):
    """The imaginary part of a conjugate is a view of the positive values that
    torch negates where it reads them; the kernels would not."""
    x = torch.randn(5, 1, dtype=torch.complex64, device=cuda).conj().imag
    plain, w = x.resolve_neg(), torch.ones(1, device=cuda)
    assert x.is_neg() and torch.equal(x, plain) and not plain.is_neg()
    one = torch._neg_view(torch.ones(1, 1, device=cuda))
    for call in (lambda: mx.quantize128(x), lambda: mx.rms_norm_quantize(x, w),
                 lambda: mx.rms_norm_quantize(plain[:1], w, one), lambda: mx.rms_norm_bwd(one, one, w),
                 lambda: mx.rms_norm_bwd(one.resolve_neg(), one.resolve_neg(), w, grad_residual=one)):
        with pytest.raises(ValueError, match="resolve_neg"):
            call()
    codes, scales = mx.quantize128(one.resolve_neg())
    with pytest.raises(ValueError, match="resolve_neg"):
        mx.gemm128(codes, torch._neg_view(scales), codes, scales)
    assert torch.equal(mx.quantize128(plain)[0] >> 7, (plain < 0).byte())


def test_layers_without_tokens_and_of_one_dimension(mx, cuda):
    _, _, nw, w = layer_inputs(1, 256, 136)
    w.requires_grad_()
    x = torch.empty(0, 256, device=cuda, dtype=torch.bfloat16, requires_grad=True)
    y, h = mx.rms_norm_linear128(x, nw, w)
    (mx.linear128(x, w).sum() + y.sum()).backward()
    assert y.shape == (0, 136) and x.grad.shape == (0, 256) and not w.grad.any()
    one = layer_inputs(1, 256, 136)[0]
    assert torch.equal(mx.linear128(one[0], w), mx.linear128(one, w)[0])


def test_layers_refuse(mx, cuda):
    x, r, nw, w = layer_inputs(4, 256, 136)
    for call in (lambda: mx.linear128(x.float(), w), lambda: mx.linear128(x, w.float()),
                 lambda: mx.linear128(x, w[:, :128]), lambda: mx.rms_norm_linear128(x, nw.float(), w),
                 lambda: mx.rms_norm_linear128(x, nw, w, residual=r[:2]),
                 lambda: mx.rms_norm_linear128(x, nw, w, residual=r.float())):
        with pytest.raises(ValueError):
            call()


def test_norm_in_place_of_x(mx, cuda):
    for cols in (512, 509, 8200):
        x, r = values(9, cols, torch.float16, 1), values(9, cols, torch.float16, 2)
        x = x.contiguous()
        w = torch.ones(cols, device=cuda, dtype=torch.float16)
        want = mx.rms_norm_quantize(x, w, r)
        got = mx.rms_norm_quantize(x, w, r, h_out=x)
        for a, b in zip(got[:3], want[:3]):
            assert torch.equal(a, b)


def test_calls_on_two_streams_at_once(mx, cuda):
    """Nothing is shared between calls: two streams at once give what each gives
    alone, many times over."""
    x, r, nw, w = layer_inputs(300, 1024, 1536)
    wq = mx.quantize128(w, block=True)

    def work(a, b):
        c, s, h, _ = mx.rms_norm_quantize(a, nw, b)
        return mx.gemm128(c, s, *wq), *mx.rms_norm_bwd(a, h, nw), *mx.quantize128(a, direction="both")

    want = [work(x, r), work(r, x)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, (a, b) in enumerate(((x, r), (r, x))):
            with torch.cuda.stream(streams[i]):
                got[i].append(work(a, b))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_offsets_beyond_32_bits(mx, cuda):
    """2.3e9 elements: the last rows come out as they do alone."""
    rows, cols, tail = 70016, 32768, 128
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=cuda)
    g = torch.Generator(device=cuda).manual_seed(0)
    for i in range(0, rows, 4376):
        x[i:i + 4376] = torch.randn(4376, cols, generator=g, device=cuda)
    w = torch.ones(cols, device=cuda, dtype=torch.bfloat16)
    last = x[-tail:].clone()
    c, s, ct, st = mx.quantize128(x, direction="both")
    lc, ls, lct, lst = mx.quantize128(last, direction="both")
    assert torch.equal(c[-tail:], lc) and torch.equal(s[-tail:], ls)
    assert torch.equal(ct[:, -tail:], lct) and torch.equal(st[:, -1:], lst)
    b = mx.quantize128(last[:40], block=True)
    d = mx.gemm128(c, s, *b, out_dtype=torch.float32)
    v = [P.decode(q.cpu().numpy(), E4M3) * P.spread(z.cpu().numpy(), q.shape[0], cols, k)
         for q, z, k in ((lc, ls, False), (*b, True))]
    mag = np.abs(v[0]) @ np.abs(v[1]).T
    assert np.all(np.abs(f64(d[-tail:]) - v[0] @ v[1].T) <= (256 + cols / 128 + 12) * U32 * mag)
    del ct, st, d
    nc, ns, h, _ = mx.rms_norm_quantize(x, w, x)
    mc, ms, mh, _ = mx.rms_norm_quantize(last, w, last)
    assert torch.equal(nc[-tail:], mc) and torch.equal(ns[-tail:], ms) and torch.equal(h[-tail:], mh)
    del nc, ns, c, s
    gh, _ = mx.rms_norm_bwd(x, h, w)
    assert torch.equal(gh[-tail:], mx.rms_norm_bwd(last, mh, w)[0])


def test_padding_of_rows_is_zero_or_nan(mx, cuda):
    """Past cols a row's codes are zeros up to a multiple of 16, and NaN where
    the row's last tile holds one."""
    for cols in (24, 20):   # the norm's two kinds of kernels
        x = values(40, cols, torch.bfloat16, 5)
        x[3, 1] = float("nan")
        x[5] = 0.0
        x = x.to(cuda)
        for codes in (mx.quantize128(x)[0], mx.quantize128(x, direction="both")[0],
                      mx.rms_norm_quantize(x, torch.ones_like(x[0]), eps=0.0)[0]):
            pad = codes.as_strided((40, 32 - cols), (32, 1), cols).cpu()
            bad = codes[:, 0].cpu() == 0x7F
            assert bad[3] and bad.sum() <= 2
            assert (pad[bad] == 0x7F).all() and (pad[~bad] == 0).all()


def test_layers_without_gradients_keep_nothing(mx, cuda, monkeypatch):
    """Under no_grad the layers make no transposed operands, whatever their
    inputs require; the results are the same."""
    from fp8_quantization_mx_b200 import ops128
    x, r, nw, w = [t.requires_grad_() for t in layer_inputs(64, 256, 384)]
    y, (z, h) = mx.linear128(x, w), mx.rms_norm_linear128(x, nw, w, r)
    made, quantize = [], ops128.quantize128
    monkeypatch.setattr(ops128, "quantize128",
                        lambda *a, direction="rows", **k: (made.append(direction),
                                                           quantize(*a, direction=direction, **k))[1])
    with torch.no_grad():
        y0, (z0, h0) = mx.linear128(x, w), mx.rms_norm_linear128(x, nw, w, r)
    assert made == ["rows"] * 3
    assert torch.equal(y, y0) and torch.equal(z, z0) and torch.equal(h, h0)
    assert not (y0.requires_grad or z0.requires_grad or h0.requires_grad)
