"""The token operators against their definitions in 64 bits.

u = 2^-24 is one rounding in 32 bits.  Tolerances, each a count of roundings:
 - norm: h is one rounding; a row's sum of squares is a tree whose longest
   chain is CHAIN(cols) additions (a thread's own values, then 10 across the
   block), halved by the root; division, eps, root and two products add 5.
 - 8 bits: q is reproduced bit for bit in 32 bits on the CPU; the scale takes
   the norm's roundings and two more.
 - product: the sum is exact; its conversion, the scales' product and the
   product with it are 3 roundings of the product term, the bias and the
   residual one each of the running sum.
The last rounding is half a step of the output's type.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-45, torch.bfloat16: 1e-40, torch.float16: 2.0 ** -25}
ALL = [torch.float32, torch.bfloat16, torch.float16]


def CHAIN(cols):
    return max(64, cols // 1024 + 1) + 10


@pytest.fixture(scope="module")
def nat():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from bigvgan_waveform_decoder_alias_b200 import build_native, native
    build_native.build()
    native.lib()
    return native


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def close(got, want, tol):
    """|got - want| <= tol, elementwise; not-finite values must agree."""
    got, want = got.double(), want.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
    over = ((got - want).abs() - tol)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, f"over the tolerance by {float(over.max())}"


def norm64(x, residual, gain, eps):
    h = x.double() if residual is None else x.double() + residual.double()
    rstd = 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    return h, rstd, h * rstd * (1.0 if gain is None else gain.double())


def check_norm(x, residual, gain, eps, y, h):
    h64, _, y64 = norm64(x, residual, gain, eps)
    rel = (CHAIN(x.shape[-1]) / 2 + 8) * U
    close(y, y64, y64.abs() * (HALF[x.dtype] + rel) * 1.001 + TINY[x.dtype])
    if h is not None:
        close(h, h64, h64.abs() * (HALF[x.dtype] + U) * 1.001 + TINY[x.dtype])


def expected_q(x, residual, gain):
    """q bit for bit: single 32-bit operations on the CPU."""
    h = x.float().cpu().numpy()
    if residual is not None:
        h = h + residual.float().cpu().numpy()
    t = h if gain is None else (h * gain.float().cpu().numpy()).astype(np.float32)
    a = np.abs(t).max(-1, keepdims=True).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint(t * (np.float32(127.0) / a).astype(np.float32))
    return np.where(a > 0, q, 0).astype(np.int8), a[..., 0]


SIZES = [(1, 1), (1, 8), (3, 7), (2, 32), (5, 127), (4, 128), (3, 255), (2, 1000), (7, 1024),
         (1, 1537), (3, 2048), (2, 2056), (5, 4096), (1, 8192), (2, 8200), (3, 11000),
         (1, 16384), (2, 16392), (1, 20001), (2, 32768), (1, 32776), (2, 70000),
         # enough rows for every SM: through the ring of the persistent kernel
         (1000, 24), (301, 512), (700, 520), (1300, 1024), (299, 1537), (333, 2048), (900, 4096),
         (600, 8192), (297, 16384), (450, 32768)]


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm_matches_definition(nat, dtype, rows, cols):
    g = gen(rows * 100003 + cols)
    x, r = randn(g, rows, cols).to(dtype), (3 * randn(g, rows, cols)).to(dtype)
    gain = (1 + 0.3 * randn(g, cols)).to(dtype)
    y, h = nat.bv_rms_norm(x, gain, eps=1e-5, residual=r)
    check_norm(x, r, gain, 1e-5, y, h)
    y = nat.bv_rms_norm(x, None, eps=1e-5)
    check_norm(x, None, None, 1e-5, y, None)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm_int8_matches_definition(nat, dtype, rows, cols):
    g = gen(rows * 100003 + cols + 1)
    x, r = randn(g, rows, cols).to(dtype), (3 * randn(g, rows, cols)).to(dtype)
    gain = 1 + 0.3 * randn(g, cols)  # f32 gain on every type
    q, scale, h = nat.bv_rms_norm_int8(x, gain, eps=1e-5, residual=r)
    want_q, a = expected_q(x, r, gain)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)
    _, rstd, y64 = norm64(x, r, gain, 1e-5)
    want = torch.from_numpy(a).cuda().double() * rstd[:, 0] / 127
    rel = (CHAIN(cols) / 2 + 10) * U
    close(scale, want, want * rel)
    # the values it stands for are half a step off, and the step's own error
    close(q.double() * scale.double()[:, None], y64, want[:, None] * (0.5 + 127 * rel + 1e-4))
    h64 = norm64(x, r, gain, 1e-5)[0]
    close(h, h64, h64.abs() * (HALF[dtype] + U) * 1.001 + TINY[dtype])


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize_rows(nat, dtype, rows, cols):
    x = (5 * randn(gen(cols), rows, cols)).to(dtype)
    q, scale = nat.bv_quantize_rows(x)
    want_q, a = expected_q(x, None, None)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)
    want = torch.from_numpy(a).cuda().double() / 127
    close(scale, want, want * 2 * U)


def test_many_rows(nat):
    """More rows than a grid of one block a row would hold at once."""
    x = randn(gen(3), 300001, 40).to(torch.bfloat16)
    check_norm(x, None, None, 1e-6, nat.bv_rms_norm(x), None)
    q, _ = nat.bv_quantize_rows(x)
    np.testing.assert_array_equal(q.cpu().numpy(), expected_q(x, None, None)[0])


@pytest.mark.parametrize("cols", [64, 1537, 4096, 20001])
@pytest.mark.parametrize("more", [0, 400])
def test_special_rows(nat, cols, more):
    """Rows of zeros, of one value, tiny and huge rows, infinities and NaN:
    each shows in its own row only, alone and ahead of many more rows."""
    g = gen(5)
    x = randn(g, 9 + more, cols)
    x[1] = 0
    x[2] = 0
    x[2, cols // 2] = -3.0
    x[3] *= 1e-42
    x[4] *= 1e30                # squares past 32 bits
    x[5, cols // 3] = float("inf")
    x[6, 0] = float("nan")
    x[7] *= 3e-38
    gain = 1 + 0.3 * randn(g, cols)
    y = nat.bv_rms_norm(x, gain, eps=1e-6)
    h64, rstd, y64 = norm64(x, None, gain, 1e-6)
    ok = [0, 1, 2, 3, 4, *range(7, 9 + more)]
    # rows 3 and 7 lie below 2^-126 in part: one step of 2^-149 there
    rel = (CHAIN(cols) / 2 + 9) * U
    close(y[ok], y64[ok], y64[ok].abs() * rel + 2.0 ** -149 * 1e4)
    assert torch.isnan(y[6]).all() and not torch.isfinite(y[5]).all()
    q, scale = nat.bv_rms_norm_int8(x, gain, eps=1e-6)
    assert torch.isnan(scale[[5, 6]]).all() and torch.isfinite(scale[ok]).all()
    assert int(q[[1, 5, 6]].abs().max()) == 0 and float(scale[1]) == 0.0
    assert int(q[2].abs().max()) == 127 and int((q[2] != 0).sum()) == 1
    t64 = (x * gain).double()
    a64 = t64.abs().amax(-1, keepdim=True)
    for row in (0, 3, 4, *range(7, 9 + more, 57)):
        want = torch.round(127 * t64[row] / a64[row])
        # row 3's products are whole multiples of 2^-149: its q follows the
        # rounded products; elsewhere values next to a border may go either way
        assert float((q[row].double() - want).abs().max()) <= 1
        assert int(q[row].abs().max()) == 127
    q, scale = nat.bv_quantize_rows(x)
    assert torch.isnan(scale[[5, 6]]).all() and int(q[[1, 5, 6]].abs().max()) == 0
    close(scale[ok], x[ok].double().abs().amax(-1) / 127,
          x[ok].double().abs().amax(-1) / 127 * 2 * U + 2.0 ** -149)


def test_norm_of_the_largest_values(nat):
    x = torch.full((2, 512), 3.0e38, device="cuda")
    x[1, ::2] = -3.0e38
    y = nat.bv_rms_norm(x, torch.full((512,), 2.0, device="cuda"))
    # 1 / rms is below 2^-126: a step of 2^-149 there is 2^-21 of it
    close(y, 2.0 * torch.sign(x).double(), torch.full_like(x, 2.0).double() * (40 * U + 2.0 ** -21))


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("cols,pad", [(64, 64), (100, 3), (256, 8), (1537, 7), (4096, 16)])
@pytest.mark.parametrize("n", [6, 333])
def test_strided_rows_and_what_lies_between(nat, dtype, cols, pad, n):
    """Rows of wider matrices; the columns beside them stay as they were."""
    g = gen(cols + pad)
    ld = cols + pad
    big = [randn(g, n, ld).to(dtype) for _ in range(4)]
    x, r, h, y = (b[:, pad // 2:pad // 2 + cols] for b in big)
    keep = [b.clone() for b in big]
    gain = (1 + 0.3 * randn(g, cols)).to(dtype)
    nat.bv_rms_norm(x, gain, residual=r, h=h, y=y)
    kx, kr = (k[:, pad // 2:pad // 2 + cols] for k in keep[:2])
    check_norm(kx, kr, gain, 1e-6, y, h)
    for b, k in zip(big[2:], keep[2:]):
        assert torch.equal(b[:, :pad // 2], k[:, :pad // 2])
        assert torch.equal(b[:, pad // 2 + cols:], k[:, pad // 2 + cols:])
    qb = torch.full((n + 1, ld), 99, device="cuda", dtype=torch.int8)
    q = qb[:n, pad // 2:pad // 2 + cols]
    nat.bv_rms_norm_int8(x, gain, residual=r, h=h, q=q)
    np.testing.assert_array_equal(q.cpu().numpy(), expected_q(kx, kr, gain)[0])
    outside = torch.ones_like(qb, dtype=torch.bool)
    outside[:n, pad // 2:pad // 2 + cols] = False
    assert (qb[outside] == 99).all()


@pytest.mark.parametrize("cols", [96, 1001, 8192, 40000])
@pytest.mark.parametrize("over", ["x", "residual"])
@pytest.mark.parametrize("rows", [5, 700])
def test_sum_in_place(nat, cols, over, rows):
    g = gen(cols)
    x, r = randn(g, rows, cols).to(torch.bfloat16), randn(g, rows, cols).to(torch.bfloat16)
    kx, kr = x.clone(), r.clone()
    y, h = nat.bv_rms_norm(x, None, residual=r, h=x if over == "x" else r)
    assert h is (x if over == "x" else r)
    check_norm(kx, kr, None, 1e-6, y, h)
    assert torch.equal(r if over == "x" else x, kr if over == "x" else kx)


@pytest.mark.parametrize("cols", [200, 1001, 1024])
@pytest.mark.parametrize("dtype", ALL)
def test_many_broadcast_rows(nat, cols, dtype):
    """One row read for all (stride 0), as x and as the residual."""
    g = gen(cols)
    x, r = randn(g, 400, cols).to(dtype), randn(g, 1, cols).to(dtype).expand(400, cols)
    y, h = nat.bv_rms_norm(x, None, residual=r)
    check_norm(x, r, None, 1e-6, y, h)
    y, h = nat.bv_rms_norm(r, None, residual=x)
    check_norm(r, x, None, 1e-6, y, h)
    q, _ = nat.bv_quantize_rows(r)
    np.testing.assert_array_equal(q.cpu().numpy(), expected_q(r, None, None)[0])


def test_rows_that_start_differently(nat):
    """x, residual, sum and y each off a 16-byte boundary by another amount."""
    g = gen(18)
    for rows, cols in ((3, 700), (400, 1500)):
        x, r, h, y = (torch.zeros(rows * cols + 8, device="cuda", dtype=torch.bfloat16)
                      [o:o + rows * cols].view(rows, cols) for o in (0, 1, 3, 6))
        x.copy_(randn(g, rows, cols))
        r.copy_(randn(g, rows, cols))
        nat.bv_rms_norm(x, None, residual=r, h=h, y=y)
        check_norm(x, r, None, 1e-6, y, h)
        q = torch.zeros(rows * cols + 8, device="cuda", dtype=torch.int8)[3:3 + rows * cols]
        q = q.view(rows, cols)
        nat.bv_quantize_rows(r, q=q)
        np.testing.assert_array_equal(q.cpu().numpy(), expected_q(r, None, None)[0])


def test_gains_that_start_anywhere(nat):
    g = gen(19)
    for dtype in ALL:
        for cols in (1000, 1024, 1031):
            gain = (1 + 0.3 * randn(g, cols + 3)).to(dtype)[3:]
            for rows in (4, 400):
                x = randn(g, rows, cols).to(dtype)
                check_norm(x, None, gain, 1e-6, nat.bv_rms_norm(x, gain), None)


def test_broadcast_rows_and_leading_dims(nat):
    g = gen(8)
    x = randn(g, 2, 3, 200)
    r = randn(g, 1, 200).expand(6, 200).view(2, 3, 200)
    y, h = nat.bv_rms_norm(x, None, residual=r)
    assert y.shape == x.shape
    check_norm(x, r, None, 1e-6, y, h)
    q, scale = nat.bv_quantize_rows(x)
    assert q.shape == x.shape and scale.shape == (2, 3)


def test_empty_rows(nat):
    x = torch.empty(0, 64, device="cuda")
    assert nat.bv_rms_norm(x).shape == (0, 64)
    q, s = nat.bv_rms_norm_int8(x)
    assert q.shape == (0, 64) and s.shape == (0,)
    w, ws = nat.bv_quantize_rows(randn(gen(0), 8, 64))
    assert nat.bv_int8_matmul(q, s, w, ws).shape == (0, 8)
    assert nat.bv_int8_matmul(q, s, w, ws, channels_first=True).shape == (8, 0)


# ------------------------------------------------------------ integer product


def int8(g, rows, cols, pad=True):
    ld = (cols + 15) // 16 * 16 if pad else cols
    return torch.randint(-128, 128, (rows, ld), device="cuda", generator=g,
                         dtype=torch.int8)[:, :cols]


def check_product(a, sa, w, sw, bias, residual, y, dtype, cf):
    p = (a.double() @ w.double().t()) * sa.double()[:, None] * sw.double()
    b = torch.zeros_like(p) if bias is None else bias.double().expand_as(p)
    r = torch.zeros_like(p) if residual is None else \
        (residual.double().t() if cf else residual.double())
    want = p + b + r
    tol = U * (3 * p.abs() + (p + b).abs() + want.abs()) * 1.01 + HALF[dtype] * want.abs() * 1.01
    got = y.t() if cf else y
    close(got, want, tol + TINY[dtype])


SHAPES = [(1, 1, 1), (1, 5, 3), (2, 16, 32), (1, 128, 64), (3, 33, 127), (16, 256, 128),
          (17, 100, 130), (32, 512, 1000), (64, 64, 4096), (100, 777, 1111), (128, 128, 256),
          (129, 257, 129), (255, 300, 640), (333, 1024, 512), (1, 4096, 4096), (1, 2000, 131071),
          (5, 40, 8200), (513, 130, 2050), (1000, 32, 1024), (2049, 96, 96), (700, 700, 700),
          (1, 40000, 64), (20000, 1, 48), (4100, 260, 4096)]


@pytest.mark.parametrize("pad", ["both", "a", "w", "none"])
@pytest.mark.parametrize("cf", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_matches_definition(nat, M, N, K, cf, pad):
    """pad: the operands whose rows start on 16 bytes whatever K is."""
    g = gen(M * 31 + N * 7 + K)
    a, w = int8(g, M, K, pad in ("both", "a")), int8(g, N, K, pad in ("both", "w"))
    sa, sw = (torch.rand(n, device="cuda", generator=g) * 0.01 + 1e-4 for n in (M, N))
    bias = randn(g, N)
    y = nat.bv_int8_matmul(a, sa, w, sw, bias=bias, channels_first=cf)
    assert y.shape == ((N, M) if cf else (M, N)) and y.dtype == torch.float32
    check_product(a, sa, w, sw, bias, None, y, torch.float32, cf)
    for dtype in (torch.bfloat16, torch.float16):
        sd = sw * (200.0 / K ** 0.5 / 73 ** 2) if dtype == torch.float16 else sw
        res = randn(g, *y.shape).to(dtype)
        y2 = nat.bv_int8_matmul(a, sa, w, sd, residual=res, channels_first=cf)
        assert y2.dtype == dtype
        check_product(a, sa, w, sd, None, res, y2, dtype, cf)


@pytest.mark.parametrize("M,N", [(1, 64), (200, 300), (1024, 512)])
def test_product_of_extreme_values(nat, M, N):
    """Every product 2^14 at the largest depth: sums of 131071 * 2^14 < 2^31."""
    K = 131071
    a = torch.full((M, K + 1), -128, device="cuda", dtype=torch.int8)[:, :K]
    w = torch.full((N, K + 1), -128, device="cuda", dtype=torch.int8)[:, :K]
    w[::2] = 127
    one = torch.ones(max(M, N), device="cuda")
    y = nat.bv_int8_matmul(a, one[:M], w, one[:N])
    want = torch.where(torch.arange(N, device="cuda") % 2 == 0, -128.0 * 127 * K, 16384.0 * K)
    assert torch.equal(y, want.float().expand(M, N))  # one rounding, the same on both sides


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("cf", [False, True])
@pytest.mark.parametrize("M,N,K,oy,py", [(70, 90, 96, 0, 6), (70, 90, 96, 1, 5), (300, 256, 512, 3, 2),
                                         (5, 1000, 200, 2, 8), (257, 129, 64, 1, 1)])
def test_product_strided_output(nat, dtype, cf, M, N, K, oy, py):
    """Outputs and residuals inside wider matrices, starting anywhere."""
    g = gen(M + N + oy)
    a, w = int8(g, M, K), int8(g, N, K)
    sa, sw = (torch.rand(n, device="cuda", generator=g) * 0.01 for n in (M, N))
    R, C = (N, M) if cf else (M, N)
    yb = torch.full((R + 1, C + oy + py), 7.0, device="cuda", dtype=dtype)
    rb = randn(g, R, C + 3).to(dtype)
    y, res = yb[:R, oy:oy + C], rb[:, 1:1 + C]
    nat.bv_int8_matmul(a, sa, w, sw, residual=res, y=y, channels_first=cf)
    check_product(a, sa, w, sw, None, res, y, dtype, cf)
    outside = torch.ones_like(yb, dtype=torch.bool)
    outside[:R, oy:oy + C] = False
    assert (yb[outside] == 7.0).all()


@pytest.mark.parametrize("off_a,off_w", [(0, 1), (3, 0), (5, 13), (8, 4)])
@pytest.mark.parametrize("M,N,K", [(1, 70, 200), (4, 300, 512), (40, 60, 300), (300, 500, 130)])
def test_product_operands_inside_wider_rows(nat, M, N, K, off_a, off_w):
    """Operands that start anywhere; the bytes around them are not theirs."""
    g = gen(M + N + K + off_a)
    a, w = int8(g, M, K + 20, False)[:, off_a:off_a + K], int8(g, N, K + 33, False)[:, off_w:off_w + K]
    sa, sw = (torch.rand(n, device="cuda", generator=g) * 0.01 for n in (M, N))
    for cf in (False, True):
        y = nat.bv_int8_matmul(a, sa, w, sw, channels_first=cf)
        check_product(a, sa, w, sw, None, None, y, torch.float32, cf)


def test_product_adds_in_place(nat):
    g = gen(4)
    a, w = int8(g, 300, 256), int8(g, 130, 256)
    sa, sw = (torch.rand(n, device="cuda", generator=g) * 0.01 for n in (300, 130))
    y = randn(g, 300, 130)
    before = y.clone()
    assert nat.bv_int8_matmul(a, sa, w, sw, residual=y, y=y) is y
    check_product(a, sa, w, sw, None, before, y, torch.float32, False)


def test_product_operands_may_be_broadcast_and_shared(nat):
    g = gen(6)
    row = int8(g, 1, 128)
    a = row.expand(40, 128)
    s = torch.ones(40, device="cuda")
    y = nat.bv_int8_matmul(a, s, a, s)
    assert torch.equal(y, torch.full_like(y, float((row.double() ** 2).sum())))


def test_product_nan_scale_stays_in_its_row(nat):
    g = gen(7)
    a, w = int8(g, 64, 96), int8(g, 48, 96)
    sa, sw = torch.ones(64, device="cuda"), torch.ones(48, device="cuda")
    sa[5] = float("nan")
    a[5] = 0
    y = nat.bv_int8_matmul(a, sa, w, sw)
    assert torch.isnan(y[5]).all() and torch.isfinite(y[:5]).all() and torch.isfinite(y[6:]).all()


@pytest.mark.parametrize("M", [1, 2, 5, 33, 64, 200])
def test_tokens_do_not_see_their_batch(nat, M):
    """A token's result is the same bits alone and in any batch."""
    g = gen(9)
    a, w = int8(g, 200, 1000), int8(g, 300, 1000)
    sa, sw = (torch.rand(n, device="cuda", generator=g) * 0.01 for n in (200, 300))
    bias = randn(g, 300)
    whole = nat.bv_int8_matmul(a, sa, w, sw, bias=bias)
    assert torch.equal(nat.bv_int8_matmul(a[:M], sa[:M], w, sw, bias=bias), whole[:M])
    x = randn(g, 200, 1000).to(torch.bfloat16)
    q, s = nat.bv_rms_norm_int8(x)
    q1, s1 = nat.bv_rms_norm_int8(x[:M])
    assert torch.equal(q[:M], q1) and torch.equal(s[:M], s1)


def test_large_offsets(nat):
    """Rows past 2^31 elements: a view of few rows with a long stride."""
    ld = (1 << 31) // 4 + 64
    buf = torch.zeros(5 * ld, device="cuda", dtype=torch.bfloat16)
    x = buf.as_strided((5, 512), (ld, 1))
    g = gen(10)
    x.copy_(randn(g, 5, 512))
    y = buf.as_strided((5, 512), (ld, 1), 4096)
    nat.bv_rms_norm(x, y=y)
    check_norm(x.clone(), None, None, 1e-6, y, None)
    del x, y, buf
    ld = (1 << 28)
    buf = torch.zeros(9 * ld + 4096, device="cuda", dtype=torch.int8)
    a = buf.as_strided((10, 512), (ld, 1))
    a.copy_(int8(g, 10, 512))
    w = int8(g, 64, 512)
    sa, sw = torch.ones(10, device="cuda"), torch.ones(64, device="cuda")
    check_product(a, sa, w, sw, None, None, nat.bv_int8_matmul(a, sa, w, sw), torch.float32, False)
    check_product(w, sw, a, sa, None, None, nat.bv_int8_matmul(w, sw, a, sa), torch.float32, False)


# ---------------------------------------------- streams, graphs, the whole path


def test_streams_and_two_calls_at_once(nat):
    g = gen(11)
    x = [randn(g, 700, 1024).to(torch.bfloat16) for _ in range(2)]
    w, sw = nat.bv_quantize_rows(randn(g, 512, 1024))
    def layer(v, stream=None):
        q, s = nat.bv_rms_norm_int8(v, stream=stream)
        return nat.bv_int8_matmul(q, s, w, sw, stream=stream)
    want = [layer(v) for v in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    for _ in range(5):
        got = [layer(v, s) for v, s in zip(x, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (40, 300, 4096), (700, 1024, 1001), (600, 4096, 512)])
def test_launches_keep_their_order(nat, M, N, K):
    """Kernels that may be scheduled early still read what the one before them
    wrote, and overwrite nothing it reads: a chain over the same few buffers,
    with other kernels between, against the same chain with a wait after each
    step."""
    g = gen(20)
    w, sw = nat.bv_quantize_rows(randn(g, N, K))
    back, sb = nat.bv_quantize_rows(randn(g, K, N))
    start = randn(g, M, K)

    def chain(wait):
        def step(r):
            if wait:
                torch.cuda.synchronize()
            return r
        x = start.clone()
        total = torch.zeros_like(x)
        q = torch.empty(M, (K + 15) // 16 * 16, device="cuda", dtype=torch.int8)[:, :K]
        p = torch.empty(M, (N + 15) // 16 * 16, device="cuda", dtype=torch.int8)[:, :N]
        s, sp = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        y, z = torch.empty(M, N, device="cuda"), torch.empty(M, K, device="cuda")
        for i in range(40):
            step(nat.bv_rms_norm_int8(x, None, residual=start, h=x, q=q, scale=s))
            step(nat.bv_int8_matmul(q, s, w, sw, y=y))
            step(nat.bv_quantize_rows(y, q=p, scale=sp))
            step(nat.bv_int8_matmul(p, sp, back, sb, residual=x, y=z))
            step(nat.bv_rms_norm(z, None, y=x))
            if i % 3 == 0:
                step(total.add_(x))
                step(z.zero_())
        return total
    want = chain(True)
    assert torch.isfinite(want).all()
    for _ in range(3):
        assert torch.equal(chain(False), want)


@pytest.mark.parametrize("rows", [3, 500])
def test_calls_wait_for_events_of_other_streams(nat, rows):
    """A call behind an event waits for what the event stands for, although a
    kernel of the same kind ran just before it on its own stream."""
    g = gen(21)
    big = randn(g, 4096, 4096)
    other = randn(g, rows, 1024)
    w, sw = nat.bv_quantize_rows(randn(g, 64, 1024))
    x = torch.zeros(rows, 1024, device="cuda")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for i in range(8):
        x.zero_()
        fresh = randn(g, rows, 1024)
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            for _ in range(3):
                big @ big  # keeps s1 busy for milliseconds
            x.copy_(fresh)
            ready = torch.cuda.Event()
            ready.record(s1)
        with torch.cuda.stream(s2):
            nat.bv_rms_norm(other)
            s2.wait_event(ready)
            q, s = nat.bv_rms_norm_int8(x)
            y = nat.bv_int8_matmul(q, s, w, sw)
        torch.cuda.synchronize()
        q1, s1_ = nat.bv_rms_norm_int8(fresh)
        assert torch.equal(q, q1) and torch.equal(s, s1_)
        assert torch.equal(y, nat.bv_int8_matmul(q1, s1_, w, sw))


def test_captured_and_replayed(nat):
    """Two graphs of the same layer, replayed in turn on new inputs."""
    g = gen(12)
    w, sw = nat.bv_quantize_rows(randn(g, 256, 512))
    x = [torch.zeros(40, 512, device="cuda") for _ in range(2)]
    r = [torch.zeros(40, 512, device="cuda") for _ in range(2)]
    def layer(i):
        q, s, h = nat.bv_rms_norm_int8(x[i], residual=r[i])
        return nat.bv_int8_matmul(q, s, w, sw), h
    for i in range(2):
        layer(i)  # once outside a capture: kernel attributes
    graphs, outs = [], []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(layer(i))
        graphs.append(gr)
    for _ in range(3):
        for i in range(2):
            x[i].copy_(randn(g, 40, 512))
            r[i].copy_(randn(g, 40, 512))
        for gr in graphs:
            gr.replay()
        for i in range(2):
            y, h = layer(i)
            assert torch.equal(outs[i][0], y) and torch.equal(outs[i][1], h)
    torch.cuda.synchronize()


def layer64(x, residual, gain, q_w, s_w, bias, eps):
    """The front end in 64 bits from the 8-bit weights: values next to a
    rounding border may differ by one step."""
    h, rstd, _ = norm64(x, residual, gain, eps)
    t = h if gain is None else h * gain.double()
    a = t.abs().amax(-1, keepdim=True)
    rows = torch.round(127 * t / a) * a * rstd / 127
    return rows, rows @ (q_w.double() * s_w.double()[:, None]).t() + \
        (0 if bias is None else bias.double())


@pytest.mark.parametrize("by_side", [False, True])
@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("S,T,D,C", [(2, 1, 64, 32), (2, 37, 200, 32), (1, 300, 1024, 32),
                                     (2, 250, 1001, 64)])
def test_token_front_end(nat, S, T, D, C, dtype, by_side):
    g = gen(S * T + D)
    x, r = randn(g, S, T, D).to(dtype), randn(g, S, T, D).to(dtype)
    gain, weight, bias = 1 + 0.2 * randn(g, D), randn(g, C, D) / D ** 0.5, randn(g, C)
    front = nat.TokenFrontEnd(gain, weight, bias)
    z = front(x, r, by_side=by_side)
    assert z.shape == ((S, C, T) if by_side else (C, S, T))
    rows, want = layer64(x, r, gain, front.w, front.w_scale, bias, 1e-6)
    want = want.permute(0, 2, 1) if by_side else want.permute(2, 0, 1)
    # one step of one value for each 4096 values of a row, rounded up, is far
    # more than borders take; the rest is 32-bit arithmetic
    step = float(rows.abs().amax() / 127 * (front.w_scale.max() * 127))
    close(z, want, (want.abs() + 1) * 100 * U + step * (D // 4096 + 1))
    # and the calls it stands for, bit for bit
    q, s = nat.bv_rms_norm_int8(x.view(S * T, D), gain, residual=r.view(S * T, D))[:2]
    y = nat.bv_int8_matmul(q, s, front.w, front.w_scale, bias=bias)
    y = y.view(S, T, C)
    assert torch.equal(z, (y.permute(0, 2, 1) if by_side else y.permute(2, 0, 1)))


@pytest.mark.parametrize("with_front_end", [False, True])
def test_decode_tokens(nat, oracle, with_front_end):
    """Hidden states to waveform, against the oracle decoding the 64-bit
    latents of the same 8-bit layer."""
    from bigvgan_waveform_decoder_alias_b200 import synth
    geo = synth.tiny_geometry(pre_channels=64, up_channels=(48, 32, 16), in_channels=16)
    s = synth.NormalStream(77)
    params = s.normal((synth.param_count(geo),), 0.0, 0.02)
    L = 24 if with_front_end else geo.in_channels
    fe = None
    if with_front_end:
        fe = (s.normal((L,)), np.abs(s.normal((L,))) + 0.5, s.normal((geo.in_channels, L, 1)) * 0.2,
              s.normal((geo.in_channels,)))
    dec = nat.Decoder(geo, params, front_end=fe)
    g = gen(13)
    x = randn(g, 2, 9, 128).to(torch.bfloat16)
    front = nat.TokenFrontEnd(1 + 0.1 * randn(g, 128), randn(g, L, 128) / 11, randn(g, L))
    y = dec.decode_tokens(x, front)
    z = front(x, by_side=not with_front_end)
    assert torch.equal(y, dec.decode(z))
    z = z.cpu().numpy()
    if with_front_end:
        z = oracle.latent_front_end(z, *fe)
    want = oracle.decode(geo, params, np.ascontiguousarray(z, np.float32))
    err = np.linalg.norm(y.cpu().numpy() - want) / np.linalg.norm(want)
    assert err < 1e-4  # the decoder's own tolerance


def test_decode_tokens_music(nat):
    """The DAV decoder takes the front end's latents by side."""
    from bigvgan_waveform_decoder_alias_b200 import synth
    geo = synth.MUSIC3_DAV
    s = synth.NormalStream(78)
    dec = nat.DavDecoder(geo, synth.draw_dav_params(s, geo))
    g = gen(17)
    front = nat.TokenFrontEnd(None, randn(g, geo.latent_channels, 96) / 10)
    x, r = randn(g, 2, 4, 96), randn(g, 2, 4, 96)
    y = dec.decode_tokens(x, front, residual=r)
    assert y.shape == (2, 1, 4 * geo.hop)
    assert torch.equal(y, dec.decode(front(x, r, by_side=True)))


def test_captured_without_a_call_before():
    """Shapes whose kernels no call has used yet, captured in a new process
    after one call of another shape; replays equal eager calls."""
    import subprocess
    import sys
    code = """
import torch
from bigvgan_waveform_decoder_alias_b200 import native
def call(m, n, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((m, k), device="cuda", generator=g)
    w = torch.randint(-128, 128, (n, k), device="cuda", generator=g, dtype=torch.int8)
    sw = torch.rand(n, device="cuda", generator=g)
    def f():
        q, s, h = native.bv_rms_norm_int8(x, residual=x)
        return native.bv_int8_matmul(q, s, w, sw, out_dtype=torch.bfloat16), h
    return f
call(8, 16, 32, 0)()
torch.cuda.synchronize()
for i, (m, n, k) in enumerate([(1, 300, 64), (30, 200, 4096), (700, 4096, 256), (600, 5000, 520),
                               (900, 700, 999), (4, 64, 40000)]):
    f = call(m, n, k, i)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    graph.replay()
    torch.cuda.synchronize()
    want = f()
    assert all(torch.equal(a, b) for a, b in zip(out, want)), (m, n, k)
print("captured")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_refusals(nat):
    g = gen(14)
    x = randn(g, 4, 64)
    q, s = nat.bv_quantize_rows(x)
    bad = [lambda: nat.bv_rms_norm(x.double()), lambda: nat.bv_rms_norm(x, x[0, :63]),
           lambda: nat.bv_rms_norm(x, residual=x.half()), lambda: nat.bv_rms_norm(x, y=x),
           lambda: nat.bv_rms_norm(x, eps=0.0), lambda: nat.bv_rms_norm(x[:, ::2]),
           lambda: nat.bv_rms_norm(x.t()), lambda: nat.bv_rms_norm(x, residual=x[:3]),
           lambda: nat.bv_rms_norm(x, x[0].bfloat16()),
           lambda: nat.bv_int8_matmul(q, s, q[:, :32], s), lambda: nat.bv_int8_matmul(q, s, x, s),
           lambda: nat.bv_int8_matmul(q, s[:3], q, s),
           lambda: nat.bv_int8_matmul(q, s, q, s, out_dtype=torch.float64),
           lambda: nat.bv_int8_matmul(q, s, q, s, y=torch.empty(4, 5, device="cuda")),
           lambda: nat.bv_int8_matmul(q, s, q, s, residual=torch.empty(5, 4, device="cuda")),
           lambda: nat.bv_rms_norm(torch.empty(3, 0, device="cuda"))]
    for call in bad:
        with pytest.raises(nat.BVError):
            call()


def test_timing_classes(nat):
    """The launches are counted and tagged like the library's others."""
    g = gen(15)
    nat.timing(True)
    nat.timing_reset()
    try:
        n0 = nat.launch_count()
        q, s = nat.bv_rms_norm_int8(randn(g, 16, 256))
        w, sw = nat.bv_quantize_rows(randn(g, 64, 256))
        nat.bv_int8_matmul(q, s, w, sw)
        assert nat.launch_count() - n0 == 3
        got = nat.timing_read(64)
    finally:
        nat.timing(False)
        nat.timing_reset()
    assert {"rms_norm", "quantize_rows", "int8_matmul"} <= set(got)


def _status(nat):
    import ctypes
    return nat.lib().bv_sync_status(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))


@pytest.mark.parametrize("call", ["pair", "tile", "split", "copied", "copied_split", "rows"])
def test_bounded_waits_report_and_leave_the_context_usable(nat, call):
    """The bounded waits made to run out at once by the library's testing hook:
    the status word says so, and the same call at the default limit is right."""
    g = gen(16)
    M, N, K, pad = {"pair": (600, 4096, 640, True), "tile": (100, 300, 640, True),
                    "split": (20, 256, 4096, True), "copied": (100, 300, 650, False),
                    "copied_split": (20, 256, 4090, False), "rows": (700, 0, 1024, True)}[call]
    if call == "rows":
        x = randn(g, M, K)
        run = lambda: nat.bv_rms_norm(x)  # noqa: E731
    else:
        a, w = int8(g, M, K), int8(g, N, K, pad)
        sa, sw = (torch.rand(n, device="cuda", generator=g) * 0.01 for n in (M, N))
        run = lambda: nat.bv_int8_matmul(a, sa, w, sw)  # noqa: E731
    run()
    assert _status(nat) == 0
    nat.set_wait_limit(0)
    try:
        run()
        st = _status(nat)
    finally:
        nat.set_wait_limit(-1)
    assert st == 5, st  # BV_ERR_TIMEOUT
    y = run()
    assert _status(nat) == 0
    if call == "rows":
        check_norm(x, None, None, 1e-6, y, None)
    else:
        check_product(a, sa, w, sw, None, None, y, torch.float32, False)


def test_front_end_is_called_at_once_on_another_stream(nat):
    """Made behind queued work on one stream and called on another without a
    wait between: the call reads the finished weight."""
    g = gen(22)
    big = randn(g, 4096, 4096)
    x = randn(g, 2, 30, 256)
    other = torch.cuda.Stream()
    for _ in range(6):
        weight = randn(g, 32, 256)
        torch.cuda.synchronize()
        for _ in range(5):
            big @ big  # keeps the current stream busy for milliseconds
        front = nat.TokenFrontEnd(None, weight)
        z = front(x, stream=other)
        other.synchronize()
        q, s = nat.bv_quantize_rows(weight)
        assert torch.equal(front.w, q) and torch.equal(front.w_scale, s)
        assert torch.equal(z, front(x))


@pytest.mark.parametrize("short", [1, 500])
def test_the_longest_rows(nat, short):
    """A row of 2^31 - short values: neither the count of its groups nor the
    step past its end may leave 32 bits.  Whole numbers up to 127, so q is x."""
    cols, step = 2 ** 31 - short, 1 << 26
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    x = torch.empty(1, cols, device="cuda", dtype=torch.bfloat16)
    squares = 0.0
    for at in range(0, cols, step):
        i = torch.arange(at, min(at + step, cols), device="cuda")
        v = ((i * 2654435761) >> 7) % 255 - 127
        x[0, at:at + step] = v
        squares += float((v * v).sum())
    q, scale = nat.bv_quantize_rows(x)
    assert float(scale) == 1.0
    for at in range(0, cols, step):
        assert torch.equal(q[0, at:at + step], x[0, at:at + step].to(torch.int8)), at
    del q
    y, h = nat.bv_rms_norm(x, residual=x)
    rstd = (4 * squares / cols + 1e-6) ** -0.5
    rel = (CHAIN(cols) / 2 + 8) * U + HALF[torch.bfloat16]
    for at in range(0, cols, step):
        part = x[0, at:at + step].float()
        assert torch.equal(h[0, at:at + step].float(), 2 * part), at
        want = 2 * part * rstd
        assert bool(((y[0, at:at + step].float() - want).abs() <= want.abs() * rel * 1.001).all()), at


@pytest.mark.parametrize("lift", [1.0, 1e20])
def test_sum_of_many_equal_squares(nat, lift):
    """2^16 values of a row to each thread: the sum of so many squares in 32 bits
    would lose a part of each.  (Those of the lifted row are past 32 bits.)"""
    cols = 1 << 26
    x = torch.full((1, cols), 1.14 * lift, device="cuda")
    y = nat.bv_rms_norm(x, eps=1e-6)
    want = 1.0 / (1.0 + 1e-6 / float(x[0, 0]) ** 2) ** 0.5
    # a part's 64 sums, the joint sum in 64 bits and its rounding, 10 sums over the
    # block, halved by the root; division, eps, root and product
    close(y, torch.full_like(y, want).double(), torch.full_like(y, want).double() * (75 / 2 + 8) * U)
    q, scale = nat.bv_rms_norm_int8(x, eps=1e-6)
    assert bool((q == 127).all())
    assert abs(float(scale) * 127 / want - 1) <= (75 / 2 + 10) * U


# ------------------------------- products in many tiles, in place, in batches


@pytest.mark.parametrize("cf", [False, True])
@pytest.mark.parametrize("rows,cols,K", [
    # rows (the dimension y keeps consecutive) x columns x depth, so many that a
    # pair of CTAs works through five tiles of 256 rows and more, each with more
    # steps of 128 than its ring of stages has slots: 256 columns a tile, ragged in
    # every direction and in whole tiles, then 192, 128 and 64 columns
    (4865, 4901, 1000), (5120, 4864, 1024), (33001, 571, 1000), (95500, 100, 1300),
    (95499, 49, 1400)])
def test_product_in_many_tiles(nat, rows, cols, K, cf):
    M, N = (rows, cols) if cf else (cols, rows)
    g = gen(rows + cols)
    a, w = int8(g, M, K), int8(g, N, K)
    sa, sw = (torch.rand(n, device="cuda", generator=g) * 0.01 + 1e-4 for n in (M, N))
    bias = randn(g, N)
    y = nat.bv_int8_matmul(a, sa, w, sw, bias=bias, channels_first=cf)
    check_product(a, sa, w, sw, bias, None, y, torch.float32, cf)
    sd = sw * (200.0 / K ** 0.5 / 73 ** 2)  # inside fp16's range
    for dtype in (torch.bfloat16, torch.float16):
        y = randn(g, *y.shape).to(dtype)
        before = y.clone()
        nat.bv_int8_matmul(a, sa, w, sd, bias=bias, residual=y, y=y, channels_first=cf)
        check_product(a, sa, w, sd, bias, before, y, dtype, cf)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("cf", [False, True])
@pytest.mark.parametrize("pad", [True, False])
@pytest.mark.parametrize("rows,cols,K", [
    (1001, 1, 600), (1000, 3, 601),            # dot products
    (130, 301, 256), (1000, 200, 1003),        # tiles
    (257, 20, 4100), (300, 60, 5000),          # tiles whose depth a cluster shares
    (2002, 701, 500), (4000, 512, 640)])       # tiles of pairs
def test_product_adds_in_place_everywhere(nat, rows, cols, K, pad, cf, dtype):
    """The residual is y itself, each kernel, both layouts; with 16-bit types
    whole words are written of which a neighbour read one half."""
    M, N = (rows, cols) if cf else (cols, rows)
    g = gen(rows + cols + K)
    a, w = int8(g, M, K, pad), int8(g, N, K, pad)
    sa, sw = (torch.rand(n, device="cuda", generator=g) * 0.01 + 1e-4 for n in (M, N))
    sw = sw * (200.0 / K ** 0.5 / 73 ** 2)
    y = randn(g, *((N, M) if cf else (M, N))).to(dtype)
    before = y.clone()
    assert nat.bv_int8_matmul(a, sa, w, sw, residual=y, y=y, channels_first=cf) is y
    check_product(a, sa, w, sw, None, before, y, dtype, cf)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("cols", [1000, 1024, 5000])
def test_tokens_in_batches_of_any_size(nat, dtype, cols):
    """From 296 rows on rows go through another kernel, and a product of many
    tokens through others: q and a product are the same bits, a row's scale and
    norm the same to the roundings of their sums' orders."""
    g = gen(cols)
    x = randn(g, 2000, cols).to(dtype)
    gain = 1 + 0.3 * randn(g, cols)
    w, sw = nat.bv_quantize_rows(randn(g, 2100, cols))
    bias = randn(g, 2100)
    q, s = nat.bv_rms_norm_int8(x, gain)
    y = nat.bv_rms_norm(x, gain)
    z = nat.bv_int8_matmul(q, s, w, sw, bias=bias)
    rel = 2 * (CHAIN(cols) / 2 + 10) * U  # each of the two off by half of it
    for first, n in ((0, 1), (7, 3), (100, 40), (0, 295), (5, 296), (3, 1700)):
        part = slice(first, first + n)
        q1, s1 = nat.bv_rms_norm_int8(x[part], gain)
        assert torch.equal(q1, q[part])
        close(s1, s[part], s[part].double() * rel)
        y1 = nat.bv_rms_norm(x[part], gain).double()
        assert bool(((y1 - y[part].double()).abs() <=
                     y1.abs() * (rel + 2 * HALF[dtype]) * 1.001 + TINY[dtype]).all())
        assert torch.equal(nat.bv_int8_matmul(q[part], s[part], w, sw, bias=bias), z[part])


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("T,D,C", [(30, 64, 32), (200, 1024, 32), (50, 1001, 64)])
def test_front_end_against_the_unquantised_projection(nat, dtype, T, D, C):
    """How far the 8 bits move the latents from norm and projection in 64 bits:
    half a step (and its own 32-bit error) of every value of the rows and of the
    weight, against the other's absolute values, and of both together."""
    g = gen(T + D + C)
    x = randn(g, 1, T, D).to(dtype)
    gain, weight, bias = 1 + 0.2 * randn(g, D), randn(g, C, D) / D ** 0.5, randn(g, C)
    z = nat.TokenFrontEnd(gain, weight, bias)(x)[:, 0].t().double()
    y64 = norm64(x, None, gain, 1e-6)[2][0]
    w64 = weight.double()
    want = y64 @ w64.t() + bias.double()
    rel = 127 * (CHAIN(D) / 2 + 10) * U + 1e-4
    dy = y64.abs().amax(-1, keepdim=True) / 127 * (0.5 + rel)
    dw = w64.abs().amax(-1, keepdim=True).t() / 127 * (0.5 + rel)
    tol = y64.abs().sum(-1, keepdim=True) * dw + dy * w64.abs().sum(-1) + D * dy * dw
    close(z, want, tol + (want.abs() + 1) * 100 * U)


@pytest.mark.parametrize("rows", [3, 500])
def test_captured_calls_wait_for_other_branches(nat, rows):
    """A graph with two branches: a call behind the join reads what the other
    branch wrote, although a kernel of the same kind is ahead of it on its own;
    two such graphs replayed on two streams at once stay apart."""
    g = gen(23)
    big = randn(g, 2048, 2048)
    w, sw = nat.bv_quantize_rows(randn(g, 64, 1024))
    graphs, ins, outs = [], [], []
    for i in range(2):
        x, src, other = (torch.zeros(rows, 1024, device="cuda") for _ in range(3))
        nat.bv_int8_matmul(*nat.bv_rms_norm_int8(x), w, sw)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                big @ big  # the other branch is the longer one
                big @ big
                x.copy_(src)
            nat.bv_rms_norm(other)
            main.wait_stream(side)
            q, s = nat.bv_rms_norm_int8(x)
            y = nat.bv_int8_matmul(q, s, w, sw)
        graphs.append(graph)
        ins.append((x, src))
        outs.append((q, s, y))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(6):
        for x, src in ins:
            x.zero_()
            src.copy_(randn(g, rows, 1024))
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for (_, src), (q, s, y) in zip(ins, outs):
            q1, s1 = nat.bv_rms_norm_int8(src)
            assert torch.equal(q, q1) and torch.equal(s, s1)
            assert torch.equal(y, nat.bv_int8_matmul(q1, s1, w, sw))
