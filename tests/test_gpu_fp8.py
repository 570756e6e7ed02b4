"""Block-scaled 8-bit quantisation and matrix product against plain 64-bit
forms (worker_ref), at sizes that fill no tile, with strides, alignments,
formats, special values, streams and graphs.

Codes and scales have to be equal.  The product's tolerance: the products of
codes are exact; each of the K / 32 additions into an fp32 accumulator (and a
few more: segments, clusters, the addend) may lose up to 2^-22 of the sum of
the magnitudes, and the result is rounded once to its type."""
import numpy as np
import pytest

import worker_ref as ref
from helpers import need_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return need_cuda()


def fp8(torch, fmt):
    return torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2


def values(rows, cols, seed, spread=3.0):
    g = np.random.default_rng([301, seed, rows, cols])
    x = g.standard_normal((rows, cols)) * np.exp(spread * g.standard_normal((rows, 1)) * 0.5)
    return (x * np.exp(spread * 0.3 * g.standard_normal((1, cols)))).astype(np.float32)


def as_type(torch, x, dtype):
    t = torch.from_numpy(x).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def check_quantize(torch, g, x, fmt, square, both=(True, True)):
    """x: a CUDA tensor (any strides that the call takes)."""
    rows, cols = x.shape
    q, s = g.fp8_matrix(rows, cols, fp8(torch, fmt))
    qt, st = g.fp8_matrix(cols, rows, fp8(torch, fmt))
    for t in (s, st):
        t.fill_(77)
    g.gar_fp8_quantize(x, q if both[0] else None, s if both[0] else None, qt if both[1] else None,
                       st if both[1] else None, square=square)
    host = x.float().cpu().numpy()
    for use, codes, scales, src in ((both[0], q, s, host), (both[1], qt, st, host.T)):
        if not use:
            continue
        want, bytes_ = ref.quantize(src, fmt, square)
        np.testing.assert_array_equal(scales.cpu().numpy(), ref.pack_scales(bytes_))
        np.testing.assert_array_equal(codes.float().cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (128, 1), (3, 130), (77, 1000), (128, 128), (129, 127),
                                       (200, 513), (511, 65), (300, 1024)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("square", [False, True])
def test_quantize(env, rows, cols, fmt, dtype, square):
    torch, g = env
    check_quantize(torch, g, as_type(torch, values(rows, cols, 1), dtype), fmt, square)


@pytest.mark.parametrize("both", [(True, False), (False, True)])
def test_quantize_one_order(env, both):
    torch, g = env
    check_quantize(torch, g, as_type(torch, values(150, 260, 2), "bf16"), "e4m3", False, both)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_strides_and_alignment(env, dtype):
    torch, g = env
    wide = as_type(torch, values(140, 700, 3), dtype)
    check_quantize(torch, g, wide[:, 5:400], "e4m3", False)
    check_quantize(torch, g, wide[:, 8:408], "e4m3", True)
    check_quantize(torch, g, wide[::2, 3:260], "e5m2", False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("square", [False, True])
def test_quantize_special_values(env, dtype, square):
    """Zeros, values at the scale's steps, the smallest and largest of the type, infinities and NaN."""
    torch, g = env
    x = values(260, 390, 4)
    x[5] = 0.0
    x[130:, :128] = 0.0
    x[7, 3] = 448.0
    x[8, :] = 448.0 * 2.0 ** -9
    x[9, 4] = np.nextafter(np.float32(448.0), np.float32(1e9))
    x[10, 5], x[10, 6] = 1e-42, -0.0
    x[11] = 3e-39
    x[12, 100] = 3.3e38
    x[13, 20], x[14, 21], x[15, 22] = np.inf, -np.inf, np.nan
    x[16, :] = np.nan
    x[17, 200] = np.float32(2.0 ** -133)
    check_quantize(torch, g, as_type(torch, x, dtype), "e4m3", square)
    check_quantize(torch, g, as_type(torch, x, dtype), "e5m2", square)


def test_quantize_writes_only_its_columns(env):
    torch, g = env
    x = as_type(torch, values(70, 100, 5), "f32")
    buf = torch.full((70, 112), 0x5A, dtype=torch.uint8, device="cuda")
    q = buf.view(torch.float8_e4m3fn)[:, :100]
    s = torch.empty((1, 70, 4), dtype=torch.uint8, device="cuda")
    bt = torch.full((100, 80), 0x5A, dtype=torch.uint8, device="cuda")
    st = torch.empty((1, 100, 4), dtype=torch.uint8, device="cuda")
    g.gar_fp8_quantize(x, q, s, bt.view(torch.float8_e4m3fn)[:, :70], st)
    assert (buf[:, 100:] == 0x5A).all() and (bt[:, 70:] == 0x5A).all()


# ------------------------------------------------------------------- product
def operand(torch, g, rows, cols, fmt, seed, scale=1.0, square=False):
    x = torch.from_numpy(values(rows, cols, seed) * np.float32(scale)).cuda()
    q, s = g.fp8_matrix(rows, cols, fp8(torch, fmt))
    g.gar_fp8_quantize(x, q, s, square=square)
    return q, s


def decoded(torch, q, s):
    rows, cols = q.shape
    b = s.permute(1, 0, 2).reshape(rows, -1)[:, :(cols + 127) // 128].double()
    return q.double() * torch.exp2(b - 127).repeat_interleave(128, 1)[:, :cols]


def check_product(torch, q, s, r, t, d, c=None):
    a, b = decoded(torch, q, s), decoded(torch, r, t)
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    if c is not None:
        want, size = want + c.double(), size + c.double().abs()
    K = q.shape[1]
    tol = (K / 32 + 8) * 2.0 ** -22 * size + want.abs() * (2.0 ** -8 if d.dtype == torch.bfloat16 else 2.0 ** -23) + 1e-37
    off = (d.double() - want).abs()
    assert bool((off <= tol).all()), f"{int((off > tol).sum())} of {off.numel()} off, worst {(off / tol).max().item():.3g}"


SHAPES = [(1, 1, 1), (1, 8, 128), (1, 4096, 512), (5, 130, 129), (16, 1024, 2048), (31, 257, 384), (32, 128, 640),
          (33, 300, 512), (64, 64, 1000), (65, 100, 1536), (100, 200, 5000), (129, 129, 129), (256, 520, 256),
          (300, 1000, 700), (1003, 333, 1000), (2049, 17, 511), (2300, 2333, 300), (4100, 1300, 640)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_matmul(env, m, n, k, dtype):
    torch, g = env
    fa, fb = ("e4m3", "e5m2") if (m + n) % 3 == 0 else ("e5m2", "e4m3") if (m + n) % 3 == 1 else ("e4m3", "e4m3")
    (q, s), (r, t) = operand(torch, g, m, k, fa, 11), operand(torch, g, n, k, fb, 12, 0.1, square=True)
    out = torch.float32 if dtype == "f32" else torch.bfloat16
    d = torch.full((m, n), 7.0, dtype=out, device="cuda")
    g.gar_fp8_matmul(q, s, r, t, d)
    check_product(torch, q, s, r, t, d)
    c = torch.randn((m, n), device="cuda").to(out)
    g.gar_fp8_matmul(q, s, r, t, d, c=c)
    check_product(torch, q, s, r, t, d, c)
    acc = c.clone()
    g.gar_fp8_matmul(q, s, r, t, acc, c=acc)  # in place: the same bits
    assert torch.equal(acc, d)
    assert g.gar_sync_status() == 0


@pytest.mark.parametrize("k", [8192 + 128, 20000])
@pytest.mark.parametrize("m,n", [(40, 300), (2500, 2400)])
def test_matmul_long_sums(env, m, n, k):
    """Sums over many k: within 1e-6 of the result in the mean, as in short ones."""
    torch, g = env
    (q, s), (r, t) = operand(torch, g, m, k, "e4m3", 13, square=True), operand(torch, g, n, k, "e4m3", 14, square=True)
    d = torch.empty((m, n), device="cuda")
    g.gar_fp8_matmul(q, s, r, t, d)
    check_product(torch, q, s, r, t, d)
    want = decoded(torch, q, s) @ decoded(torch, r, t).t()
    assert ((d.double() - want).norm() / want.norm()).item() < 2e-6


@pytest.mark.parametrize("m,n", [(9, 50), (200, 70), (2400, 2310)])
def test_matmul_strides(env, m, n):
    """d and c inside wider matrices, at odd offsets; codes inside wider matrices; nothing else written."""
    torch, g = env
    k = 333
    (q0, s), (r0, t) = operand(torch, g, m, k, "e4m3", 15), operand(torch, g, n, k, "e4m3", 16)
    q = torch.zeros((m, 512), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, 16:16 + k]
    q.view(torch.uint8).copy_(q0.view(torch.uint8))
    for dt in (torch.float32, torch.bfloat16):
        big = torch.full((m + 2, n + 7), 3.0, dtype=dt, device="cuda")
        d = big[1:m + 1, 3:3 + n]
        c = torch.randn((m, n + 1), device="cuda").to(dt)[:, 1:]
        g.gar_fp8_matmul(q, s, r0, t, d, c=c)
        check_product(torch, q, s, r0, t, d, c)
        edge = big.clone()
        edge[1:m + 1, 3:3 + n] = 3.0
        assert (edge == 3.0).all()


def test_matmul_empty(env):
    torch, g = env
    q, s = g.fp8_matrix(4, 0)
    r, t = g.fp8_matrix(5, 0)
    c = torch.randn((4, 5), device="cuda")
    d = torch.full((4, 5), 9.0, device="cuda")
    g.gar_fp8_matmul(q, s, r, t, d)
    assert (d == 0).all()
    g.gar_fp8_matmul(q, s, r, t, d, c=c)
    assert torch.equal(d, c)
    q, s = g.fp8_matrix(0, 64)
    r, t = g.fp8_matrix(5, 64)
    g.gar_fp8_matmul(q, s, r, t, torch.empty((0, 5), device="cuda"))


@pytest.mark.parametrize("m,n", [(20, 40), (2400, 2400)])
def test_matmul_nan_stays_in_its_row_and_column(env, m, n):
    torch, g = env
    k = 512
    (q, s), (r, t) = operand(torch, g, m, k, "e4m3", 17), operand(torch, g, n, k, "e4m3", 18)
    q.view(torch.uint8)[3, 200] = 0x7F
    r.view(torch.uint8)[11, 7] = 0xFF
    d = torch.empty((m, n), device="cuda")
    g.gar_fp8_matmul(q, s, r, t, d)
    want = torch.zeros((m, n), dtype=torch.bool, device="cuda")
    want[3] = True
    want[:, 11] = True
    assert torch.equal(torch.isnan(d), want)


def test_matmul_exact_integers(env):
    """Small integers: the product is exact, and so are a linear layer's gradients against differences.

    f(W) = sum G o (X W^T): its derivative by one weight is the difference of f over one step of it."""
    torch, g = env
    rng = np.random.default_rng(19)
    T, N, K = 130, 40, 150
    X, W, G = (rng.integers(-4, 5, s).astype(np.float32) for s in ((T, K), (N, K), (T, N)))

    def both(x):
        t = torch.from_numpy(x).cuda()
        a, b = g.fp8_matrix(*x.shape), g.fp8_matrix(x.shape[1], x.shape[0])
        g.gar_fp8_quantize(t, *a, *b)
        return a, b

    (x, xt), (w, wt), (u, ut) = both(X), both(W), both(G)
    y, dw, dx = (torch.empty(s, device="cuda") for s in ((T, N), (N, K), (T, K)))
    g.gar_fp8_matmul(*x, *w, y)
    g.gar_fp8_matmul(*ut, *xt, dw)
    g.gar_fp8_matmul(*u, *wt, dx)
    np.testing.assert_array_equal(y.cpu().numpy(), X @ W.T)

    def f(X_, W_):
        return float((G.astype(np.float64) * (X_.astype(np.float64) @ W_.astype(np.float64).T)).sum())

    for i, j in ((0, 0), (39, 149), (17, 128)):
        E = np.zeros_like(W)
        E[i, j] = 1.0
        assert dw[i, j].item() == f(X, W + E) - f(X, W)
    for i, j in ((0, 0), (129, 149), (64, 127)):
        E = np.zeros_like(X)
        E[i, j] = 1.0
        assert dx[i, j].item() == f(X + E, W) - f(X, W)


def test_matmul_is_repeatable_and_follows_streams_and_graphs(env):
    torch, g = env
    for m, n, k in ((16, 512, 4096), (2400, 2400, 1024)):
        (q, s), (r, t) = operand(torch, g, m, k, "e4m3", 20), operand(torch, g, n, k, "e4m3", 21)
        d = [torch.empty((m, n), device="cuda") for _ in range(3)]
        g.gar_fp8_matmul(q, s, r, t, d[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g.gar_fp8_matmul(q, s, r, t, d[1], stream=side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g.gar_fp8_matmul(q, s, r, t, d[2])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d[0], d[1]) and torch.equal(d[0], d[2])


def test_offsets_beyond_32_bits(env):
    """More than 2^31 elements in x, its codes and the product."""
    torch, g = env
    m, n, k = 70000, 32768, 128
    x = torch.randn((m, n), device="cuda", dtype=torch.bfloat16)
    q, s = g.fp8_matrix(m, n)
    qt, st = g.fp8_matrix(n, m)
    g.gar_fp8_quantize(x, q, s, qt, st)
    tail = slice(m - 100, m)
    want, bytes_ = ref.quantize(x[tail, n - 300:].float().cpu().numpy()[:, 300 % 128:], "e4m3", False)
    np.testing.assert_array_equal(q[tail, n - 256:].float().cpu().numpy(), want)
    a = x[m - 112:].float()  # the last 112 rows are the columns' last block (70000 = 546 * 128 + 112)
    want, _ = ref.quantize(a[:, n - 50:].cpu().numpy().T, "e4m3", False)
    np.testing.assert_array_equal(qt[n - 50:, m - 112:].float().cpu().numpy(), want)
    del q, qt
    (q, s), (r, t) = operand(torch, g, 1, k, "e4m3", 22), operand(torch, g, n, k, "e4m3", 23)
    xs = x[:, :k].contiguous()
    q, s = g.fp8_matrix(m, k)
    g.gar_fp8_quantize(xs, q, s)
    g.gar_fp8_matmul(q, s, r, t, x)
    check_product(torch, q[m - 200:], s[:, m - 200:], r, t, x[m - 200:])


# rows that start anywhere in a line of 16 bytes, at both ends of the matrix and inside it
@pytest.mark.parametrize("rows,cols", [(8, 8), (130, 263), (257, 129), (64, 1031)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lead,pad", [(0, 0), (0, 1), (1, 0), (3, 2), (5, 3), (7, 9)])
def test_quantize_rows_that_start_anywhere(env, rows, cols, dtype, lead, pad):
    torch, g = env
    x = as_type(torch, values(rows, cols, 31), dtype)
    flat = torch.full((rows * (cols + lead + pad),), float("nan"), device="cuda", dtype=x.dtype)
    y = flat.view(rows, cols + lead + pad)[:, lead:lead + cols]
    y.copy_(x)
    check_quantize(torch, g, y, "e4m3", False)


def test_split_products_that_share_sms(env):
    """Two streams of products whose k is split over clusters, two CTAs an SM: the same results as one after another."""
    torch, g = env
    sizes = [(16, 4096, 2048), (33, 2000, 4096), (64, 1024, 8192), (5, 700, 3000)]
    ops = [(operand(torch, g, m, k, "e4m3", 31), operand(torch, g, n, k, "e4m3", 32)) for m, n, k in sizes]
    want = []
    for (m, n, _), (a, b) in zip(sizes, ops):
        want.append(torch.empty((m, n), device="cuda"))
        g.gar_fp8_matmul(*a, *b, want[-1])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.zeros_like(d) for d in want] for _ in streams]
    torch.cuda.synchronize()
    for i in range(50):
        for s, (stream, outs) in enumerate(zip(streams, got)):
            for j in (range(4) if s == 0 else (2, 0, 3, 1)):
                g.gar_fp8_matmul(*ops[j][0], *ops[j][1], outs[j], stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for outs in got for a, b in zip(outs, want)) and g.gar_sync_status() == 0


def product_error(torch, g, m, n, k, seed, addend):
    """Relative error, in the norm, of an fp32 product of values with a mean, whose sums grow with k."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def codes(rows):
        q, s = g.fp8_matrix(rows, k)
        g.gar_fp8_quantize(torch.randn((rows, k), generator=gen, device="cuda") + 0.5, q, s)
        return q, s

    a, b = codes(m), codes(n)
    want = decoded(torch, *a) @ decoded(torch, *b).t()
    d, c = torch.empty((m, n), device="cuda"), None
    if addend:
        c = torch.randn((m, n), generator=gen, device="cuda") * k ** 0.5
        want += c.double()
        d.copy_(c)
    g.gar_fp8_matmul(*a, *b, d, c=d if addend else None)  # the addend in place
    again = torch.empty_like(d)
    g.gar_fp8_matmul(*a, *b, again, c=c)
    assert torch.equal(d, again)
    return ((d.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("addend", [False, True])
@pytest.mark.parametrize("m,n,k", [(256, 2048, 65536), (16, 300, 262144), (100, 130, 100001), (70, 5000, 40000)])
def test_matmul_long_sums_of_few_tiles(env, m, n, k, addend):
    """An accumulator of the tensor core adds 8192 k at most, so that its error, which grows with them where the sum does,
    is that of a product with k = 8192 (one accumulator there: many tiles).  Beyond it, up to 32 parts are added in fp32
    to nearest: 2^-24 sqrt(1/3) sqrt(sum of (j / 32)^2) = 1.2e-7 in the mean square."""
    torch, g = env
    one = product_error(torch, g, 2560, 2400, 8192, 34, False)
    assert product_error(torch, g, m, n, k, 33, addend) <= 1.05 * one + 2.5e-7
