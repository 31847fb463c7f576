"""FP8 quantization with a scale for 128 values, products of quantized matrices and the linear layer.

Tolerances. Codes and scales are defined in fp32 arithmetic, one rounding an operation, and are equal bit for
bit; dequantized values are one rounded product (bf16: of the fp32 product, 2^-8 and 2^-24). In a product the
matrix unit cuts each of eight neighbouring products at 2^-13 of the largest one's power of two, which the
oracle's fp8_cut_product does alike; the 16 sums of eight of a block are joined in fp32 with 16 additions off by
2^-23 of the sum of magnitudes at most: 2^-19; the scales' product, and the fused multiply-add of each block,
add 2^-24 of it and of all blocks' sum. Against the product itself seven of eight may be cut by 2^-13 of
the largest, 7 2^-13 sum over eights of max |a w| <= 7 2^-13 sqrt(K / 8 sum (a w)^2) by Cauchy and Schwarz,
with the magnitude of a subnormal factor taken as the smallest normal one. Results in bf16 add 2^-8 of
themselves, in fp32 2^-24."""
import ctypes

import numpy as np
import pytest

from oracle import qgalore_oracle as O

torch = pytest.importorskip("torch")

BF16, FP32, INT8 = torch.bfloat16, torch.float32, torch.int8
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
DT = {"e4m3": E4M3, "e5m2": E5M2}


def B():
    from quantized_rank_gradient_amd import binding
    return binding


def f64(t):
    return t.detach().double().cpu().numpy()


def values(m, n, seed, dtype=FP32):
    """Rows and columns of different sizes, a row and a run of zeros, and entries of every size down to
    what a scale loses."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, n)) * np.exp(rng.standard_normal((1, n))) * 10.0 ** rng.uniform(-4, 4, (m, 1))
    x *= np.where(rng.random((m, n)) < 0.1, 10.0 ** rng.uniform(-8, 0, (m, n)), 1.0)
    if m > 2:
        x[1] = 0
    if n > 128:
        x[0, :128] = 0
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def int8_weights(m, n, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-127, 128, (m, n), generator=g, dtype=INT8)
    return q, (0.5 + torch.rand(-(-m * n // 256), generator=g)) * 1e-3


def weight32(q, s):
    m, n = q.shape
    return q.float() * s.repeat_interleave(256)[:m * n].view(m, n)


def codes64(Q, n):
    """Codes as values, and that the padding is zero."""
    v = Q.cpu().float().numpy().astype(np.float64)
    assert (v[:, n:] == 0).all()
    return v[:, :n]


def check_quantized(Q, S, x32, fmt, block):
    q, s = O.fp8_quantize(x32, fmt, block)
    m, n = x32.shape
    assert tuple(Q.shape) == (m, -(-n // 16) * 16) and Q.dtype == DT[fmt]
    assert np.array_equal(S.cpu().numpy(), s)
    assert np.array_equal(codes64(Q, n), q)


SIZES = [(1, 1), (1, 16), (3, 17), (2, 130), (127, 128), (128, 127), (129, 129), (128, 256), (200, 1000),
         (1, 5461), (1376, 40), (257, 512)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", [False, True])
def test_quantize(m, n, fmt, block):
    b = B()
    for dtype in (BF16, FP32):
        x = values(m, n, m + n, dtype)
        x32 = x.float().numpy()
        got = b.fp8_quantize(x.cuda(), fmt=fmt, block=block, columns=True)
        check_quantized(*got[:2], x32, fmt, block)
        check_quantized(*got[2:], np.ascontiguousarray(x32.T), fmt, block)
        for rows in (True, False):   # one order alone
            one = b.fp8_quantize(x.cuda(), fmt=fmt, block=block, rows=rows, columns=not rows)
            for p, q in zip(one, got[:2] if rows else got[2:]):
                assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", SIZES + [(130, 5461)])
def test_quantize_int8_weights(m, n):
    q, s = int8_weights(m, n, m)
    w = weight32(q, s).numpy()
    for block in (False, True):
        got = B().fp8_quantize(q.cuda(), scales=s.cuda(), block=block, columns=True)
        check_quantized(*got[:2], w, "e4m3", block)
        check_quantized(*got[2:], np.ascontiguousarray(w.T), "e4m3", block)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_every_finite_code_and_every_border_rounds_to_even(fmt):
    """All values of the format and the middles between neighbours, next to the largest one so that the
    scale is 1."""
    top = O.FP8_MAX[fmt]
    code = torch.arange(256, dtype=torch.uint8).view(DT[fmt]).float()
    v = torch.unique(code[torch.isfinite(code)])
    mid = (v[1:] + v[:-1]) / 2
    near = torch.cat([mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    x = torch.cat([v, mid, near])
    x = torch.cat([x, torch.zeros(-len(x) % 127)]).view(-1, 127)
    x = torch.cat([x, torch.full((len(x), 1), top)], 1).contiguous()
    Q, S = B().fp8_quantize(x.cuda(), fmt=fmt)
    assert (S == 1).all()
    assert np.array_equal(codes64(Q, 128), O.fp8_round(x.double().numpy(), fmt))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_tiny_huge_nan_and_infinity(fmt):
    x = torch.zeros(6, 256)
    x[0, :128] = 1e-40                    # below the smallest scale's reach
    x[1] = 2.0 ** -126
    x[2, 5], x[2, 6] = float("nan"), 3.0
    x[3, 200], x[3, 201] = -float("inf"), 1.0
    x[4] = torch.finfo(FP32).max
    Q, S, Qt, St = B().fp8_quantize(x.cuda(), fmt=fmt, columns=True)
    v = Q.cpu().float()
    assert (S > 0).all() and float(S[0, 5]) == 2.0 ** -126 and float(S[0, 0]) == 2.0 ** -126
    keep = [0, 1, 4, 5]
    q, s = O.fp8_quantize(x[keep].numpy(), fmt)
    assert np.array_equal(v[keep].double().numpy(), q) and np.array_equal(S[:, keep].cpu().numpy(), s)
    assert torch.isnan(v[2, 5]) and v[2, 6] == O.FP8_MAX[fmt] and torch.isnan(v[2]).sum() == 1
    assert torch.isinf(S[1, 3]) and torch.isnan(v[3, 200]) and v[3, 201] == 0
    d = B().fp8_dequantize(Q, S, 256, dtype=FP32).cpu()
    assert torch.isnan(d[3, 128:]).all() and (d[3, :128] == 0).all()
    assert torch.isnan(d).any(1).tolist() == [False, False, True, True, False, False]
    assert torch.isnan(Qt.cpu().float()[5, 2]) and not torch.isnan(Qt.cpu().float()[5, :2]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("block", [False, True])
def test_dequantize(m, n, block):
    b = B()
    for fmt in ("e4m3", "e5m2"):
        Q, S = b.fp8_quantize(values(m, n, 1).cuda(), fmt=fmt, block=block)
        exact = codes64(Q, n) * O.fp8_spread(S.cpu().numpy(), m, n)
        for dtype, eps in ((BF16, 2.0 ** -8 + 2.0 ** -23), (FP32, 2.0 ** -24)):
            got = b.fp8_dequantize(Q, S, n, block=block, dtype=dtype)
            assert got.dtype == dtype and tuple(got.shape) == (m, n)
            assert (np.abs(f64(got) - exact) <= eps * np.abs(exact) + 2.0 ** -133).all()


def operand(m, k, seed, fmt="e4m3", block=False):
    """A quantized matrix on the GPU, its codes and the scale of each in float64."""
    Q, S = B().fp8_quantize(values(m, k, seed).clamp(-1e3, 1e3).cuda(), fmt=fmt, block=block)
    return Q, S, (codes64(Q, k), O.fp8_spread(S.cpu().numpy(), m, k))


def near(got, a, w, fmt="e4m3", name=""):
    """got against the codes and scales a and w: to the plain product where the cuts allow for, and as the
    matrix unit forms it on all rows and columns of a small product, and on 40 of each of a large one."""
    (qa, sa), (qw, sw) = a, w
    K, eps = qa.shape[1], 2.0 ** -8 if got.dtype == BF16 else 2.0 ** -24
    got = f64(got)

    def check(got, want, err, what):
        bad = np.abs(got - want) > err + eps * (np.abs(want) + err) + 1e-37
        assert not bad.any(), (name, what, int(bad.sum()), float(np.abs(got - want)[bad].max()))
    add = 2.0 ** -19 + (-(-K // 128) + 2) * 2.0 ** -24

    def floor(q, low):
        return np.where(q == 0, 0, np.maximum(np.abs(q), low))
    low = 2.0 ** -6 if fmt == "e4m3" else 2.0 ** -14
    sq = (floor(qa, low) * sa) ** 2 @ ((floor(qw, 2.0 ** -6) * sw) ** 2).T
    mag = np.abs(qa * sa) @ np.abs(qw * sw).T
    check(got, (qa * sa) @ (qw * sw).T, 7 * 2.0 ** -13 * np.sqrt(-(-K // 8) * sq) + add * mag, "product")
    rng = np.random.default_rng(1)
    i, j = np.arange(len(qa)), np.arange(len(qw))
    if qa.size * len(qw) > 10_000_000:
        pick = lambda n: np.unique(np.r_[0, n - 1, rng.integers(0, n, 40)])  # noqa: E731
        i, j = pick(len(qa)), pick(len(qw))
    cut = O.fp8_cut_product(qa[i], sa[i], qw[j], sw[j], fmt)
    check(got[np.ix_(i, j)], cut, add * mag[np.ix_(i, j)], "cut product")


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 16, 128), (1, 17, 130), (2, 100, 5461), (15, 33, 16),
                                   (16, 1000, 1376), (17, 5, 3), (17, 129, 129), (31, 300, 512),
                                   (64, 64, 64), (65, 127, 1000), (128, 128, 128), (129, 257, 384),
                                   (200, 5461, 40), (1000, 1376, 512), (300, 40, 8000), (48, 4100, 264)])
@pytest.mark.parametrize("block", [False, True])
def test_matmul(M, N, K, block):
    b = B()
    for fmt in ("e4m3", "e5m2"):
        A, SA, a = operand(M, K, 1, fmt)
        Q, S, w = operand(N, K, 2, block=block)
        for dtype in (BF16, FP32):
            near(b.fp8_matmul(A, SA, Q, S, K, dtype=dtype), a, w, fmt, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(3000, 4100, 200), (2048, 6401, 136), (4097, 2900, 129)])
@pytest.mark.parametrize("block", [False, True])
def test_matmul_of_many_tiles(M, N, K, block):
    b = B()
    A, SA, a = operand(M, K, 1, "e5m2")
    Q, S, w = operand(N, K, 2, block=block)
    near(b.fp8_matmul(A, SA, Q, S, K), a, w, "e5m2")


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1500, 2070, 50), (2000, 1990, 130), (1700, 1900, 260), (1930, 1800, 700),
                                   (1921, 2048, 384), (450, 11000, 200), (385, 9990, 530)])
@pytest.mark.parametrize("block", [False, True])
def test_matmul_of_a_round_of_tiles(M, N, K, block):
    """About as many tiles of 128 as there are CUs, with a block of K or two, or more than are loaded ahead."""
    b = B()
    A, SA, a = operand(M, K, 1)
    Q, S, w = operand(N, K, 2, block=block)
    whole = torch.full((M * N + 128,), 7.0, dtype=BF16, device="cuda")
    out = b.fp8_matmul(A, SA, Q, S, K, out=whole[64:64 + M * N].view(M, N))
    near(out, a, w)
    assert (whole[:64] == 7).all() and (whole[64 + M * N:] == 7).all()
    wide = b.fp8_matmul(A, SA, Q, S, K, dtype=FP32)
    near(wide, a, w)
    for _ in range(3):
        assert torch.equal(wide, b.fp8_matmul(A, SA, Q, S, K, dtype=FP32))


PARTS = [(128, 64, 4096), (100, 130, 5461), (65, 63, 20000), (257, 129, 3000), (130, 1001, 8193),
         (400, 1376, 20000), (1000, 70, 11008), (70, 300, 60000), (513, 511, 9000)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", PARTS)
@pytest.mark.parametrize("block", [False, True])
def test_matmul_in_parts(M, N, K, block):
    """Few tiles and a long K: with a workspace the parts' sums go there and nowhere else, whatever it held
    (a NaN), and are added in order."""
    b = B()
    need = b.lib().qgalore_fp8_matmul_workspace_bytes(M, N, K)
    A, SA, a = operand(M, K, 1, "e5m2")
    Q, S, w = operand(N, K, 2, block=block)
    area = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    for dtype in (BF16, FP32):
        whole = torch.full((M * N + 128,), 7.0, dtype=dtype, device="cuda")
        out = whole[64:64 + M * N].view(M, N)
        b.fp8_matmul(A, SA, Q, S, K, dtype=dtype, out=out, workspace=area[256:256 + need])
        near(out, a, w, "e5m2", dtype)
        assert (whole[:64] == 7).all() and (whole[64 + M * N:] == 7).all()
        assert (area[:256] == 0xFF).all() and (area[256 + need:] == 0xFF).all()
        assert (area != 0xFF).any()
        assert torch.equal(out, b.fp8_matmul(A, SA, Q, S, K, dtype=dtype))
    out = torch.empty(M, N, dtype=BF16, device="cuda")
    desc = b.Fp8MmDesc(M, N, K, 1, int(block), 0, None, 0, torch.cuda.current_stream().cuda_stream)
    assert b.lib().qgalore_fp8_matmul(ctypes.byref(desc), A.data_ptr(), SA.data_ptr(), Q.data_ptr(),
                                      S.data_ptr(), out.data_ptr()) == 0
    near(out, a, w, "e5m2", "without a workspace")


@pytest.mark.gpu
@pytest.mark.parametrize("block", [False, True])
def test_matrices_of_nearly_2_31_bytes(block):
    """INT8 weights, bf16 values and a product's result up to the limit: the last rows, from a whole block and
    group on, are those of a call of their own."""
    b, m, at = B(), 32767, 32512   # 127 * 256
    g = torch.Generator("cuda").manual_seed(1)
    for n, dtype in ((65521, INT8), (32767, BF16)):
        scales = None
        if dtype == INT8:
            x = torch.randint(-127, 128, (m, n), generator=g, dtype=INT8, device="cuda")
            scales = torch.rand(-(-m * n // 256), generator=g, device="cuda") + 0.5
        else:
            x = torch.randn((m, n), generator=g, device="cuda", dtype=BF16)
        Q, S, Qt, St = b.fp8_quantize(x, scales=scales, block=block, columns=True)
        q, s, qt, st = b.fp8_quantize(x[at:].clone(), block=block, columns=True,
                                      scales=None if scales is None else scales[at * n // 256:].clone())
        assert torch.equal(Q[at:].view(torch.uint8), q.view(torch.uint8))
        assert torch.equal(Qt.view(torch.uint8)[:, at:], qt.view(torch.uint8))
        assert torch.equal(S[:, at // 128 if block else at:], s) and torch.equal(St[at // 128:], st)
        if dtype == BF16:
            v = b.fp8_dequantize(Q, S, n, block=block)
            assert torch.equal(v[at:], b.fp8_dequantize(q, s, n, block=block))
    del x, scales, Q, S, Qt, St, v
    n, K = 32767, 130
    A, SA = b.fp8_quantize(torch.randn((m, K), generator=g, device="cuda"))
    W, SW = b.fp8_quantize(torch.randn((n, K), generator=g, device="cuda"), block=block)
    out = b.fp8_matmul(A, SA, W, SW, K)
    part = b.fp8_matmul(A[at:].clone(), SA[:, at:].contiguous(), W, SW, K)
    assert torch.equal(out[at:], part)
    del out
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(1, 16), (8, 300), (16, 40), (17, 300), (64, 512), (200, 130)])
@pytest.mark.parametrize("block", [False, True])
def test_matmul_of_the_longest_k(M, N, block):
    """2^20 ones a row, with scales of small whole numbers: every sum is one, below 2^24, in any order."""
    K, b = 1 << 20, B()
    (qa, sa), (qb, sb) = b.fp8_shapes(M, K), b.fp8_shapes(N, K, block)
    A, W = (torch.ones(q, device="cuda").to(E4M3) for q in (qa, qb))
    k = torch.arange(K // 128, device="cuda")[:, None]
    SA = (1 + (k + torch.arange(M, device="cuda")) % 3).float()
    SB = (1 + (k + torch.arange(sb[1], device="cuda")) % 2).float()
    assert SA.shape == sa and SB.shape == sb
    want = 128 * (SA.double().T.cpu() @ SB.double().cpu())
    want = want[:, torch.arange(N) // 128] if block else want
    assert want.max() < 2 ** 24
    for dtype in (FP32, BF16):
        assert torch.equal(b.fp8_matmul(A, SA, W, SB, K, dtype=dtype).cpu(), want.to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(5, 70, 200), (100, 130, 200), (3000, 4100, 140)])
def test_nan_and_infinite_scales_stay_in_their_rows(M, N, K):
    b = B()
    A, SA, a = operand(M, K, 1)
    Q, S, w = operand(N, K, 2)
    clean = b.fp8_matmul(A, SA, Q, S, K)
    A.view(torch.uint8)[3, 10] = 0x7F
    SA[1, M - 1] = float("inf")
    Q.view(torch.uint8)[N - 2, 130] = 0xFF
    out = b.fp8_matmul(A, SA, Q, S, K)
    bad = torch.isnan(out)
    assert bad[3].all() and bad[:, N - 2].all()
    assert not torch.isfinite(out[M - 1]).all()
    ok = torch.ones(M, N, dtype=torch.bool, device="cuda")
    ok[3], ok[M - 1] = False, False
    ok[:, N - 2] = False
    assert torch.equal(out[ok], clean[ok])


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(7, 37, 300), (100, 129, 300), (3000, 4100, 140)])
def test_matmul_writes_its_result_alone_and_equal_bits(M, N, K):
    b = B()
    A, SA, _ = operand(M, K, 1)
    for block in (False, True):
        Q, S, _ = operand(N, K, 2, block=block)
        for dtype in (BF16, FP32):
            whole = torch.full((M * N + 128,), 7.0, dtype=dtype, device="cuda")
            out = whole[64:64 + M * N].view(M, N)
            b.fp8_matmul(A, SA, Q, S, K, dtype=dtype, out=out)
            assert (whole[:64] == 7).all() and (whole[64 + M * N:] == 7).all()
            for _ in range(3):
                assert torch.equal(out, b.fp8_matmul(A, SA, Q, S, K, dtype=dtype))


def layer(m, n, seed=5):
    """An FP8 weight made of INT8 weights, its transpose, and its values."""
    q, s = int8_weights(m, n, seed)
    W, S, Wt, St = B().fp8_quantize(q.cuda(), scales=s.cuda(), block=True, columns=True)
    return W, S, Wt, St, (codes64(W, n), O.fp8_spread(S.cpu().numpy(), m, n))


def quantized(x, fmt="e4m3"):
    q, s = O.fp8_quantize(x, fmt)
    return q, O.fp8_spread(s, *x.shape)


LAYERS = [(1, 64, 128), (2, 65, 129), (8, 40, 7000), (8, 40, 9000), (3, 136, 20000), (16, 1376, 512), (17, 1376, 512), (40, 300, 5461), (128, 512, 1376),
          (1000, 1376, 512), (333, 1000, 264), (1, 4096, 11008), (3000, 4200, 200), (100, 200, 5000),
          (5000, 200, 300), (4000, 4000, 40)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,m,n", LAYERS)
def test_linear(T, m, n):
    b = B()
    W, S, Wt, St, w = layer(m, n)
    x, dy = values(T, n, 3, BF16), values(T, m, 4, BF16)
    x32, dy32 = x.float().numpy(), dy.float().numpy()
    near(b.fp8_linear_fwd(x.cuda(), W, S), quantized(x32), w, name="Y")
    Xt, Sx = b.fp8_quantize(x.cuda(), rows=False, columns=True)
    for fmt in ("e4m3", "e5m2"):
        dX, G = b.fp8_linear_bwd(dy.cuda(), Wt, St, Xt, Sx, fmt=fmt)
        near(dX, quantized(dy32, fmt), (w[0].T, w[1].T), fmt, "dX")
        near(G, quantized(np.ascontiguousarray(dy32.T), fmt), quantized(np.ascontiguousarray(x32.T)), fmt, "G")
        one, none = b.fp8_linear_bwd(dy.cuda(), Wt, St, fmt=fmt)
        assert none is None and torch.equal(one, dX)
        none, one = b.fp8_linear_bwd(dy.cuda(), Xt=Xt, Sx=Sx, fmt=fmt)
        assert none is None and torch.equal(one, G)


@pytest.mark.gpu
def test_linear_equals_its_parts():
    """The layer's products are those of its quantized operands, for few tokens too, whose quantization
    goes on in the product."""
    b = B()
    for T in (1, 5, 8, 9, 16, 17, 33, 64, 65, 100):
        W, S, Wt, St, _ = layer(200, 1000)
        x = values(T, 1000, T, BF16).cuda()
        Q, SQ = b.fp8_quantize(x)
        assert torch.equal(b.fp8_linear_fwd(x, W, S), b.fp8_matmul(Q, SQ, W, S, 1000))


@pytest.mark.gpu
def test_linear_gradients_against_differences():
    """With operands that quantize without a rounding and products that are not cut (7 2^k up to 448, the
    smallest product 2^6 49) the layer is the plain product but for the rounding to bf16, and its gradients
    are those of sum(Y dY), by central differences."""
    b = B()
    T, m, n = 20, 24, 136
    rng = np.random.default_rng(3)

    def exact(r, c):
        v = 7.0 * 2.0 ** rng.integers(3, 7, (r, c)) * rng.choice([-1, 0, 1], (r, c))
        v[:, ::127], v[::127] = 448.0, 448.0   # in every run of a row and of a column
        return v
    x, dy, w = exact(T, n), exact(T, m), exact(m, n)

    def gpu(v, dt=BF16):
        return torch.from_numpy(v.astype(np.float32)).to(dt).cuda()
    W, S, Wt, St = b.fp8_quantize(gpu(w), block=True, columns=True)
    Y = b.fp8_linear_fwd(gpu(x), W, S)
    assert (np.abs(f64(Y) - x @ w.T) <= 2.0 ** -8 * np.abs(x @ w.T)).all()
    Xt, Sx = b.fp8_quantize(gpu(x), rows=False, columns=True)
    dX, G = b.fp8_linear_bwd(gpu(dy), Wt, St, Xt, Sx, fmt="e4m3")

    def loss(x, w):
        return (x @ w.T * dy).sum()
    for got, v, f in ((dX, x, lambda d: loss(x + d, w) - loss(x - d, w)),
                      (G, w, lambda d: loss(x, w + d) - loss(x, w - d))):
        for _ in range(4):
            d = rng.integers(-2, 3, v.shape).astype(np.float64)
            err = 2.0 ** -7.9 * np.abs(f64(got) * d).sum()
            assert abs(f(d) / 2 - (f64(got) * d).sum()) <= err


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 130])
def test_linear_captured_and_replayed_on_another_stream(T):
    b = B()
    W, S, Wt, St, _ = layer(264, 300)
    x, dy = values(T, 300, 1, BF16).cuda(), values(T, 264, 2, BF16).cuda()

    def both(stream=None):
        Xt, Sx = b.fp8_quantize(x, rows=False, columns=True, stream=stream)
        return [b.fp8_linear_fwd(x, W, S, stream=stream),
                *b.fp8_linear_bwd(dy, Wt, St, Xt, Sx, stream=stream)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = both()
    s = torch.cuda.Stream()
    for k in range(4):
        x.copy_(values(T, 300, 20 + k, BF16))
        dy.copy_(values(T, 264, 30 + k, BF16))
        graph.replay()
        s.wait_stream(torch.cuda.current_stream())
        want = both(s)
        torch.cuda.synchronize()
        for p, q in zip(got, want):
            assert torch.equal(p, q)


@pytest.mark.gpu
def test_products_in_parts_captured_beside_eager_ones_with_other_workspaces():
    """Two graphs and eager calls, each with a workspace of its own, in turn and on two streams at once."""
    b = B()
    T, m, n = 130, 264, 5000
    W, S, _, _, _ = layer(m, n)
    x = values(T, n, 1, BF16).cuda()
    need = b.lib().qgalore_fp8_linear_fwd_workspace_bytes(T, m, n)
    areas = [torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for k in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[k]):
            got.append(b.fp8_linear_fwd(x, W, S, workspace=areas[k]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(4):
        x.copy_(values(T, n, 40 + k, BF16))
        torch.cuda.synchronize()
        want = b.fp8_linear_fwd(x, W, S, workspace=areas[2])
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        again = b.fp8_linear_fwd(x, W, S, workspace=areas[2])
        torch.cuda.synchronize()
        assert torch.equal(got[0], want) and torch.equal(got[1], want) and torch.equal(again, want)


# ---------------------------------------------------------------------- on the CPU ---
def test_oracle_rounds_as_torch_does():
    rng = np.random.default_rng(1)
    for fmt, top in O.FP8_MAX.items():
        y = rng.standard_normal(20000) * 10.0 ** rng.uniform(-9, 2, 20000)
        y = np.clip(y, -top, top).astype(np.float32)
        want = torch.from_numpy(y).to(DT[fmt]).double().numpy()
        assert np.array_equal(O.fp8_round(y, fmt), want)


FAKE, FAR = 0x10000, 1 << 33


def at(k):
    return FAKE + FAR * k


def quant(d=None, src=at(0), ws=None, Q=at(1), S=at(2), Qt=at(3), St=at(4), **kw):
    b = B()
    desc = b.Fp8Desc(40, 200, 0, 0, 0, None)
    for k, v in kw.items():
        setattr(desc, k, v)
    return b.lib().qgalore_fp8_quantize(ctypes.byref(desc), src, ws, Q, S, Qt, St)


def dequant(Q=at(1), S=at(2), out=at(3), **kw):
    b = B()
    desc = b.Fp8Desc(40, 200, 0, 0, 0, None)
    for k, v in kw.items():
        setattr(desc, k, v)
    return b.lib().qgalore_fp8_dequantize(ctypes.byref(desc), Q, S, out)


def matmul(A=at(0), SA=at(1), Bq=at(2), SB=at(3), out=at(4), **kw):
    b = B()
    desc = b.Fp8MmDesc(40, 60, 200, 0, 0, 0, None, 0, None)
    for k, v in kw.items():
        setattr(desc, k, v)
    return b.lib().qgalore_fp8_matmul(ctypes.byref(desc), A, SA, Bq, SB, out)


def linear(fwd, X=at(0), W=at(1), S=at(2), Xt=at(3), Sx=at(4), Y=at(5), G=at(6), **kw):
    b = B()
    desc = b.Fp8LinearDesc(40, 60, 200, 1, at(7), 1 << 30, None)
    for k, v in kw.items():
        setattr(desc, k, v)
    if fwd:
        return b.lib().qgalore_fp8_linear_fwd(ctypes.byref(desc), X, W, S, Y)
    return b.lib().qgalore_fp8_linear_bwd(ctypes.byref(desc), X, W, S, Xt, Sx, Y, G)


def test_fp8_refusals_come_before_any_device_call():
    gpu = torch.cuda.is_available()
    for k in ("src", "Q", "S", "Qt", "St"):
        assert quant(**{k: None}) == 1, k
    assert quant(Q=None, S=None, Qt=None, St=None) == 1
    assert quant(source=2) == 1 and quant(ws=at(5)) == 1    # INT8 weights and scales go together
    for k in ("src", "Q", "Qt"):
        assert quant(**{k: at(9) + 8}) == 3, k
    for k in ("S", "St"):
        assert quant(**{k: at(9) + 2}) == 3, k
    for k in ("Q", "S", "out"):
        assert dequant(**{k: None}) == 1 and dequant(**{k: at(9) + 2}) == 3, k
    for bad in (dict(rows=0), dict(cols=0), dict(rows=-3), dict(rows=1 << 20, cols=1 << 11),
                dict(rows=1 << 30, cols=1), dict(rows=1 << 29, cols=8),
                dict(rows=1 << 62, cols=1 << 62)):
        assert quant(**bad) == 2 and dequant(**bad) == 2, bad
    for bad in (dict(format=2), dict(format=-1), dict(block=2), dict(source=3)):
        assert quant(**bad) == 5 and dequant(**bad) == 5, bad
    assert dequant(source=2) == 5
    for k in ("A", "SA", "Bq", "SB", "out"):
        assert matmul(**{k: None}) == 1 and matmul(**{k: at(9) + 2}) == 3, k
    for bad in (dict(M=0), dict(N=0), dict(K=0), dict(K=(1 << 20) + 1), dict(M=1 << 20, N=1 << 12),
                dict(M=-1), dict(M=1 << 40, N=1 << 40)):
        assert matmul(**bad) == 2, bad
    for bad in (dict(a_format=2), dict(b_block=2), dict(out_dtype=2)):
        assert matmul(**bad) == 5, bad
    for k in ("X", "W", "S", "Y"):
        assert linear(True, **{k: None}) == 1 and linear(True, **{k: at(9) + 2}) == 3, k
    for k in ("X", "W", "S", "Xt", "Sx"):
        assert linear(False, **{k: None}) == 1, k
    for k in ("X", "W", "S", "Xt", "Sx", "Y", "G"):
        assert linear(False, **{k: at(9) + 2}) == 3, k
    assert linear(False, Y=None, G=None) == 1
    for f in (True, False):
        for bad in (dict(T=0), dict(m=0), dict(n=0), dict(T=1 << 40), dict(n=(1 << 20) + 1, T=1, m=1)):
            assert linear(f, **bad) == 2, bad
        assert linear(f, workspace=None) == 1 and linear(f, workspace=at(7) + 8) == 3
        assert linear(f, workspace_bytes=64) == 4
    assert linear(False, format=2) == 5
    if not gpu:
        assert quant() == 7 and dequant() == 7 and matmul() == 7
        assert quant(source=2, ws=at(5)) == 7 and quant(Qt=None, St=None) == 7
        assert linear(True) == 7 and linear(False) == 7
        assert linear(True, T=8, workspace=None, workspace_bytes=0) == 7
        assert linear(False, Y=None, W=None, S=None) == 7 and linear(False, G=None, Xt=None, Sx=None) == 7


def test_fp8_results_over_what_a_call_reads_are_refused():
    for out, size in (("Q", 40 * 208), ("S", 4 * 2 * 40), ("Qt", 200 * 48), ("St", 4 * 200)):
        p = dict(src=at(0), Q=at(1), S=at(2), Qt=at(3), St=at(4))
        for k in p:
            if k != out:
                assert quant(**{**p, k: p[out] + (size - 16)}) == 5, (out, k)
    assert quant(source=2, ws=at(1) + 16) == 5
    assert dequant(out=at(1) + 16) == 5 and dequant(out=at(2) + 16) == 5
    for k in range(4):
        assert matmul(out=at(k) + 16) == 5, k
    for k in (0, 1, 2):
        assert linear(True, Y=at(k)) == 5 and linear(True, workspace=at(k)) == 5, k
    assert linear(True, Y=at(7) + 64) == 5
    for k in range(5):
        for o in ("Y", "G", "workspace"):
            assert linear(False, **{o: at(k)}) == 5, (k, o)
    assert linear(False, Y=at(6) + 16) == 5 and linear(False, G=at(7) + 64) == 5


def test_fp8_matmul_workspace():
    L = B().lib()
    q = L.qgalore_fp8_matmul_workspace_bytes
    assert q(16, 4096, 11008) == 0 and q(64, 4096, 896) == 0 and q(0, 1, 1) == 0 and q(-1, 5, 9) == 0
    assert q(64, 4096, 897) == q(64, 4096, 1 << 18) == 8 * 64 * 4096 * 4
    assert q(17, 3, 1025) == 8 * 52 * 4
    assert q(4096, 4096, 4096) == 16 << 20 and q(1 << 14, 1 << 15, 1025) == 16 << 20
    big = dict(K=2000, workspace=at(9), workspace_bytes=8 * 40 * 60 * 4)
    assert matmul(**{**big, "workspace": at(9) + 8}) == 3
    assert matmul(**{**big, "workspace_bytes": big["workspace_bytes"] - 1}) == 4
    for k in range(5):
        assert matmul(**{**big, "workspace": at(k) + 16}) == 5, k
        if k > 0:
            assert matmul(**{**big, "workspace": at(k) - big["workspace_bytes"] + 16}) == 5, k
    if not torch.cuda.is_available():
        assert matmul(**big) == 7 and matmul(K=2000) == 7
        assert matmul(workspace=at(9), workspace_bytes=0) == 7      # none is needed


def test_fp8_workspaces_never_fall_as_tokens_come():
    L = B().lib()
    for m, n in ((64, 64), (1376, 512), (300, 5461)):
        for q in (L.qgalore_fp8_linear_fwd_workspace_bytes, L.qgalore_fp8_linear_bwd_workspace_bytes):
            sizes = [q(T, m, n) for T in (1, 2, 15, 16, 17, 18, 100, 127, 128, 129, 1000, 4096)]
            assert sizes == sorted(sizes)
            assert q(0, m, n) == 0 and q(1 << 40, m, n) == 0
        assert L.qgalore_fp8_linear_fwd_workspace_bytes(8, m, n) == 0


def test_fp8_binding_refuses_other_calls():
    b = B()
    x = torch.zeros(4, 32)
    for kw in (dict(X=x.half()), dict(X=x.double())):
        with pytest.raises(TypeError):
            b.fp8_quantize(**kw)
    for kw in (dict(X=x, scales=torch.ones(1)), dict(X=x.to(INT8)), dict(X=x, rows=False),
               dict(X=x, fmt="e3m4"), dict(X=x)):
        with pytest.raises(ValueError):
            b.fp8_quantize(**kw)
    with pytest.raises(TypeError):
        b.fp8_dequantize(x, torch.ones(1, 4), 32)
    with pytest.raises(ValueError):
        b.fp8_linear_bwd(x, Wt=x)
    with pytest.raises(ValueError):
        b.fp8_linear_bwd(x)


def test_fp8_struct_layouts_match_the_header(tmp_path):
    from tests.test_gpu_resnorm import layouts
    b = B()
    layouts(tmp_path, {"qg_fp8_desc": b.Fp8Desc, "qg_fp8_mm_desc": b.Fp8MmDesc,
                       "qg_fp8_linear_desc": b.Fp8LinearDesc})
